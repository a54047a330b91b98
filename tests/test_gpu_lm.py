"""Blocks with positions and dropout, and the token head: the operators in a run, as a
language model has them.

Each operator is compared with the oracle on the inputs that the run gave it, at that
operator's own bounds (test_gpu_rope, test_gpu_logp, block_util); the TT layers have
tests of their own."""

import numpy as np
import pytest

from block_util import NORM_TOL, TOL as ATTN_TOL, assert_near
from oracle import block_oracle as B
from oracle import token_oracle as K
from oracle import tt_oracle as O
from parity_util import TOL
from tensor_train_compressed_tt_gb300 import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_block import FORWARD  # noqa: E402
from test_gpu_logp import _check_fwd, _check_grad  # noqa: E402
from test_gpu_rope import _bound_fwd  # noqa: E402
from token_util import f64, within  # noqa: E402

HEADS, DIM, N = 12, 64, 768
HEAD_IN, HEAD_OUT = (12, 8, 8), (16, 16, 20)
EPS, P = 1e-5, 0.1


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from tensor_train_compressed_tt_gb300 import _build
    _build.build()


def _block_params(seed):
    inp = synth.draw_encoder(1, seed)
    r = np.random.default_rng(seed)
    params = {n: torch.from_numpy(synth.pack(li.cores, li.diags)).cuda()
              for n, li in inp.layers.items()}
    for n in ("g1", "b1", "g2", "b2"):
        params[n] = torch.from_numpy(r.uniform(0.5, 1.5, N).astype(np.float32)).cuda()
    for n in ("gq", "gk"):
        params[n] = torch.from_numpy(r.uniform(0.5, 1.5, DIM).astype(np.float32)).cuda()
    return params


def _head(vocab, seed, **kw):
    from tensor_train_compressed_tt_gb300 import ttc
    from tensor_train_compressed_tt_gb300.encoder import TTTokenHead
    r = np.random.default_rng(seed)
    ranks = ttc.tt_default_ranks(HEAD_IN, HEAD_OUT, 30)
    head = TTTokenHead(HEAD_IN, HEAD_OUT, ranks, vocab, **kw)
    shape = synth.LayerShape(HEAD_IN, HEAD_OUT, tuple(ranks))
    cores = [(0.3 * r.standard_normal(s)).astype(np.float32) for s in shape.core_shapes()]
    diags = [r.uniform(0.5, 1.5, n).astype(np.float32) for n in shape.diag_sizes()]
    params = {"head": torch.from_numpy(synth.pack(cores, diags)).cuda(),
              "gf": torch.from_numpy(r.uniform(0.5, 1.5, N).astype(np.float32)).cuda(),
              "bf": torch.from_numpy(r.uniform(-0.5, 0.5, N).astype(np.float32)).cuda()}
    return head, params, ([c.astype(np.float64) for c in cores],
                          [d.astype(np.float64) for d in diags])


def _setup(lens, seed, dropout=P, blocks=2, vocab=5000, **window):
    from tensor_train_compressed_tt_gb300.encoder import TTTransformerBlock
    from tensor_train_compressed_tt_gb300.layer import TTRotary, TTSeqs
    T = sum(lens)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    seqs = TTSeqs.packed(torch.from_numpy(off).cuda(), T, max(lens))
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    rotary = TTRotary(HEADS, DIM, eps=EPS)
    blks = [TTTransformerBlock(HEADS, rotary=rotary, dropout=dropout, site=2 * i, **window)
            for i in range(blocks)]
    params = [_block_params(seed + i) for i in range(blocks)]
    head, hp, hl = _head(vocab, seed + 9, dropout=dropout, site=2 * blocks)
    r = np.random.default_rng(seed)
    x = torch.from_numpy(r.standard_normal((T, N)).astype(np.float32)).cuda().bfloat16()
    t = r.integers(0, vocab, T)
    t[::7] = -1
    return dict(T=T, seqs=seqs, pos=torch.from_numpy(pos).cuda(), blks=blks, params=params,
                head=head, hp=hp, hl=hl, x=x, targets=torch.from_numpy(t.astype(np.int32)).cuda(),
                dlogp=torch.full((T,), -1.0 / T, device="cuda"),
                spans=[(a, e, a, e) for a, e in zip(off[:-1], off[1:])],
                bufs=[blk.buffers(T, seqs) for blk in blks], hb=head.buffers(T))


def _step(m, rng):
    """One training step of the whole model."""
    x, res = m["x"], None
    for blk, p, b in zip(m["blks"], m["params"], m["bufs"]):
        x, res = blk.forward(x, res, m["seqs"], p, b, pos=m["pos"], rng=rng)
    logp, dx, dres = m["head"].step(x, res, m["targets"], m["dlogp"], m["hp"], m["hb"], rng=rng)
    ins = [(m["x"], None)] + [(b["y_ffn"], b["s2"]) for b in m["bufs"][:-1]]
    for blk, p, b, (xi, ri) in reversed(list(zip(m["blks"], m["params"], m["bufs"], ins))):
        got = blk.backward(xi, ri, dx, dres, m["seqs"], p, b, pos=m["pos"], rng=rng)
        dx, dres = got if rng is not None else (got, got)
    return logp, dx


def _results(m):
    # dx_o belongs to the TT layers' own step
    keep = lambda b: {k: t for k, t in b.items()  # noqa: E731
                      if not k.startswith("ws_") and k not in ("dx_o", "entropy")}
    return [keep(b) for b in m["bufs"]] + [keep(m["hb"])]


@pytest.mark.parametrize("lens,window,vocab", [((65, 1, 30), dict(right=0), 5000),
                                               ((40, 17), dict(left=9, right=0, sinks=2), 5120)])
def test_training_step_against_oracle(lens, window, vocab):
    from tensor_train_compressed_tt_gb300.layer import TTDropout
    m = _setup(lens, 60, vocab=vocab, **window)
    T, seed, offset = m["T"], 77, 5
    rng = TTDropout.state(seed, offset)
    # the logits before their gradient takes their place
    logits = []
    real = m["head"].probs.loss

    def loss(x, *a, **k):
        logits.append(x.clone())
        return real(x, *a, **k)

    m["head"].probs.loss = loss
    logp, dx = _step(m, rng)
    torch.cuda.synchronize()
    f, pos, tol, atol = K.rope_freqs(DIM), m["pos"].cpu().numpy(), NORM_TOL["bf16"], \
        ATTN_TOL["bf16"]
    heads = lambda a: a.reshape(T, HEADS, DIM)  # noqa: E731
    keep = lambda site: K.drop_factor((T, N), P, seed, offset, site)  # noqa: E731
    x, res = f64(m["x"]), 0.0
    outs = []
    for i, (p, b) in enumerate(zip(m["params"], m["bufs"])):
        v, w = {k: f64(t) for k, t in b.items() if not k.startswith("ws_")}, \
            {k: f64(p[k]) for k in ("g1", "b1", "g2", "b2", "gq", "gk")}
        h, s, _ = B.norm_forward(x * keep(2 * i), w["g1"], w["b1"], res + 0 * x)
        assert_near(v["s1"], s, tol, "s1")
        assert O.rel_err(v["h1"], h) <= 2 * tol
        for n in "qk":
            ref = K.rope_forward(heads(v["y_" + n]), pos, f, DIM, w["g" + n], EPS)
            within(heads(v["r" + n]), ref, _bound_fwd(ref, DIM, "bf16"), "r" + n)
        q, k, val = heads(v["rq"]), heads(v["rk"]), heads(v["y_v"])
        assert_near(heads(v["att"]), B.attn_forward(q, k, val, m["spans"], **window)[0], atol,
                    "attention")
        h, s, _ = B.norm_forward(v["y_o"] * keep(2 * i + 1), w["g2"], w["b2"], v["s1"])
        assert_near(v["s2"], s, tol, "s2")
        outs.append((v, w))
        x, res = v["y_ffn"], v["s2"]
    hv = {k: f64(t) for k, t in m["hb"].items() if not k.startswith("ws_")}
    hw = {k: f64(m["hp"][k]) for k in ("gf", "bf")}
    h, s, _ = B.norm_forward(x * keep(4), hw["gf"], hw["bf"], res)
    assert_near(hv["s"], s, tol, "head: s")
    lg = logits[0]
    assert O.rel_err(f64(lg), O.chained_forward(*m["hl"], 3, hv["h"])[:, :vocab]) <= TOL["bf16"]
    t = m["targets"].cpu().numpy()
    _check_fwd(lg, t, 1.0, 0, (logp, m["hb"]["lse"], None))
    _check_grad(lg, t, f64(m["dlogp"]), None, 1.0, "bf16", m["hb"]["dlogits"][:, :vocab],
                "dlogits")
    if vocab < 5120:
        assert float(m["hb"]["dlogits"][:, vocab:].float().abs().max()) == 0
    rdh, rdc, _ = O.chained_backward(*m["hl"], 3, hv["h"], hv["dlogits"])
    assert O.rel_err(hv["dh"], rdh) <= TOL["bf16"]
    shape = synth.LayerShape(HEAD_IN, HEAD_OUT, tuple(m["head"].linear.ranks))
    for got, ref in zip(synth.unpack(shape, m["hb"]["dp_head"].cpu().numpy())[0], rdc):
        assert O.rel_err(got, ref) <= TOL["bf16"]
    ds, dg, db = B.norm_backward(hv["s"], hv["dh"], hw["gf"])
    assert_near(hv["ds"], ds, tol, "head: ds")
    assert_near(hv["dx"], ds * keep(4), tol, "head: dx")
    assert O.rel_err(hv["dgf"], dg) <= tol and O.rel_err(hv["dbf"], db) <= tol
    # the blocks backward, on what each was given
    dffn, ds2 = hv["dx"], hv["ds"]
    for i in (1, 0):
        v, w = outs[i]
        ds, dg, db = B.norm_backward(v["s2"], v["dx_ffn"], w["g2"], ds2)
        assert_near(v["ds2"], ds, tol, "ds2")
        assert_near(v["da"], ds * keep(2 * i + 1), tol, "da")
        assert O.rel_err(v["dg2"], dg) <= tol and O.rel_err(v["db2"], db) <= tol
        q, k, val = heads(v["rq"]), heads(v["rk"]), heads(v["y_v"])
        d = B.attn_backward(q, k, val, heads(v["datt"]), m["spans"], **window)
        assert_near(heads(v["dv"]), d[2], atol, "dv")
        for n, g in zip("qk", d):
            # dq in front of the rotation is not kept: the oracle's through both
            rx, rg = K.rope_backward(heads(v["y_" + n]), g, pos, f, DIM, w["g" + n], EPS)
            assert O.rel_err(heads(v["d" + n]), rx) <= atol + tol
            assert O.rel_err(v["dg" + n], rg) <= 2 * atol
        ds, dg, db = B.norm_backward(v["s1"], v["dx_qkv"], w["g1"], v["ds2"])
        assert_near(v["ds1"], ds, tol, "ds1")
        assert_near(v["dx"], ds * keep(2 * i), tol, "dx")
        assert O.rel_err(v["dg1"], dg) <= tol and O.rel_err(v["db1"], db) <= tol
        dffn, ds2 = v["dx"], v["ds1"]
    assert torch.equal(dx, m["bufs"][0]["dx"])


def test_steps_in_a_graph_are_the_eager_ones():
    """Captured with the offset's step: each replay drops other elements, the same ones
    as an eager step at that offset."""
    from tensor_train_compressed_tt_gb300.layer import TTDropout
    m = _setup((50, 33), 61, right=0)
    rng = TTDropout.state(3)
    _step(m, rng)  # the kernels' set-up
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _step(m, rng)
        rng[1] += 1
    seen = []
    for k in range(2):
        g.replay()
        torch.cuda.synchronize()
        got = [{n: t.clone() for n, t in b.items()} for b in _results(m)]
        _step(m, TTDropout.state(3, k))
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, _results(m))):
            for n in a:
                if n.startswith("dp_"):  # sums over tokens by reductions in any order
                    assert O.rel_err(f64(a[n]), f64(b[n])) <= TOL["bf16"], (i, n)
                else:
                    assert torch.equal(a[n], b[n]), (i, n)
        seen.append(got[0]["s1"])
    assert int(rng[1]) == 2 and not torch.equal(*seen)


def test_without_dropout_the_plain_block_runs():
    """rng=None: nothing is dropped, and the block's own capture takes positions."""
    m = _setup((30, 12), 62, blocks=1, right=0)
    blk, p, b = m["blks"][0], m["params"][0], m["bufs"][0]
    ds2 = torch.randn_like(m["x"])
    blk.step(m["x"], None, m["x"], ds2, m["seqs"], p, b, pos=m["pos"])
    names = ("y_ffn", "s2", "ds1", "dgq", "dgk", "dg1", "db2")
    want = {k: b[k].clone() for k in names}
    torch.cuda.synchronize()
    g = blk.capture(m["x"], None, m["x"], ds2, m["seqs"], p, b, pos=m["pos"])
    for k in names:
        b[k].zero_()
    g.replay()
    torch.cuda.synchronize()
    for k in names:
        assert torch.equal(b[k], want[k]), k
    # packed sequences: the distances alone count
    blk.forward(m["x"], None, m["seqs"], p, b)
    assert O.rel_err(f64(b["y_ffn"]), f64(want["y_ffn"])) <= FORWARD


@pytest.mark.parametrize("rows_type", [torch.int64, torch.int32])
def test_decode_continues_a_forward(rows_type):
    """The last token of each sequence by the cache, whose keys are the rotated ones."""
    from tensor_train_compressed_tt_gb300.layer import TTSeqs
    lens, room = (50, 1, 33), 64
    m = _setup(lens, 63, blocks=1, right=0)
    blk, p, b = m["blks"][0], m["params"][0], m["bufs"][0]
    y, s2 = blk.forward(m["x"], None, m["seqs"], p, b, pos=m["pos"])
    n = len(lens)
    keys = torch.full((n * room, HEADS, DIM), float("nan"), dtype=torch.bfloat16, device="cuda")
    values = keys.clone()
    last, rows = [], []
    for i, (a, e, _, _) in enumerate(m["spans"]):
        c = int(e - a) - 1
        keys[i * room:i * room + c] = b["rk"][a:a + c].view(c, HEADS, DIM)
        values[i * room:i * room + c] = b["y_v"][a:a + c].view(c, HEADS, DIM)
        last.append(int(e) - 1)
        rows.append(i * room + c)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    one = TTSeqs(i32(range(n)), i32(range(1, n + 1)), i32([i * room for i in range(n)]),
                 i32([r + 1 for r in rows]), n, n * room, 1, room)
    bd = blk.buffers(n, one)
    at = torch.tensor(rows, device="cuda").to(rows_type)
    with pytest.raises(ValueError):
        blk.decode(m["x"][last].contiguous(), None, keys, values, at, one, p, bd)
    yd, sd = blk.decode(m["x"][last].contiguous(), None, keys, values, at, one, p, bd,
                        pos=m["pos"][last].contiguous())
    assert O.rel_err(f64(yd), f64(y[last])) <= FORWARD
    assert O.rel_err(f64(sd), f64(s2[last])) <= FORWARD
    ref = K.rope_forward(f64(bd["y_k"]).reshape(n, HEADS, DIM), m["pos"].cpu().numpy()[last],
                         K.rope_freqs(DIM), DIM, f64(p["gk"]), EPS)
    within(f64(keys[rows]), ref, _bound_fwd(ref, DIM, "bf16"), "cached keys")
    assert torch.equal(values[rows].view(n, N), bd["y_v"])
    # and the head on it: the most likely tokens
    head, hp, _ = _head(5000, 64, top=5)
    hb = head.buffers(n)
    logp, lse, ent, top, top_logp = head.forward(yd, sd, hp, hb)
    assert logp is None
    _check_fwd(hb["logits"][:, :5000], None, 1.0, 5, (None, lse, ent, top, top_logp))


def test_refusals():
    from tensor_train_compressed_tt_gb300.encoder import TTTransformerBlock
    from tensor_train_compressed_tt_gb300.layer import TTDropout, TTRotary
    with pytest.raises(ValueError):
        TTTransformerBlock(HEADS, rotary=TTRotary(HEADS, 32))
    with pytest.raises(ValueError):
        TTTransformerBlock(HEADS, rotary=TTRotary(HEADS, DIM, kv_heads=4))
    with pytest.raises(ValueError):
        _head(5121, 0)
    m = _setup((8,), 65, dropout=0.0, blocks=1)
    rng = TTDropout.state(1)
    with pytest.raises(ValueError):
        m["blks"][0].forward(m["x"], None, m["seqs"], m["params"][0], m["bufs"][0], rng=rng)
    with pytest.raises(ValueError):
        m["head"].step(m["x"], None, m["targets"], m["dlogp"], m["hp"], m["hb"], rng=rng)

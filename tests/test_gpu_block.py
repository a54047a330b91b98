"""The whole encoder block: normalisations, residual sums and attention between
the TT layers, its training step and its step of single tokens.

Each operator is compared with the oracle on the inputs that the block gave it,
at that operator's own tolerance, and the whole block with the oracle's chain of
all of them.  Tolerance of the chain: the operators' norm-wise tolerances added
along the longest path (norm 2.1e-3, Q K V 2e-2, attention 6e-3, O 2e-2, norm
2.1e-3, FFN 2e-2: 7e-2 forward, the same again backward), doubled for paths that
meet in a product."""

import numpy as np
import pytest

from block_util import NORM_TOL, TOL as ATTN_TOL, assert_near
from oracle import block_oracle as B
from oracle import tt_oracle as O
from parity_util import TOL
from tensor_train_compressed_tt_gb300 import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HEADS, DIM, N = 12, 64, 768
FORWARD, BACKWARD = 0.14, 0.28


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from tensor_train_compressed_tt_gb300 import _build
    _build.build()


def _heads(a):
    return a.reshape(-1, HEADS, DIM)


def _flat(a):
    return a.reshape(-1, N)


def _f64(t):
    return t.double().cpu().numpy()


def _setup(lens, seed, **window):
    from tensor_train_compressed_tt_gb300.encoder import TTTransformerBlock
    from tensor_train_compressed_tt_gb300.layer import TTSeqs
    T = sum(lens)
    inp = synth.draw_encoder(T, seed)
    blk = TTTransformerBlock(HEADS, **window)
    dev = lambda a: torch.from_numpy(a).cuda().bfloat16()  # noqa: E731
    rng = np.random.default_rng(seed)
    weights = {nm: rng.uniform(0.5, 1.5, N).astype(np.float32) for nm in ("g1", "b1", "g2", "b2")}
    params = {nm: torch.from_numpy(synth.pack(li.cores, li.diags)).cuda()
              for nm, li in inp.layers.items()}
    params.update({nm: torch.from_numpy(w).cuda() for nm, w in weights.items()})
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    seqs = TTSeqs.packed(torch.from_numpy(off).cuda(), T, max(lens))
    layers = {nm: ([c.astype(np.float64) for c in li.cores], [e.astype(np.float64) for e in li.diags])
              for nm, li in inp.layers.items()}
    spans = [(a, b, a, b) for a, b in zip(off[:-1], off[1:])]
    return blk, seqs, spans, params, layers, weights, dev(inp.x), dev(inp.xo), \
        dev(inp.dy["ffn"]), dev(inp.dy["o"])


def _tt(layers, nm, x):
    return O.chained_forward(*layers[nm], 3, x)


def _chain_forward(layers, w, x, res, spans, window):
    """Every value of the block, in 64 bits throughout."""
    v = {}
    v["h1"], v["s1"], _ = B.norm_forward(x, w["g1"], w["b1"], res)
    for nm in "qkv":
        v[nm] = _tt(layers, nm, v["h1"])
    att, _ = B.attn_forward(*(_heads(v[nm]) for nm in "qkv"), spans, **window)
    v["att"] = _flat(att)
    v["h2"], v["s2"], _ = B.norm_forward(_tt(layers, "o", v["att"]), w["g2"], w["b2"], v["s1"])
    v["ffn"] = O.ffn_forward(layers["up"], layers["down"], 3, 3, v["h2"])
    return v


def _chain_backward(layers, w, v, dffn, ds2_out, spans, window):
    g = {}
    dh2, _, _ = O.ffn_backward(layers["up"], layers["down"], 3, 3, v["h2"], dffn)
    ds2, g["dg2"], g["db2"] = B.norm_backward(v["s2"], dh2, w["g2"], ds2_out)
    datt = O.chained_backward(*layers["o"], 3, v["att"], ds2)[0]
    d = B.attn_backward(*(_heads(v[nm]) for nm in "qkv"), _heads(datt), spans, **window)
    dh1 = sum(O.chained_backward(*layers[nm], 3, v["h1"], _flat(x))[0] for nm, x in zip("qkv", d))
    g["ds1"], g["dg1"], g["db1"] = B.norm_backward(v["s1"], dh1, w["g1"], ds2)
    return g


@pytest.mark.parametrize("lens,window", [((65, 1, 40), {}),
                                         ((130, 7), dict(left=20, right=0, sinks=3))])
def test_training_step_against_oracle(lens, window):
    blk, seqs, spans, params, layers, w, x, res, dffn, ds2 = _setup(lens, 50, **window)
    b = blk.buffers(sum(lens), seqs)
    y, s2 = blk.forward(x, res, seqs, params, b)
    ds1 = blk.backward(x, res, dffn, ds2, seqs, params, b)
    torch.cuda.synchronize()
    v = {k: _f64(t) for k, t in b.items() if not k.startswith("ws_")}
    ntol, atol = NORM_TOL["bf16"], ATTN_TOL["bf16"]
    # operator by operator, on the block's own values
    h, s, _ = B.norm_forward(_f64(x), w["g1"], w["b1"], _f64(res))
    assert_near(v["s1"], s, ntol, "s1")
    assert O.rel_err(v["h1"], h) <= 2 * ntol  # s rounded, then y
    for nm in "qkv":
        assert O.rel_err(v[f"y_{nm}"], _tt(layers, nm, v["h1"])) <= TOL["bf16"], nm
    q, k, val = (_heads(v[f"y_{nm}"]) for nm in "qkv")
    o, _ = B.attn_forward(q, k, val, spans, **window)
    assert_near(_heads(v["att"]), o, atol, "attention")
    assert O.rel_err(v["y_o"], _tt(layers, "o", v["att"])) <= TOL["bf16"]
    h, s, _ = B.norm_forward(v["y_o"], w["g2"], w["b2"], v["s1"])
    assert_near(v["s2"], s, ntol, "s2")
    assert O.rel_err(v["h2"], h) <= 2 * ntol
    dx, dg, db = B.norm_backward(v["s2"], v["dx_ffn"], w["g2"], _f64(ds2))
    assert_near(v["ds2"], dx, ntol, "ds2")
    assert O.rel_err(v["dg2"], dg) <= ntol and O.rel_err(v["db2"], db) <= ntol
    d = B.attn_backward(q, k, val, _heads(v["datt"]), spans, **window)
    for nm, ref in zip(("dq", "dk", "dv"), d):
        assert_near(_heads(v[nm]), ref, atol, nm)
    dx, dg, db = B.norm_backward(v["s1"], v["dx_qkv"], w["g1"], v["ds2"])
    assert_near(v["ds1"], dx, ntol, "ds1")
    assert O.rel_err(v["dg1"], dg) <= ntol and O.rel_err(v["db1"], db) <= ntol
    # the whole chain
    ref = _chain_forward(layers, w, _f64(x), _f64(res), spans, window)
    assert O.rel_err(_f64(y), ref["ffn"]) <= FORWARD
    assert O.rel_err(_f64(s2), ref["s2"]) <= FORWARD
    g = _chain_backward(layers, w, ref, _f64(dffn), _f64(ds2), spans, window)
    assert O.rel_err(_f64(ds1), g["ds1"]) <= BACKWARD
    for nm in ("dg1", "db1", "dg2", "db2"):
        assert O.rel_err(v[nm], g[nm]) <= BACKWARD, nm


def test_first_block_takes_no_residual():
    lens = (33, 12)
    blk, seqs, spans, params, layers, w, x, _, dffn, _ = _setup(lens, 51, right=0)
    b = blk.buffers(sum(lens), seqs)
    y, _ = blk.forward(x, None, seqs, params, b)
    ds1 = blk.backward(x, None, dffn, None, seqs, params, b)
    ref = _chain_forward(layers, w, _f64(x), None, spans, dict(right=0))
    assert O.rel_err(_f64(y), ref["ffn"]) <= FORWARD
    g = _chain_backward(layers, w, ref, _f64(dffn), None, spans, dict(right=0))
    assert O.rel_err(_f64(ds1), g["ds1"]) <= BACKWARD


def test_training_step_replays_from_a_graph():
    lens = (100, 29)
    blk, seqs, _, params, _, _, x, res, dffn, ds2 = _setup(lens, 52, right=0)
    b = blk.buffers(sum(lens), seqs)

    def step():
        blk.forward(x, res, seqs, params, b)
        blk.backward(x, res, dffn, ds2, seqs, params, b)

    step()
    torch.cuda.synchronize()
    names = ("y_ffn", "s2", "ds1", "dg1", "db1", "dq", "dk", "dv")
    eager = {k: b[k].clone() for k in names}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in names:
        b[k].zero_()
    g.replay()
    torch.cuda.synchronize()
    for k in names:
        assert torch.equal(b[k], eager[k]), k


@pytest.mark.parametrize("window", [dict(right=0), dict(left=16, right=0, sinks=2)])
def test_decode_continues_a_forward(window):
    """The last token of each sequence, by the cache, against the same token in a
    forward of the whole sequence (both within FORWARD / 2 of the exact block)."""
    from tensor_train_compressed_tt_gb300.layer import TTSeqs
    lens, room = (50, 1, 33), 64
    blk, seqs, spans, params, layers, w, x, res, _, _ = _setup(lens, 53, **window)
    T, n = sum(lens), len(lens)
    b = blk.buffers(T, seqs)
    y, s2 = blk.forward(x, res, seqs, params, b)
    keys = torch.full((n * room, HEADS, DIM), float("nan"), dtype=torch.bfloat16, device="cuda")
    values = keys.clone()
    last, rows = [], []
    for i, (a, e, _, _) in enumerate(spans):
        m = int(e - a) - 1
        keys[i * room:i * room + m] = b["y_k"][a:a + m].view(m, HEADS, DIM)
        values[i * room:i * room + m] = b["y_v"][a:a + m].view(m, HEADS, DIM)
        last.append(int(e) - 1)
        rows.append(i * room + m)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    first = np.arange(n) * room
    one = TTSeqs(i32(range(n)), i32(range(1, n + 1)), i32(first.tolist()),
                 i32([r + 1 for r in rows]), n, n * room, 1, room)
    bd = blk.buffers(n, one)
    row = torch.tensor(rows, device="cuda")
    yd, sd = blk.decode(x[last].contiguous(), res[last].contiguous(), keys, values, row, one,
                        params, bd)
    assert O.rel_err(_f64(yd), _f64(y[last])) <= FORWARD
    assert O.rel_err(_f64(sd), _f64(s2[last])) <= FORWARD
    o, _ = B.attn_forward(_heads(_f64(bd["y_q"])), _f64(keys), _f64(values),
                          [(i, i + 1, f, r + 1) for i, (f, r) in enumerate(zip(first, rows))],
                          **window)
    assert_near(_heads(_f64(bd["att"])), o, ATTN_TOL["bf16"], "attention against the cache")


@pytest.mark.parametrize("n", [1, 2, 4, 5])
@pytest.mark.parametrize("window", [dict(right=0), dict(left=1500, right=0, sinks=4)])
def test_decode_against_a_long_cache(n, window):
    """Few sequences and long caches: the keys of a head are split over several
    clusters, whose shares meet in the workspace of the block's buffers."""
    from tensor_train_compressed_tt_gb300.layer import TTSeqs
    room = 2500
    blk, _, _, params, _, _, x, res, _, _ = _setup((1,) * n, 54, **window)
    lk = [room - 3 * i for i in range(n)]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    first = [i * room for i in range(n)]
    one = TTSeqs(i32(list(range(n))), i32(list(range(1, n + 1))), i32(first),
                 i32([f + m for f, m in zip(first, lk)]), n, n * room, 1, room)
    b = blk.buffers(n, one)
    r = np.random.default_rng(55)
    keys, values = (torch.from_numpy(r.standard_normal((n * room, HEADS, DIM)).astype(np.float32))
                    .cuda().bfloat16() for _ in range(2))
    rows = torch.tensor([f + m - 1 for f, m in zip(first, lk)], device="cuda")
    blk.decode(x, res, keys, values, rows, one, params, b)
    assert torch.equal(keys[rows].view(n, N), b["y_k"])
    assert torch.equal(values[rows].view(n, N), b["y_v"])
    o, _ = B.attn_forward(_heads(_f64(b["y_q"])), _f64(keys), _f64(values),
                          [(i, i + 1, f, f + m) for i, (f, m) in enumerate(zip(first, lk))],
                          **window)
    assert_near(_heads(_f64(b["att"])), o, ATTN_TOL["bf16"], "attention against the cache")


def test_one_workspace_for_both_passes():
    """TTAttention.workspace's default serves the forward and the backward of its sequences."""
    from tensor_train_compressed_tt_gb300.layer import TTAttention, TTSeqs
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    op = TTAttention(4, DIM)
    seqs = TTSeqs(i32([0]), i32([1]), i32([0]), i32([4000]), 1, 4000, 1, 4000)
    q = torch.randn(1, 4, DIM, device="cuda").bfloat16()
    k = torch.randn(4000, 4, DIM, device="cuda").bfloat16()
    ws = op.workspace(seqs)
    assert ws.numel() >= op.workspace(seqs, False).numel()
    o, lse = op.forward(q, k, k, seqs, ws=ws)
    o2, lse2 = op.forward(q, k, k, seqs)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for a, b in zip(op.backward(q, k, k, o, lse, q, seqs, ws=ws),
                    op.backward(q, k, k, o, lse, q, seqs)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("first", [False, True])
def test_step_and_its_graph_run_the_whole_block(first):
    lens = (70, 31)
    blk, seqs, _, params, _, _, x, res, dffn, ds2 = _setup(lens, 56, left=40, right=0, sinks=1)
    if first:
        res = ds2 = None
    b = blk.buffers(sum(lens), seqs)
    blk.forward(x, res, seqs, params, b)
    blk.backward(x, res, dffn, ds2, seqs, params, b)
    names = ["y_ffn", "s2", "ds1", "dg1", "db1", "dg2", "db2"]
    want = {k: b[k].clone() for k in names}
    params_of = [k for k in b if k.startswith("dp_")]

    def clear():
        for k in names + params_of:
            b[k].zero_()

    clear()
    blk.step(x, res, dffn, ds2, seqs, params, b)
    for k in names:
        assert torch.equal(b[k], want[k]), k
    torch.cuda.synchronize()
    g = blk.capture(x, res, dffn, ds2, seqs, params, b)
    clear()
    g.replay()
    torch.cuda.synchronize()
    for k in names:
        assert torch.equal(b[k], want[k]), k
    assert all(float(b[k].abs().max()) > 0 for k in params_of)

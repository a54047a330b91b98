"""Ends of the ranges of rotary positions, log probabilities and dropout on the GPU against the
fp64 oracle, at the bounds of their other tests (test_gpu_rope, test_gpu_logp)."""

import numpy as np
import pytest

from oracle import token_oracle as K

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tensor_train_compressed_tt_gb300.layer import TTLogProbs  # noqa: E402
from test_gpu_logp import TINY, _check_fwd, _check_grad, _f32, _i32, _rows, _status  # noqa: E402
from test_gpu_rope import _case as _rope_case  # noqa: E402
from test_gpu_rope import _plan  # noqa: E402
from token_util import DT, HALF, f64, nan, rand, within  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from tensor_train_compressed_tt_gb300 import _build
    _build.build()


@pytest.mark.parametrize("heads,kv", [(1, 1), (2, 1), (12, 12), (16, 4), (71, 71)])
def test_rope_workspace_of_the_most_tokens_serves_fewer(heads, kv):
    """One workspace for the largest batch: its size never falls as the tokens grow, and a
    shorter last batch runs in it with the results of its own."""
    from tensor_train_compressed_tt_gb300 import ttc
    from tensor_train_compressed_tt_gb300.layer import TTRotary
    op = TTRotary(heads, 32, kv_heads=kv)
    sizes = [ttc.tt_workspace_size(op.plan, T) for T in (*range(1600), 5000, 40000, 2 ** 31 - 1)]
    assert sizes == sorted(sizes)
    r = np.random.default_rng(heads)
    n = heads + kv
    for few, most in ((101, 102), (1216 * 2 // n, 1216 * 2 // n + 1), (33, 4096)):
        q, k, dq, dk = (rand(r, (few, h, 32), "bf16") for h in (heads, kv, heads, kv))
        ws = op.workspace(most)
        want = op.backward(dq, dk, None, q, k)
        for a, b in zip(op.backward(dq, dk, None, q, k, ws=ws), want):
            assert torch.equal(a, b)


def _far_rows(V, act, r):
    """Rows whose log-sum is so large that its rounding to fp32 loses some or all of the
    logarithm of the sum, between ordinary ones."""
    x = r.standard_normal((12, V))
    x[1] = -1e9                          # a finite mask on everything
    x[2], x[2, V // 2] = -1e9, 3.0       # and on all but one
    x[3] = -3e38
    x[4] = 3e38
    x[5] += 7000.0
    x[6] -= 300.0
    x[7] = 1e9 + 128.0 * r.integers(0, 2, V)
    x[8] = -np.inf
    x[9], x[9, ::2] = -20000.0, -np.inf  # half of it masked, the rest equal
    x[10], x[10, V - 1] = -3e38, 3e38
    return x


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 2.5])
@pytest.mark.parametrize("V,pad,shift,dpad", [
    (2, 0, 0, 0), (13, 1, 0, 1), (700, 0, 0, 0), (3001, 1, 3, 1), (3000, 0, 0, 1), (40001, 7, 1, 7),
    (100, 0, 1, 3)])
def test_gradient_where_the_log_sum_is_large(V, pad, shift, dpad, scale, act):
    """From the forward's lse, which at 1e9 is rounded to 64: the weights are the row's own all
    the same, as tt_logp_loss has them, and sum to one.  With scale 2.5 the log-sums of the
    type's ends are infinite.  The bounds are those of the pass that rounds nothing between."""
    r = np.random.default_rng(V)
    x = _rows(_far_rows(V, act, r), act, pad, shift)
    T = x.shape[0]
    t = r.integers(0, V, T)
    t[4], t[6], t[9] = -1, 0, V - 1
    g, h = r.standard_normal(T).astype(np.float32), r.standard_normal(T).astype(np.float32)
    op = TTLogProbs(V, DT[act], scale=scale)
    ent = nan((T,), torch.float32)
    _, lse, _, _, _ = op.forward(x, _i32(t), entropy=ent)
    for dent in (None, h):
        d = _rows(np.full((T, V), np.nan), act, dpad, shift)
        args = (_f32(g), ent if dent is not None else None, None if dent is None else _f32(dent))
        op.backward(x, _i32(t), lse, *args, dlogits=d)
        _check_grad(x, t, g, dent, scale, act, d, "dlogits")
        if dpad == pad:  # in place
            whole = x.as_strided((T, V + pad), (V + pad, 1), x.storage_offset())
            y = torch.empty(T * (V + pad) + shift, dtype=DT[act], device="cuda")[shift:]
            y = y.view(T, V + pad).copy_(whole)[:, :V]
            op.backward(y, _i32(t), lse, *args, dlogits=y)
            assert torch.equal(y, d)
    assert _status() == 0


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(6, 40), (6, 3000), (6, 40000), (6, 131072), (700, 14000),
                                 (310, 60001)])
def test_masked_targets_of_rows_that_are_not_finite(T, V, act):
    """A NaN or +infinity makes the whole row's results NaN, also of a target or an alternative
    whose logit is -infinity; without one those are -infinity."""
    x = torch.randn(T, V, device="cuda").to(DT[act])
    x[:, 8:] = -float("inf")
    x[1, 3], x[2, 4] = float("nan"), float("inf")
    t = torch.full((T,), V - 1, dtype=torch.int32, device="cuda")
    op = TTLogProbs(V, DT[act], top=20)
    logp, lse, _, ids, tops = op.forward(x, t)
    logp2 = op.loss(x, t, torch.ones(T, device="cuda"))[0]
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[1:3] = True
    for a in (logp, logp2):
        assert torch.isnan(a[bad]).all() and (a[~bad] == -float("inf")).all()
    assert torch.isnan(lse[bad]).all() and torch.isnan(tops[bad]).all()
    assert torch.isfinite(tops[~bad][:, :8]).all() and (tops[~bad][:, 8:] == -float("inf")).all()
    assert int(ids.min()) >= 0 and int(ids.max()) < V


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,dim", [(1024, 1024, 8), (1024, 1, 40), (1000, 125, 33),
                                          (130, 130, 256)])
def test_rope_of_many_heads(heads, kv, dim, act):
    _rope_case(5, heads, kv, dim, act, rot=dim // 4 * 2, seed=heads)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_rope_of_many_heads_into_a_cache(act):
    r = np.random.default_rng(1)
    op = _plan(1024, 512, 24, act)
    q, k, v = (rand(r, (7, h, 24), act) for h in (1024, 512, 512))
    pos, rows = _i32(r.integers(0, 9000, 7)), _i32(r.permutation(20)[:7])
    keys, values = nan((20, 512, 24), DT[act]), nan((20, 512, 24), DT[act])
    yq, yk = op.forward(q, k, pos)
    out, _, _ = op.to_cache(q, k, v, pos, rows, keys, values)
    assert torch.equal(out, yq) and torch.equal(keys[rows.long()], yk)
    assert torch.equal(values[rows.long()], v)
    assert int(torch.isnan(keys[:, 0, 0].float()).sum()) == 13


def _many_rows(T, V, act, pad, dpad, ent):
    """The loss of many rows: some against the oracle, all against the pass of its own, in place."""
    r = np.random.default_rng(V)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(V)
    whole = torch.randn(T, V + pad, generator=gen, device="cuda").mul_(3).to(DT[act])
    x = whole[:, :V]
    x[3], x[4, V // 2:], x[5] = -np.inf, -np.inf, 0
    x[T - 1, :V - 1] = -np.inf
    t = r.integers(0, V, T)
    t[::5], t[4], t[6], t[7] = -1, 1, 0, V - 1
    g = r.standard_normal(T).astype(np.float32)
    h = r.standard_normal(T).astype(np.float32) if ent else None
    dev = None if h is None else _f32(h)
    op = TTLogProbs(V, DT[act], scale=0.9)
    e = nan((T,), torch.float32) if ent else None
    out = torch.full((T, V + dpad), float("nan"), dtype=DT[act], device="cuda")
    logp, lse, e, d = op.loss(x, _i32(t), _f32(g), dev, entropy=e, dlogits=out[:, :V])
    rows = np.r_[0:9, 151:154, 303:306, T - 2:T]
    at = torch.from_numpy(rows).cuda()
    pick = lambda a: None if a is None else a[at]  # noqa: E731
    some = lambda a: None if a is None else a[rows]  # noqa: E731
    _check_fwd(pick(x), t[rows], 0.9, 0, (pick(logp), pick(lse), pick(e)))
    _check_grad(pick(x), t[rows], g[rows], some(h), 0.9, act, pick(d), "dlogits")
    if dpad:
        assert torch.isnan(out[:, V:].float()).all()
    other = op.backward(x, _i32(t), lse, _f32(g), e, dev)
    # both are near the same value: half a step of the type each, and 2^-17 of the terms
    size = (torch.from_numpy(g).cuda().abs() + (0 if dev is None else 24 * dev.abs()))[:, None]
    near = 2.0 ** -7 if act == "bf16" else 2.0 ** -16
    assert ((d.float() - other.float()).abs() <= near * other.float().abs() + 2.0 ** -16 * size
            ).all()
    if pad == dpad:
        y = whole.clone()[:, :V]
        again = op.loss(y, _i32(t), _f32(g), dev, dlogits=y)
        assert torch.equal(y, d) and torch.equal(again[0], logp) and torch.equal(again[1], lse)
    assert _status() == 0


@pytest.mark.parametrize("ent", [False, True])
@pytest.mark.parametrize("act,V", [("bf16", 70000), ("bf16", 120001), ("bf16", 131072),
                                   ("f32", 33000), ("f32", 60001), ("f32", 100003)])
def test_loss_of_many_long_rows(act, V, ent):
    """A row an SM of 32 warps, the next one sent for ahead; above 216 KB what does not fit in
    shared memory is read again."""
    _many_rows(310, V, act, 1, 1, ent)


@pytest.mark.parametrize("ent", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,pad,dpad", [(700, 13001, 1, 2), (3000, 300, 3, 4), (700, 5000, 1, 0),
                                          (310, 60001, 2, 1)])
def test_loss_of_many_rows_that_lie_differently(T, V, pad, dpad, act, ent):
    """Rows of the gradient at another distance from a 16-byte boundary than the logits'."""
    _many_rows(T, V, act, pad, dpad, ent)


@pytest.mark.parametrize("act,V", [("bf16", 1 << 22), ("f32", (1 << 24) - 3), ("bf16", 1 << 24)])
def test_widest_rows(act, V):
    """Up to 2^24 logits.  A thread of eight CTAs of 256 adds V / 2^12 powers to each of its two
    sums: V / 2^12 roundings of 2^-24 more than the bounds of short rows have."""
    r = np.random.default_rng(2)
    x = torch.from_numpy(r.standard_normal((2, V)).astype(np.float32)).to(DT[act]).cuda()
    t, g = np.array([V - 1, V // 3]), np.array([0.5, -1.0], np.float32)
    more = V / 4096 * 2.0 ** -24
    op = TTLogProbs(V, DT[act], top=20)
    ent = nan((2,), torch.float32)
    logp, lse, _, ids, tops = op.forward(x, _i32(t), entropy=ent)
    rp, rl, re, ri, rt = K.logp_forward(f64(x), t, 1.0, 20)
    logp2, lse2, _, d = op.loss(x, _i32(t), _f32(g))
    near = 2.0 ** -19 + 2.0 ** -22 * 32 + more  # |lse| and |log p| are below 32
    for got, ref in ((logp, rp), (lse, rl), (logp2, rp), (lse2, rl)):
        within(f64(got), ref, near, "logp, lse")
    within(f64(ent), re, 2.0 ** -18 * (1 + re) + 32 * more, "entropy")
    assert np.array_equal(ids.cpu().numpy(), ri)
    within(f64(tops), rt, near, "top_logp")
    ref, size = K.logp_backward(f64(x), t, g)
    bound = HALF[act] * np.abs(ref) + (2.0 ** -18 + 2.0 ** -22 * 64 + more) * size + TINY
    within(f64(d), ref, bound, "loss: dlogits")
    within(f64(op.backward(x, _i32(t), lse, _f32(g))), ref, bound, "dlogits")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,dim", [(12, 12, 64), (6, 2, 33), (5, 5, 80)])
def test_rope_gradient_in_the_place_of_q_and_k(heads, kv, dim, act):
    r = np.random.default_rng(dim)
    op = _plan(heads, kv, dim, act, rot=dim // 2 * 2)
    q, k, dq, dk = (rand(r, (700, h, dim), act) for h in (heads, kv, heads, kv))
    want = op.backward(dq, dk, None, q, k)
    a, b = q.clone(), k.clone()
    for got, ref in zip(op.backward(dq, dk, None, a, b, dq_in=a, dk_in=b), want):
        assert torch.equal(got, ref)


def test_rope_into_a_cache_without_rows():
    """Every row is one that the cache does not have, but the negative ones."""
    op = _plan(4, 2, 64, "bf16")
    r = np.random.default_rng(0)
    q, k, v = (rand(r, (5, h, 64), "bf16") for h in (4, 2, 2))
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = _i32(range(5))
    want = op.forward(q, k, pos)[0]
    for rows, bad in (([-1] * 5, False), ([-1, 0, -2, 7, -5], True)):
        out, _, _ = op.to_cache(q, k, v, pos, _i32(rows), none, none.clone())
        assert torch.equal(out, want)
        assert (_status() != 0) == bad and _status() == 0


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-6, 1e-3, 1e3, 1e6])
@pytest.mark.parametrize("T,V", [(6, 100), (6, 5000), (6, 70001), (700, 14000)])
def test_ends_of_the_scale(T, V, scale, act):
    """From rows that are nearly even to rows of their largest logits alone."""
    r = np.random.default_rng(V)
    x = _rows((3 * r.standard_normal((T, V))).astype(np.float32), act, 1, 0)
    # a power of two of c is off where its scale is: the oracle takes the fp32 one
    s = float(np.float32(scale))
    t, g = r.integers(0, V, T), r.standard_normal(T).astype(np.float32)
    h = r.standard_normal(T).astype(np.float32)
    t[0] = -1
    op = TTLogProbs(V, DT[act], scale=scale, top=3)
    rows = np.r_[0:6] if T > 6 else np.arange(T)
    at = torch.from_numpy(rows).cuda()
    got = op.forward(x, _i32(t), entropy=nan((T,), torch.float32))
    _check_fwd(x[at], t[rows], s, 3, tuple(a[at] for a in got))
    for dent in (None, h):
        ent = None if dent is None else got[2]
        dev = None if dent is None else _f32(dent)
        d = op.backward(x, _i32(t), got[1], _f32(g), ent, dev)
        out = torch.empty(T, V + 1, dtype=DT[act], device="cuda")[:, :V]
        e = nan((T,), torch.float32) if dent is not None else None
        logp, lse, e, d2 = op.loss(x, _i32(t), _f32(g), dev, entropy=e, dlogits=out)
        _check_fwd(x[at], t[rows], s, 0, (logp[at], lse[at], None if e is None else e[at]))
        hs = None if dent is None else dent[rows]
        ref, size = K.logp_backward(f64(x[at]), t[rows], g[rows], hs, s)
        rl = K.logp_forward(f64(x[at]), scale=s)[1]
        lp = np.stack([K.log_p(s * row)[0] for row in f64(x[at])])
        err = 2.0 ** -18 + 2.0 ** -22 * np.abs(lp)
        tiny = TINY * max(1.0, s)  # that of scale 1 holds for 2.5 of it
        within(f64(d2[at]), ref, HALF[act] * np.abs(ref) + err * size + tiny, "loss: dlogits")
        # a log-sum that is taken as it is has half a step of its own: 2^-24 of 256 or 4096 at most
        most = 256.0 if act == "f32" else 4096.0
        given = 2.0 ** -22 * np.where(np.abs(rl) <= most, np.abs(rl), 0)[:, None]
        within(f64(d[at]), ref, HALF[act] * np.abs(ref) + (err + given) * size + tiny, "dlogits")


def test_a_block_without_tokens():
    """An empty batch through a block with positions and dropout, forward and backward."""
    from tensor_train_compressed_tt_gb300.encoder import TTTransformerBlock
    from tensor_train_compressed_tt_gb300.layer import TTDropout, TTRotary, TTSeqs
    from test_gpu_lm import _block_params
    rng = TTDropout.state(1)
    seqs = TTSeqs.packed(_i32([0, 0]), 0, 1)
    blk = TTTransformerBlock(12, rotary=TTRotary(12, 64), dropout=0.1, site=0)
    p, b = _block_params(0), blk.buffers(0, seqs)
    x = torch.empty(0, 768, dtype=torch.bfloat16, device="cuda")
    blk.step(x, x, x, x, seqs, p, b, rng=rng)
    for nm in ("dgq", "dgk", "dg1", "db2"):
        assert float(b[nm].abs().max()) == 0
    assert _status() == 0


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 33])
def test_rope_heads_whose_squares_exceed_fp32(dim, act):
    """Finite values over the root of an infinite sum are zeros, gradients too, as in the formula
    in fp32; an infinity or a NaN spoils its own head alone."""
    op = _plan(3, 1, dim, act, rot=dim // 2 * 2)
    r = np.random.default_rng(dim)
    q, k, dq, dk = (rand(r, (9, h, dim), act) for h in (3, 1, 3, 1))
    clean = op.forward(q, k)[0], op.backward(dq, dk, None, q, k)[0]
    q[2, 1] = 1e20
    q[3, 0, 5] = -3e38
    got = op.forward(q, k)[0], op.backward(dq, dk, None, q, k)
    for a, b in zip((got[0], got[1][0]), clean):
        for t, h in ((2, 1), (3, 0)):
            assert float(a[t, h].float().abs().max()) == 0
            a[t, h] = b[t, h]
        assert torch.equal(a, b)
    assert all(torch.isfinite(g).all() for g in got[1][2:])
    q[2, 1, 7], q[3, 0, 5] = float("nan"), float("inf")
    y = op.forward(q, k)[0]
    assert torch.isnan(y[2, 1].float()).any() and torch.isnan(y[3, 0].float()).any()
    y[2, 1], y[3, 0] = clean[0][2, 1], clean[0][3, 0]
    assert torch.equal(y, clean[0])

"""Log probabilities, entropy, top alternatives and gradients on the GPU against the
fp64 oracle.

Bounds.  A power 2^t carries 2 ulp of the instruction and |t| 2^-24 of its argument:
below 2^-19 for |t| < 32, and terms beyond that are smaller than 2^-32.  Sums and the
logarithm add a few 2^-22.  So log p and the log-sum are off by 2^-19, plus 2^-22 of
their own size (products with ln 2, the sum with the maximum), the entropy by 2^-18 of
1 + H; a gradient by half a step of its type and 2^-18 of the terms that meet (and
2^-22 of lse times them where lse is the rounded one that the caller gave).  The terms
of an entropy's gradient are h p (log p + H), whose factor in brackets carries the
absolute errors of log p and H, 2^-19 and 2^-18 (1 + H): h p times 2^-18 (1 + |log p| + H)
covers both, also where the two cancel (a row of one logit: log p = H = 0).  An element
far below its row's maximum has t of some |log p| / ln 2 or less, made of a difference, a
product and a rounded factor: 3 roundings of 2^-24 of it, which is the power's relative
error, so 2^-22 |log p| is added."""

import numpy as np
import pytest

from oracle import token_oracle as K

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from token_util import DT, HALF, f64, nan, within  # noqa: E402

# A power below 2^-126 is flushed to zero: of a gradient that takes away p (|g| + |h|
# (|log p| + H)) at most, with |log p| = 88 at that border, H below 12, |g|, |h| <= 1 and
# scale <= 2.5.
TINY = 2.0 ** -126 * (1 + 88 + 12) * 2.5


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from tensor_train_compressed_tt_gb300 import _build
    _build.build()


def _status():
    from tensor_train_compressed_tt_gb300 import ttc
    return ttc.tt_get_device_status(torch.cuda.current_stream().cuda_stream)


def _rows(x, act, pad, shift):
    """x with `pad` more columns a row, the first row `shift` elements into the buffer."""
    T, V = x.shape
    t = torch.from_numpy(x.astype(np.float32)).to(DT[act]).cuda()
    flat = torch.full((T * (V + pad) + shift,), 7.0, dtype=DT[act], device="cuda")
    out = flat[shift:].view(T, V + pad)[:, :V] if T else flat[:0].view(0, V)
    out.copy_(t)
    return out


def _i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def _f32(a):
    return torch.from_numpy(np.asarray(a, np.float32)).cuda()


def _check_fwd(x, t, scale, top, got, what=""):
    logp, lse, ent, ids, tops = K.logp_forward(f64(x), t, scale, top)
    fin = lambda a: np.where(np.isfinite(a), np.abs(a), 0)  # noqa: E731
    if got[0] is not None:
        within(f64(got[0]), logp, 2.0 ** -19 + 2.0 ** -22 * fin(logp), what + "logp")
    within(f64(got[1]), lse, 2.0 ** -19 + 2.0 ** -22 * fin(lse), what + "lse")
    if got[2] is not None:
        within(f64(got[2]), ent, 2.0 ** -18 * (1 + np.abs(ent)), what + "entropy")
    if top:
        assert np.array_equal(got[3].cpu().numpy(), ids), what + "top"
        within(f64(got[4]), tops, 2.0 ** -19 + 2.0 ** -22 * fin(tops), what + "top_logp")


def _check_grad(x, t, g, h, scale, act, d, what, given=False):
    ref, size = K.logp_backward(f64(x), t, g, h, scale)
    lse = K.logp_forward(f64(x), scale=scale)[1]
    lse = np.where(np.isfinite(lse), np.abs(lse), 0)[:, None]
    lp = np.stack([K.log_p(scale * row)[0] if row.max() > -np.inf else np.zeros_like(row)
                   for row in f64(x)]) if len(ref) else ref
    err = 2.0 ** -18 + 2.0 ** -22 * np.where(np.isfinite(lp), np.abs(lp), 0)
    if given:
        err = err + 2.0 ** -22 * lse
    within(f64(d), ref, HALF[act] * np.abs(ref) + err * size + TINY, what)


def _case(T, V, act, top=0, ent=True, scale=1.0, masked=0, pad=0, shift=0, dpad=None, seed=0,
          spread=3.0, stream=None):
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    r = np.random.default_rng(seed)
    x = spread * r.standard_normal((T, V)) + 2 * r.standard_normal(V)
    if masked:
        x[:, r.permutation(V)[:V * masked // 100]] = -np.inf
    x = _rows(x, act, pad, shift)
    t = r.integers(0, V, T)
    t[r.random(T) < 0.2] = -1
    g = (r.standard_normal(T) / max(T, 1)).astype(np.float32)
    h = (0.1 * r.standard_normal(T)).astype(np.float32) if ent else None
    op = TTLogProbs(V, DT[act], scale=scale, top=top)
    f32 = torch.float32
    e = nan((T,), f32) if ent else None
    got = op.forward(x, _i32(t), entropy=e, logp=nan((T,), f32), lse=nan((T,), f32),
                     stream=stream)
    _check_fwd(x, t, scale, top, got)
    dpad = pad if dpad is None else dpad
    d = _rows(np.full((T, V), np.nan), act, dpad, shift)
    args = dict(dlogp=_f32(g), dentropy=None if h is None else _f32(h), stream=stream)
    # the pass of its own takes the exact log-sum and entropy, rounded
    _, lse, en, _, _ = K.logp_forward(f64(x), scale=scale)
    op.backward(x, _i32(t), _f32(lse), entropy=_f32(en) if ent else None, dlogits=d, **args)
    _check_grad(x, t, g, h, scale, act, d, "dlogits", given=True)
    d2 = _rows(np.full((T, V), np.nan), act, dpad, shift)
    logp, lse, en, _ = op.loss(x, _i32(t), entropy=nan((T,), f32) if ent else None, dlogits=d2,
                               logp=nan((T,), f32), lse=nan((T,), f32), **args)
    _check_fwd(x, t, scale, 0, (logp, lse, en), "loss: ")
    _check_grad(x, t, g, h, scale, act, d2, "loss: dlogits")
    if dpad and T:
        for out in (d, d2):  # the columns behind the row stay as they were
            whole = out.as_strided((T, V + dpad), (V + dpad, 1), out.storage_offset())
            assert float((whole[:, V:].float() - 7).abs().sum()) == 0
    assert _status() == 0


VOCABS = [1, 2, 3, 7, 8, 9, 14, 15, 16, 100, 255, 256, 257, 511, 512, 513, 1000, 2047, 2049, 4095,
          4096, 4097, 5000, 8193]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("V", VOCABS)
def test_widths(V, act):
    _case(5, V, act, top=min(V, 5), seed=V)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 100])
@pytest.mark.parametrize("V", [3, 300, 2500, 20001])
def test_row_counts(T, V, act):
    _case(T, V, act, top=min(V, 3), ent=T % 2 == 0, seed=T)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 131072), (3, 70001), (330, 33000)])
def test_long_rows(T, V, act):
    """Rows split over a cluster; more rows than a cluster each are taken whole."""
    _case(T, V, act, top=20, seed=T)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift,dpad", [(0, 1, None), (1, 0, None), (8, 3, None), (3, 2, None),
                                            (1, 0, 4), (5, 1, 0)])
@pytest.mark.parametrize("V", [13, 300, 3001, 9000])
def test_strides_and_alignment(V, pad, shift, dpad, act):
    """Rows that start anywhere; a gradient whose rows lie differently from the logits'."""
    _case(6, V, act, top=4, pad=pad, shift=shift, dpad=dpad, seed=V + pad)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("V", [50, 3000, 40000])
@pytest.mark.parametrize("masked", [10, 90, 99])
def test_masked_logits(masked, V, act):
    _case(4, V, act, top=9, masked=masked, seed=masked)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.1, 0.7, 2.5])
def test_scale(scale, act):
    _case(6, 5000, act, top=3, scale=scale, seed=1)


@pytest.mark.parametrize("V", [12, 700, 3000, 40000])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_special_rows(V, act):
    """Equal logits; all but one masked; all masked; one far above; rising and falling;
    as the smallest and largest values of the type."""
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    inf, big = np.inf, 3e38
    x = np.zeros((8, V))
    x[1] = -inf
    x[1, V // 2] = 5.0
    x[2] = -inf
    x[3, V - 1] = 500.0
    x[4], x[5] = np.arange(V) * 0.25, -np.arange(V) * 0.25
    x[6] = -big
    x[7], x[7, 1] = -big, 100.0
    t = np.array([V - 1, V // 2, 0, 0, V - 1, 0, 3, 1])
    g, h = np.linspace(-1, 1, 8).astype(np.float32), np.linspace(1, -1, 8).astype(np.float32)
    top = min(V, 12)
    x = _rows(x, act, 0, 0)
    op = TTLogProbs(V, DT[act], top=top)
    got = op.forward(x, _i32(t), entropy=nan((8,), torch.float32))
    _check_fwd(x, t, 1.0, top, got)
    d = op.backward(x, _i32(t), got[1], _f32(g), got[2], _f32(h))
    _check_grad(x, t, g, h, 1.0, act, d, "dlogits", given=True)
    logp, lse, en, d = op.loss(x, _i32(t), _f32(g), _f32(h), entropy=nan((8,), torch.float32))
    _check_fwd(x, t, 1.0, 0, (logp, lse, en), "loss: ")
    _check_grad(x, t, g, h, 1.0, act, d, "loss: dlogits")


@pytest.mark.parametrize("V,k", [(5, 5), (700, 64), (3000, 64), (40000, 64), (40000, 1)])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["equal", "few", "steps", "block", "zeros"])
def test_ties(kind, V, k, act):
    """More values at the bound than the list of candidates holds, and next to it."""
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    r = np.random.default_rng(V)
    x = {"equal": np.full((3, V), 1.5), "few": r.integers(0, 3, (3, V)) * 1.0,
         "steps": r.integers(0, V // 4 + 2, (3, V)) % 256 * 0.5,
         "block": np.where(np.arange(V) // 8 % 40 == 3, 9.0, 0.0) + 0.0 * r.random((3, V)),
         "zeros": np.where(r.random((3, V)) < 0.5, -0.0, 0.0)}[kind]
    x = _rows(x, act, 1, 0)
    _, lse, _, ids, tops = TTLogProbs(V, DT[act], top=k).forward(x)
    _check_fwd(x, None, 1.0, k, (None, lse, None, ids, tops))


@pytest.mark.parametrize("V", [40, 3000, 40000])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_not_finite(V, act):
    """A NaN or +infinity spoils its own row alone; its top indices exist and differ."""
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    r = np.random.default_rng(9)
    x = r.standard_normal((6, V))
    x[1, 3], x[3, V - 1], x[4] = np.nan, np.inf, np.nan
    t = np.array([0, 1, 2, -1, 4, 5])
    x = _rows(x, act, 0, 0)
    g = _f32(np.ones(6))
    op = TTLogProbs(V, DT[act], top=7)
    logp, lse, en, ids, _ = op.forward(x, _i32(t), entropy=nan((6,), torch.float32))
    _, _, _, d = op.loss(x, _i32(t), g)
    d2 = op.backward(x, _i32(t), lse, g)
    bad, good = [1, 3, 4], [0, 2, 5]
    assert torch.isnan(lse[bad]).all() and torch.isfinite(lse[good]).all()
    assert torch.isnan(en[bad]).all() and torch.isfinite(en[good]).all()
    assert torch.isnan(logp[[1, 4]]).all() and float(logp[3]) == 0
    for grad in (d, d2):
        assert torch.isfinite(grad[good].float()).all()
        assert float(grad[3].float().abs().max()) == 0  # no target: no gradient
    ids = ids.cpu().numpy()
    assert ids.min() >= 0 and ids.max() < V
    assert all(len(set(row)) == 7 for row in ids.tolist())


def test_large_logits_keep_their_differences():
    """Logits of some thousands, a unit apart in f32: log p is exact to 2^-19."""
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    r = np.random.default_rng(10)
    x = _rows(5000.0 + r.standard_normal((4, 3000)), "f32", 0, 0)
    t = r.integers(0, 3000, 4)
    logp, _, ent, _, _ = TTLogProbs(3000, torch.float32).forward(
        x, _i32(t), entropy=nan((4,), torch.float32))
    rl, _, re, _, _ = K.logp_forward(f64(x), t)
    # c x is taken with a c rounded to 2^-25: a temperature off by as much
    within(f64(logp), rl, 2.0 ** -18, "logp")
    within(f64(ent), re, 2.0 ** -18 * (1 + re), "entropy")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("V", [20, 300, 3001, 70000])
def test_gradient_in_place(V, act):
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    r = np.random.default_rng(11)
    x = _rows(r.standard_normal((9, V)), act, 0, 0)
    t, g = _i32(r.integers(0, V, 9)), _f32(r.standard_normal(9))
    op = TTLogProbs(V, DT[act])
    logp, lse, _, d = op.loss(x, t, g)
    y = x.clone()
    logp2, lse2, _, _ = op.loss(y, t, g, dlogits=y)
    assert torch.equal(y, d) and torch.equal(logp, logp2) and torch.equal(lse, lse2)
    d = op.backward(x, t, lse, g)
    y = x.clone()
    op.backward(y, t, lse, g, dlogits=y)
    assert torch.equal(y, d)


def test_targets_outside_are_recorded():
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    for V in (30, 3000, 20000):
        x = torch.zeros(3, V, device="cuda")
        op = TTLogProbs(V, torch.float32)
        t = _i32([0, V, 2 ** 31 - 1])
        logp, lse, _, _, _ = op.forward(x, t)
        assert _status() != 0 and _status() == 0
        assert float(logp[1]) == 0 and float(logp[2]) == 0 and float(logp[0]) < 0
        g = torch.ones(3, device="cuda")
        for grad in (lambda: op.loss(x, t, g)[3], lambda: op.backward(x, t, lse, g)):
            d = grad()
            assert float(d[1:].abs().max()) == 0 and float(d[0].abs().max()) > 0
            assert _status() != 0


def test_without_targets_and_without_rows():
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    r = np.random.default_rng(12)
    x = _rows(r.standard_normal((5, 900)), "bf16", 0, 0)
    h = r.standard_normal(5).astype(np.float32)
    op = TTLogProbs(900)
    logp, lse, _, _, _ = op.forward(x)
    assert logp is None
    for d in (op.loss(x, None, dentropy=_f32(h))[3],
              op.backward(x, None, lse, entropy=_f32(K.logp_forward(f64(x))[2]),
                          dentropy=_f32(h))):
        _check_grad(x, np.full(5, -1), None, h, 1.0, "bf16", d, "dlogits", given=True)
    x = torch.empty(0, 900, dtype=torch.bfloat16, device="cuda")
    t, g = _i32([]), _f32([])
    logp, lse, _, d = op.loss(x, t, g)
    assert logp.shape == lse.shape == (0,) and d.shape == (0, 900)
    op.forward(x, t)
    op.backward(x, t, lse, g)


def test_results_repeat_on_streams_and_in_a_graph():
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    r = np.random.default_rng(13)
    x = _rows(r.standard_normal((40, 20001)), "bf16", 0, 0)
    t, g = _i32(r.integers(0, 20001, 40)), _f32(r.standard_normal(40))
    op = TTLogProbs(20001, top=5)
    fwd = op.forward(x, t, entropy=nan((40,), torch.float32))
    loss = op.loss(x, t, g)
    want = [fwd[0], fwd[1], fwd[2], fwd[3], fwd[4], loss[3]]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)
        e = _f32(np.zeros(40))
        side.wait_stream(torch.cuda.current_stream())
        got = op.forward(x, t, entropy=e, stream=side)
        d = op.loss(x, t, g, stream=side)[3]
        torch.cuda.synchronize()
        for a, b in zip(list(got) + [d], want):
            assert torch.equal(a, b)
    bufs = [torch.zeros_like(a) for a in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.forward(x, t, logp=bufs[0], lse=bufs[1], entropy=bufs[2], top=bufs[3], top_logp=bufs[4])
        op.loss(x, t, g, dlogits=bufs[5])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(bufs, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("row_bytes,pad", [(24800, 0), (30000, 1), (50002, 0), (70000, 3),
                                           (100000, 1)])
def test_loss_of_many_rows(row_bytes, pad, act):
    """Rows that a block keeps a ring of, in two, three or more slots and by one, two or four
    teams; from rows without a target, masked and special ones, and in place."""
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    size = {"f32": 4, "bf16": 2}[act]
    T, V = 700, row_bytes // size
    r = np.random.default_rng(row_bytes)
    g = torch.Generator(device="cuda")
    g.manual_seed(row_bytes)
    x = torch.randn(T, V + pad, generator=g, device="cuda").mul_(3).to(DT[act])
    x[3], x[4, V // 2:], x[5], x[699] = -np.inf, -np.inf, 0, 7
    whole, x = x, x[:, :V]  # a gradient laid out otherwise would not go by the ring
    t = r.integers(0, V, T)
    t[::5] = -1
    t[6], t[7], t[4] = 0, V - 1, 1
    d, h = r.standard_normal(T).astype(np.float32), r.standard_normal(T).astype(np.float32)
    d[8], h[8] = 0, 0
    op = TTLogProbs(V, DT[act], scale=0.9)
    rows = np.r_[0:12, 150:156, 303:308, 600:606, 694:700]
    for dent in (None, h):
        e = None if dent is None else nan((T,), torch.float32)
        out = torch.full_like(whole, float("nan"))[:, :V]
        logp, lse, e, got = op.loss(x, _i32(t), _f32(d), None if dent is None else _f32(h),
                                    entropy=e, dlogits=out)
        some = lambda a: None if a is None else a[torch.from_numpy(rows).cuda()]  # noqa: E731
        _check_fwd(some(x), t[rows], 0.9, 0, (some(logp), some(lse), some(e)))
        _check_grad(some(x), t[rows], d[rows], None if dent is None else h[rows], 0.9, act,
                    some(got), "dlogits")
        # every row against the pass of its own, and in place
        other = op.backward(x, _i32(t), lse, _f32(d), e, None if dent is None else _f32(h))
        near = 2.0 ** -6 if act == "bf16" else 2.0 ** -14
        keep = torch.isfinite(lse)
        a, b = got[keep].double(), other[keep].double()
        bound = near * b.abs() + 2.0 ** -14 * (torch.tensor(d).cuda()[keep].abs()
                                              + torch.tensor(h).cuda()[keep].abs())[:, None]
        assert ((a - b).abs() <= bound).all()
        y = whole.clone()[:, :V]
        logp2, lse2, _, _ = op.loss(y, _i32(t), _f32(d), None if dent is None else _f32(h),
                                    dlogits=y)
        assert torch.equal(y, got) and torch.equal(logp, logp2) and torch.equal(lse, lse2)
    assert _status() == 0


@pytest.mark.parametrize("V", [13000, 32000, 50000])
def test_loss_wait_runs_out(V):
    """A row that never comes: the block's teams leave, the status says so, and the next call
    is right."""
    from tensor_train_compressed_tt_gb300 import ttc
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    T = 700
    x = torch.randn(T, V, device="cuda").bfloat16()
    t, g = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.ones(T, device="cuda")
    op = TTLogProbs(V)
    want = op.loss(x, t, g)
    torch.cuda.synchronize()
    ttc.check(ttc.tt_set_wait_limit_ns(20_000_000), "limit")
    try:
        ttc.check(ttc.tt_debug_skip_arrival(ttc.TT_DEBUG_LOGP_LOSS), "hook")
        op.loss(x, t, g)
        assert _status() == 5 and _status() == 0
        for a, b in zip(want, op.loss(x, t, g)):
            assert a is None or torch.equal(a, b)
        assert _status() == 0
    finally:
        torch.cuda.synchronize()
        ttc.check(ttc.tt_set_wait_limit_ns(2_000_000_000), "limit")


@pytest.mark.parametrize("V", [100, 3001, 20001])
def test_rows_beyond_32_bits(V):
    """Rows 2^30 elements apart: the third begins behind 2^31."""
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    stride = 1 << 30
    flat = torch.empty(2 * stride + V, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((3, V), (stride, 1))
    r = np.random.default_rng(V)
    x.copy_(torch.from_numpy(r.standard_normal((3, V)).astype(np.float32)))
    t, g = r.integers(0, V, 3), r.standard_normal(3).astype(np.float32)
    op = TTLogProbs(V, top=5)
    got = op.forward(x, _i32(t), entropy=nan((3,), torch.float32))
    _check_fwd(x, t, 1.0, 5, got)
    want = x.clone()
    op.loss(x, _i32(t), _f32(g), dlogits=x)
    _check_grad(want, t, g, None, 1.0, "bf16", x, "loss: dlogits")
    x.copy_(want)
    op.backward(x, _i32(t), got[1], _f32(g), dlogits=x)
    _check_grad(want, t, g, None, 1.0, "bf16", x, "dlogits", given=True)


def test_wrapper_refuses():
    from tensor_train_compressed_tt_gb300.layer import TTLogProbs
    op = TTLogProbs(64, torch.float32)
    x, t, g = torch.zeros(4, 64, device="cuda"), _i32([0] * 4), _f32([0] * 4)
    for bad in (x.bfloat16(), x[:, :32], x.t(), x.cpu(),
                torch.zeros(4, 128, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            op.forward(bad, t)
    for bad in (t.long(), t[:3], t.cpu()):
        with pytest.raises(ValueError):
            op.forward(x, bad)
    with pytest.raises(ValueError):
        op.forward(x, logp=g)
    with pytest.raises(ValueError):
        op.forward(x, t, top=torch.zeros(4, 0, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        op.loss(x, t)
    with pytest.raises(ValueError):
        op.loss(x, None, g)
    with pytest.raises(ValueError):
        op.backward(x, t, g, g, dentropy=g)
    with pytest.raises(ValueError):
        op.backward(x, t, None, g)
    with pytest.raises(ValueError):
        op.backward(x, t, g, g, dlogits=x[:, :63])
    from tensor_train_compressed_tt_gb300 import ttc
    with pytest.raises(ttc.TTError):
        op.forward(x[:1].expand(4, 64), t)  # rows on one another

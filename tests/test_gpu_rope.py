"""Norm of heads with rotation by position on the GPU against the fp64 oracle.

Bounds, element by element: half a step of the output's type, and fp32 errors of
U = 2^-24 for each operation on the way.  Forward: dim terms in the sum of squares
(half of its relative error reaches 1 / sqrt), some 16 operations besides (weight,
rotation, an angle rounded to 2^-27 of a half turn), on the largest value of the
head.  Backward: two sums of dim terms and some 32 operations, on the largest of the
terms that meet, r (|g'| + |h| mean |g' h|).  The weights' gradients are sums over
tokens and heads: U for each term that joins in a chain, at most the tokens and
heads of a warp and its merges, on the sum of the magnitudes."""

import numpy as np
import pytest

from oracle import token_oracle as K

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from token_util import DT, HALF, U, f64, nan, rand, within  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from tensor_train_compressed_tt_gb300 import _build
    _build.build()


def _status():
    from tensor_train_compressed_tt_gb300 import ttc
    return ttc.tt_get_device_status(torch.cuda.current_stream().cuda_stream)


def _strided(x, packed):
    """The same values in a buffer with gaps between heads and rows."""
    if not packed:
        return x
    T, H, D = x.shape
    pad = {1: 3, 2: 8}[packed]
    big = nan((T, H + 2, D + pad), x.dtype)
    big[:, 1:H + 1, :D] = x
    return big[:, 1:H + 1, :D]


def _plan(heads, kv, dim, act, rot=None, inter=False, eps=1e-5, base=10000.0, **kw):
    from tensor_train_compressed_tt_gb300.layer import TTRotary
    return TTRotary(heads, dim, kv_heads=kv, dtype=DT[act], rot=rot, base=base, interleaved=inter,
                    norm=eps > 0, eps=eps, **kw)


def _bound_fwd(ref, dim, act):
    return HALF[act] * np.abs(ref) + (dim / 2 + 16) * U * np.abs(ref).max(axis=2, keepdims=True)


def _bound_bwd(x, dy, g, eps, ref, act, pos, f, rot, inter):
    dim = ref.shape[2]
    gx = np.abs(K.rope_backward(x, dy, pos, f, rot, interleaved=inter)[0])
    big = gx.max(axis=2, keepdims=True) * np.sqrt(2)
    if eps > 0:
        if g is not None:
            big = big * np.abs(g).max()
        r = 1 / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps)
        h = np.abs(x * r)
        big = r * (big + h * (h.mean(axis=2, keepdims=True) * big))
    return HALF[act] * np.abs(ref) + (2 * dim + 32) * U * big


def _case(T, heads, kv, dim, act, rot=None, inter=False, eps=1e-5, packed=0, weights=True, far=0,
          seed=0, stream=None):
    r = np.random.default_rng(seed)
    rot = dim if rot is None else rot
    op = _plan(heads, kv, dim, act, rot, inter, eps)
    f = K.rope_freqs(rot)
    pos = far + r.integers(0, 5000, T)
    at = torch.from_numpy(pos.astype(np.int32)).cuda()
    x = {n: _strided(rand(r, (T, h, dim), act, 1.5), packed) for n, h in (("q", heads), ("k", kv))}
    dy = {n: _strided(rand(r, (T, h, dim), act), packed) for n, h in (("q", heads), ("k", kv))}
    g = {n: rand(r, dim, "f32", 0.3, 1.0) if eps > 0 and weights else None for n in "qk"}
    out = {n: _strided(nan(x[n].shape, DT[act]), packed) for n in "qk"}
    op.forward(x["q"], x["k"], at, g["q"], g["k"], q_out=out["q"], k_out=out["k"], stream=stream)
    d = {n: _strided(nan(x[n].shape, DT[act]), packed) for n in "qk"}
    got = op.backward(dy["q"], dy["k"], at, x["q"] if eps > 0 else None,
                      x["k"] if eps > 0 else None, g["q"], g["k"], dq_in=d["q"], dk_in=d["k"],
                      stream=stream)
    torch.cuda.synchronize()
    for i, n in enumerate("qk"):
        xs, ds, w = f64(x[n]), f64(dy[n]), f64(g[n])
        ref = K.rope_forward(xs, pos, f, rot, w, eps, inter)
        within(f64(out[n]), ref, _bound_fwd(ref, dim, act), n)
        rx, rg = K.rope_backward(xs, ds, pos, f, rot, w, eps, inter)
        within(f64(d[n]), rx, _bound_bwd(xs, ds, w, eps, rx, act, pos, f, rot, inter), "d" + n)
        if eps > 0:
            du = K.rope_backward(xs, ds, pos, f, rot, interleaved=inter)[0]
            h = xs / np.sqrt((xs * xs).mean(axis=2, keepdims=True) + eps)
            terms = np.abs(du * h).sum(axis=(0, 1))
            chain = T * xs.shape[1] / min(T, 64) + dim + 64
            within(f64(got[2 + i]), rg, chain * U * (terms + terms.max()), "dg" + n)
        else:
            assert got[2 + i] is None
    assert _status() == 0


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(1, 0), (2, 2), (7, 6), (8, 8), (20, 12), (24, 24), (40, 40),
                                     (64, 64), (64, 16), (80, 32), (96, 96), (128, 128), (128, 0),
                                     (129, 66), (160, 80), (250, 250), (256, 256)])
def test_widths(dim, rot, inter, act):
    _case(21, 6, 3, dim, act, rot, inter, seed=dim)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 300, 5000])
def test_token_counts(T, act):
    _case(T, 4, 1, 64, act, seed=T)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv", [(1, 1), (12, 12), (13, 1), (16, 4), (40, 8), (71, 71)])
def test_head_counts(heads, kv, act):
    _case(40, heads, kv, 32, act, seed=heads)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [1, 2])
@pytest.mark.parametrize("eps,weights", [(0.0, False), (1e-5, False), (0.5, True)])
def test_strides_and_forms(eps, weights, packed, act):
    """Gaps of an odd number of elements, and of eight; without norm, without weights."""
    for inter in (False, True):
        _case(50, 5, 5, 64, act, 32, inter, eps, packed, weights)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 6000, -(1 << 31)])
def test_far_positions(far):
    """The oracle's own angles are off by 2^-53 of their size, 5e-7 at the farthest: two
    rows of the bound of 16 operations of a bf16 output do not show it."""
    _case(60, 2, 2, 64, "bf16", far=far)


def test_far_positions_turn_exactly():
    """Powers of two as frequencies of a turn: the angle's fraction is known exactly."""
    from tensor_train_compressed_tt_gb300.layer import TTRotary
    turns = [2.0 ** -k for k in range(1, 31)]
    op = TTRotary(1, 60, dtype=torch.float32, freqs=[2 * np.pi * t for t in turns], norm=False)
    pos = np.array([0, 1, 2, 3, 12345678, 2 ** 31 - 1, -1, -2 ** 31, 1 << 29])
    x = torch.zeros(len(pos), 1, 60, device="cuda")
    x[..., :30] = 1
    y, _ = op.forward(x, x.clone(), torch.from_numpy(pos.astype(np.int32)).cuda())
    # the frequencies are doubles: 2 pi t and 1 / 2 pi are off by 2^-52, times 2^31 turns
    ang = 2 * np.pi * ((pos[:, None] * np.array(turns)[None]) % 1.0)
    bound = 16 * U + 2 * np.pi * 2.0 ** -51 * np.abs(pos)[:, None] * np.array(turns)[None]
    within(f64(y[:, 0, :30]), np.cos(ang), bound, "cos")
    within(f64(y[:, 0, 30:]), np.sin(ang), bound, "sin")


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_given_frequencies_and_default_positions(act):
    from tensor_train_compressed_tt_gb300.layer import TTRotary
    r = np.random.default_rng(3)
    f = r.uniform(-7, 7, 16)  # more than a turn a position, and backwards
    op = TTRotary(2, 32, dtype=DT[act], freqs=f, norm=False)
    x = rand(r, (100, 2, 32), act)
    y, z = op.forward(x, x.clone())
    ref = K.rope_forward(f64(x), np.arange(100), f, 32)
    within(f64(y), ref, _bound_fwd(ref, 32, act), "y")
    assert torch.equal(y, z)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_rows_of_zeros(eps, act):
    """A head of zeros stays zero; its gradient is 1 / sqrt(eps) of the output's."""
    op = _plan(2, 2, 64, act, eps=eps)
    x = torch.zeros(5, 2, 64, dtype=DT[act], device="cuda")
    y, _ = op.forward(x, x)
    assert float(y.float().abs().max()) == 0
    dy = torch.ones_like(x)
    dq, _, dgq, _ = op.backward(dy, dy, None, x, x) if eps else op.backward(dy, dy)
    assert torch.isfinite(dq.float()).all()
    if eps:
        assert float(dgq.abs().max()) == 0
        ref = K.rope_backward(f64(x), f64(dy), np.arange(5), K.rope_freqs(64), 64, None, eps)[0]
        # 16 operations besides the rounding
        within(f64(dq), ref, (HALF[act] + 16 * U) * np.abs(ref) + 16 * U * np.abs(ref).max(), "dq")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("T,heads,kv,dim", [(1, 12, 12, 64), (16, 16, 4, 80), (300, 3, 1, 33)])
def test_into_a_cache(T, heads, kv, dim, eps, act):
    """Keys and values of new tokens to rows of a cache; other rows stay as they were, a
    negative row is skipped, one outside is skipped and recorded."""
    r = np.random.default_rng(T)
    rot = dim // 2 // 2 * 2
    op = _plan(heads, kv, dim, act, rot, eps=eps)
    q, k, v = (rand(r, (T, h, dim), act) for h in (heads, kv, kv))
    pos = r.integers(0, 90000, T)
    n = 3 * T + 5
    rows = r.permutation(n)[:T]
    keys, values = nan((n, kv, dim), DT[act]), nan((n, kv, dim), DT[act])
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    yq, yk = op.forward(q, k, i32(pos))
    out, _, _ = op.to_cache(q, k, v, i32(pos), i32(rows), keys, values)
    assert torch.equal(out, yq)
    at = torch.from_numpy(rows).cuda()
    assert torch.equal(keys[at], yk) and torch.equal(values[at], v)
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.isnan(keys[rest].float()).all() and torch.isnan(values[rest].float()).all()
    assert _status() == 0
    if T < 3:
        return
    rows[0], rows[1], rows[2] = -1, n, 2 ** 31 - 1
    keys.fill_(float("nan")), values.fill_(float("nan"))
    out, _, _ = op.to_cache(q, k, v, i32(pos), i32(rows), keys, values)
    assert _status() != 0 and _status() == 0
    assert torch.equal(out, yq)
    at = at[3:]
    assert torch.equal(keys[at], yk[3:]) and torch.equal(values[at], v[3:])
    assert int(torch.isnan(keys[:, 0, 0].float()).sum()) == n - (T - 3)


@pytest.mark.parametrize("dim", [64, 33])
def test_a_cache_beyond_32_bits(dim):
    """Rows of the cache 2^26 + 8 elements apart: the last begins behind 2^31."""
    r = np.random.default_rng(dim)
    op = _plan(2, 2, dim, "bf16", rot=dim // 2 * 2)
    n, step = 34, (1 << 26) + 8
    flat = torch.empty(n * step, dtype=torch.bfloat16, device="cuda")
    keys = flat.as_strided((n, 2, dim), (step, dim, 1))
    values = flat.as_strided((n, 2, dim), (step, dim, 1), storage_offset=1 << 20)
    q, k, v = (rand(r, (3, 2, dim), "bf16") for _ in range(3))
    pos = torch.tensor([0, 9, 4], dtype=torch.int32, device="cuda")
    rows = torch.tensor([33, 0, 32], dtype=torch.int32, device="cuda")
    op.to_cache(q, k, v, pos, rows, keys, values)
    want = op.forward(q, k, pos)[1]
    assert torch.equal(keys[rows.long()], want) and torch.equal(values[rows.long()], v)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 33])
def test_in_place(dim, act):
    r = np.random.default_rng(4)
    op = _plan(6, 2, dim, act, rot=dim // 2 * 2)
    q, k, dq, dk = (rand(r, (200, h, dim), act) for h in (6, 2, 6, 2))
    y, z = op.forward(q, k)
    a, b = q.clone(), k.clone()
    op.forward(a, b, q_out=a, k_out=b)
    assert torch.equal(a, y) and torch.equal(b, z)
    want = op.backward(dq, dk, None, q, k)
    a, b = dq.clone(), dk.clone()
    got = op.backward(a, b, None, q, k, dq_in=a, dk_in=b)
    for s, t in zip(got, want):
        assert torch.equal(s, t)


@pytest.mark.parametrize("T", [20, 3000])
def test_gradients_repeat_accumulate_and_may_be_absent(T):
    from tensor_train_compressed_tt_gb300 import ttc
    r = np.random.default_rng(5)
    q, k, dq, dk = (rand(r, (T, h, 64), "bf16") for h in (6, 2, 6, 2))
    op, acc = _plan(6, 2, 64, "bf16"), _plan(6, 2, 64, "bf16", accumulate=True)
    first = op.backward(dq, dk, None, q, k)
    for _ in range(3):
        for a, b in zip(first, op.backward(dq, dk, None, q, k)):
            assert torch.equal(a, b)
    g = [rand(r, 64, "f32") for _ in range(2)]
    old = [t.clone() for t in g]
    acc.backward(dq, dk, None, q, k, dgq=g[0], dgk=g[1])
    for t, o, one in zip(g, old, first[2:]):
        assert torch.equal(t, o + one)
    made = acc.backward(dq, dk, None, q, k)
    assert torch.equal(made[2], first[2]) and torch.equal(made[3], first[3])
    # null weight gradients at the C entry
    h = lambda t: ttc.tt_heads(t.data_ptr(), t.stride(0), 64)  # noqa: E731
    ws, cur = op.workspace(T), torch.cuda.current_stream().cuda_stream
    for a, b in ((0, 0), (1, 0), (0, 1)):
        one, x, y = torch.zeros(64, device="cuda"), torch.empty_like(dq), torch.empty_like(dk)
        ttc.check(ttc.tt_rope_backward(op.plan, T, 0, h(q), h(k), 0, 0, h(dq), h(dk), h(x), h(y),
                                       one.data_ptr() * a, one.data_ptr() * b, ws.data_ptr(),
                                       ws.numel(), cur))
        assert torch.equal(x, first[0]) and torch.equal(y, first[1])
        if a or b:
            assert torch.equal(one, first[2 if a else 3])


def test_no_tokens():
    for accumulate in (False, True):
        op = _plan(2, 1, 32, "bf16", accumulate=accumulate)
        q, k = (torch.empty(0, h, 32, dtype=torch.bfloat16, device="cuda") for h in (2, 1))
        y, z = op.forward(q, k)
        assert y.shape == q.shape and z.shape == k.shape
        g = torch.ones(32, device="cuda")
        op.backward(q, k, None, q, k, dgq=g)
        assert torch.equal(g, torch.full_like(g, float(accumulate)))


def test_streams_and_graph():
    """On a given stream while the current one is busy, and captured."""
    r = np.random.default_rng(6)
    op = _plan(12, 12, 64, "bf16")
    q, k, dq, dk = (rand(r, (999, 12, 64), "bf16") for _ in range(4))
    y = op.forward(q, k)
    d = op.backward(dq, dk, None, q, k)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)
        got = op.forward(q, k, stream=side) + op.backward(dq, dk, None, q, k, stream=side)
        torch.cuda.synchronize()
        for a, b in zip(got, y + d):
            assert torch.equal(a, b)
    bufs = [torch.zeros_like(t) for t in y + d]
    ws = op.workspace(999)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.forward(q, k, q_out=bufs[0], k_out=bufs[1])
        op.backward(dq, dk, None, q, k, dq_in=bufs[2], dk_in=bufs[3], dgq=bufs[4], dgk=bufs[5],
                    ws=ws)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(bufs, y + d):
        assert torch.equal(a, b)


def test_wrapper_refuses():
    op = _plan(2, 1, 32, "bf16")
    q, k = (torch.zeros(4, h, 32, dtype=torch.bfloat16, device="cuda") for h in (2, 1))
    p = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[:, :, ::2]), dict(k=k[:3]), dict(q=q.cpu()),
                dict(pos=p.long()), dict(pos=p[:3]), dict(gq=torch.ones(31, device="cuda")),
                dict(gk=torch.ones(32, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            op.forward(**{"q": q, "k": k, "pos": p, **bad})
    with pytest.raises(ValueError):
        op.backward(q, k, p)
    with pytest.raises(ValueError):
        op.to_cache(q, k, k, p, p.long(), k.clone(), k.clone())
    with pytest.raises(ValueError):
        op.to_cache(q, k, k, p, p, k.clone(), k[:3].clone())
    flat = _plan(2, 1, 32, "bf16", eps=0.0)
    with pytest.raises(ValueError):
        flat.forward(q, k, p, gq=torch.ones(32, device="cuda"))
    with pytest.raises(ValueError):
        flat.backward(q, k, p, dgq=torch.ones(32, device="cuda"))

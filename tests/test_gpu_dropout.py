"""Dropout on the GPU, alone and in front of the normalisation, against the oracle.

Which elements stay is compared exactly.  Values: half a step of the output's type and
two fp32 operations (the scale, the sum) alone; with the normalisation its own
tolerances (block_util)."""

import numpy as np
import pytest

from block_util import NORM_TOL, assert_near
from oracle import block_oracle as B
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


def _case(shape, act, p=0.3, res=True, seed=5, offset=0, site=0):
    from tensor_train_compressed_tt_gb300.layer import TTDropout
    r = np.random.default_rng(1)
    op = TTDropout(p, DT[act], site=site)
    rng = op.state(seed, offset)
    x = rand(r, shape, act)
    x[x == 0] = 1  # so that a zero is a dropped one
    f = K.drop_factor(shape, p, seed, offset, site)
    y = op.forward(x, rng, y=nan(shape, DT[act]))
    assert np.array_equal(f64(y) != 0, f != 0)
    ref = f64(x) * f
    within(f64(y), ref, (HALF[act] + U) * np.abs(ref), "y")
    dx = op.backward(x, rng)
    assert torch.equal(dx, y)
    if res:
        rs = rand(r, shape, act)
        y = op.forward(x, rng, res=rs, y=nan(shape, DT[act]))
        full = ref + f64(rs)
        within(f64(y), full, HALF[act] * np.abs(full) + 2 * U * (np.abs(ref) + np.abs(f64(rs))),
               "y + res")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 100, 2047, 2048, 2049, 70003])
def test_lengths(n, act):
    _case((n,), act)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("p", [0.0, 1e-6, 2.0 ** -16, 0.1, 0.5, 0.999, 1.0])
def test_probabilities(p, act):
    _case((33, 65), act, p)


@pytest.mark.parametrize("seed,offset,site", [(0, 0, 0), (-1, 0, 0), (2 ** 63 - 1, -1, 65535),
                                              (-2 ** 63, 2 ** 40 + 3, 7)])
def test_state(seed, offset, site):
    _case((40, 24), "bf16", seed=seed, offset=offset, site=site)


def test_share_and_independence():
    """The share that stays, over 2^22 elements: six standard deviations of 0.9 +- 1.5e-4;
    two sites drop the same element at 0.01 +- 4.9e-5."""
    from tensor_train_compressed_tt_gb300.layer import TTDropout
    n = 1 << 22
    x = torch.ones(n, device="cuda")
    a, b = (TTDropout(0.1, torch.float32, site=s) for s in (0, 1))
    rng = a.state(11)
    ya, yb = a.forward(x, rng) == 0, b.forward(x, rng) == 0
    for y in (ya, yb):
        assert abs(float(y.double().mean()) - 0.1) < 6 * 1.5e-4 + 2.0 ** -17
    assert abs(float((ya & yb).double().mean()) - 0.01) < 6 * 4.9e-5 + 2.0 ** -19


def test_dropped_elements_are_zero_whatever_they_held():
    from tensor_train_compressed_tt_gb300.layer import TTDropout
    op = TTDropout(0.5, torch.float32)
    rng = op.state(3)
    stay = op.forward(torch.ones(5000, device="cuda"), rng) != 0
    for v in (float("nan"), float("inf")):
        y = op.forward(torch.full((5000,), v, device="cuda"), rng)
        assert (y[~stay] == 0).all() and not torch.isfinite(y[stay]).any()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_in_place(act):
    from tensor_train_compressed_tt_gb300.layer import TTDropout
    r = np.random.default_rng(2)
    op = TTDropout(0.2, DT[act])
    rng, x, rs = op.state(4), rand(r, (300, 77), act), rand(r, (300, 77), act)
    y = op.forward(x, rng, res=rs)
    a = x.clone()
    op.forward(a, rng, res=rs, y=a)
    b = rs.clone()
    op.forward(x, rng, res=b, y=b)
    assert torch.equal(a, y) and torch.equal(b, y)


def test_elements_beyond_32_bits():
    """2^32 + 77 elements: the groups' index keeps its high bits, first, middle and last."""
    from tensor_train_compressed_tt_gb300.layer import TTDropout
    n = (1 << 32) + 77
    op = TTDropout(0.5, site=3)
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    op.forward(x, op.state(21), y=x)
    for first in (0, (1 << 31) - 40, (1 << 32) - 40, n - 60):
        keep = K.drop_bits(60, 21, 0, 3, first=first) >= 32768
        assert np.array_equal(f64(x[first:first + 60]), 2.0 * keep)


def test_a_graph_takes_the_offset_of_each_replay():
    from tensor_train_compressed_tt_gb300.layer import TTDropNorm, TTDropout
    r = np.random.default_rng(6)
    x, rs = rand(r, (100, 768), "bf16"), rand(r, (100, 768), "bf16")
    op, dn = TTDropout(0.1), TTDropNorm(768, 0.1, site=1)
    rng = op.state(9)
    y, z, s, st = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x), \
        torch.zeros(100, 2, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.forward(x, rng, y=y)
        dn.forward(x, rng, res=rs, y=z, sum=s, stats=st)
        rng[1] += 1
    seen = []
    for k in range(3):
        g.replay()
        now = op.state(9, k)
        assert torch.equal(y, op.forward(x, now))
        want = dn.forward(x, now, res=rs)
        for a, b in zip((z, s, st), want):
            assert torch.equal(a, b)
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1]) and int(rng[1]) == 3


def _norm_case(T, N, act, p=0.25, res=True, affine=True, seed=0, accumulate=False, site=2):
    from tensor_train_compressed_tt_gb300.layer import TTDropNorm
    r = np.random.default_rng(seed)
    op = TTDropNorm(N, p, DT[act], site=site, accumulate=accumulate)
    rng = op.drop.state(seed + 1, 3)
    f = K.drop_factor((T, N), p, seed + 1, 3, site)
    x = rand(r, (T, N), act, mean=0.5)
    rs = rand(r, (T, N), act) if res else None
    gamma = rand(r, N, "f32", 0.3, 1.0) if affine else None
    beta = rand(r, N, "f32", 0.3) if affine else None
    y, s, st = op.forward(x, rng, gamma, beta, res=rs, y=nan((T, N), DT[act]),
                          sum=nan((T, N), DT[act]), stats=nan((T, 2), torch.float32))
    ry, rsum, rst = B.norm_forward(f64(x) * f, f64(gamma), f64(beta), f64(rs))
    assert_near(f64(y), ry, NORM_TOL[act], "y")
    assert_near(f64(s), rsum, NORM_TOL[act], "sum")
    assert_near(f64(st), rst, 1e-5, "stats")
    if not res:
        assert np.array_equal(f64(s) != 0, f != 0)
    dy, dsum = rand(r, (T, N), act), rand(r, (T, N), act) if res else None
    _, _, st = op.norm.forward(s)  # the statistics of the rounded sum
    old = rand(r, (2, N), "f32")
    dg, db = (old[0].clone(), old[1].clone()) if accumulate else (None, None)
    dx, dres, dg, db = op.backward(s, dy, rng, gamma, st, dsum=dsum, dx=nan((T, N), DT[act]),
                                   dres=nan((T, N), DT[act]) if res else None, residual=res,
                                   dgamma=dg, dbeta=db)
    rx, rg, rb = B.norm_backward(f64(s), f64(dy), f64(gamma), f64(dsum))
    if accumulate:
        rg, rb = rg + f64(old[0]), rb + f64(old[1])
    assert_near(f64(dx), rx * f, NORM_TOL[act], "dx")
    assert (f64(dx)[f == 0] == 0).all()
    if res:
        assert_near(f64(dres), rx, NORM_TOL[act], "dres")
    else:
        assert dres is None
    assert_near(f64(dg), rg, 1e-5, "dgamma")
    assert_near(f64(db), rb, 1e-5, "dbeta")
    return op, rng, (x, rs, gamma, beta), (s, dy, gamma, st, dsum), (dx, dres, dg, db)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("N", [2, 7, 8, 12, 64, 255, 256, 512, 513, 768, 1000, 1023, 1024, 1028,
                               2048, 4096, 8200, 16384, 16385])
def test_norm_widths(N, act):
    _norm_case(13, N, act, seed=N)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 33, 257, 1200])
@pytest.mark.parametrize("N", [64, 767, 768])
def test_norm_token_counts(T, N, act):
    _norm_case(T, N, act, seed=T)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("N", [8, 512, 768, 1024, 1028, 4096, 16384, 17000])
def test_norm_weights_off_a_16_byte_boundary(N, act):
    from tensor_train_compressed_tt_gb300.layer import TTDropNorm
    r = np.random.default_rng(7)
    T, op = 37, TTDropNorm(N, 0.25, DT[act], site=2)
    rng = op.drop.state(4, 3)
    f = K.drop_factor((T, N), 0.25, 4, 3, 2)
    x, rs, dy = (rand(r, (T, N), act) for _ in range(3))
    gamma, beta = rand(r, N + 1, "f32", 0.3, 1.0)[1:], rand(r, N + 1, "f32", 0.3)[1:]
    assert gamma.data_ptr() % 16 and beta.data_ptr() % 16
    y, s, st = op.forward(x, rng, gamma, beta, res=rs, y=nan((T, N), DT[act]),
                          sum=nan((T, N), DT[act]), stats=nan((T, 2), torch.float32))
    ry, rsum, rst = B.norm_forward(f64(x) * f, f64(gamma), f64(beta), f64(rs))
    assert_near(f64(y), ry, NORM_TOL[act], "y")
    assert_near(f64(s), rsum, NORM_TOL[act], "sum")
    assert_near(f64(st), rst, 1e-5, "stats")
    _, _, st = op.norm.forward(s)  # the statistics of the rounded sum
    dx, _, dg, db = op.backward(s, dy, rng, gamma, st, dx=nan((T, N), DT[act]))
    rx, rg, rb = B.norm_backward(f64(s), f64(dy), f64(gamma))
    assert_near(f64(dx), rx * f, NORM_TOL[act], "dx")
    assert_near(f64(dg), rg, 1e-5, "dgamma")
    assert_near(f64(db), rb, 1e-5, "dbeta")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("N", [768, 1023, 17000])
def test_norm_without_residual_and_weights(N, act):
    _norm_case(20, N, act, res=False, affine=False)
    _norm_case(20, N, act, res=False, accumulate=True)


@pytest.mark.parametrize("p", [0.0, 0.9, 1.0])
def test_norm_probabilities(p):
    _norm_case(30, 768, "bf16", p)


def test_norm_without_dropout_is_the_norm():
    from tensor_train_compressed_tt_gb300.layer import TTDropNorm
    r = np.random.default_rng(8)
    op = TTDropNorm(768, 0.0)
    x, rs = rand(r, (200, 768), "bf16"), rand(r, (200, 768), "bf16")
    for a, b in zip(op.forward(x, op.drop.state(1), res=rs), op.norm.forward(x, res=rs)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("N", [768, 1023, 17000])
def test_norm_in_place_and_repeats(N):
    op, rng, fwd, bwd, want = _norm_case(300 if N < 2000 else 20, N, "bf16")
    x, rs, gamma, beta = fwd
    y, s, st = op.forward(x, rng, gamma, beta, res=rs)
    a, b = x.clone(), rs.clone()
    op.forward(a, rng, gamma, beta, res=b, sum=a, y=b)
    assert torch.equal(a, s) and torch.equal(b, y)
    s, dy, gamma, st, dsum = bwd
    d, u = dy.clone(), dsum.clone()
    got = op.backward(s, d, rng, gamma, st, dsum=u, dx=d, dres=u)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    d, u = dy.clone(), dsum.clone()
    got = op.backward(s, d, rng, gamma, st, dsum=u, dx=u, dres=d)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_no_elements_and_refusals():
    from tensor_train_compressed_tt_gb300.layer import TTDropNorm, TTDropout
    op = TTDropout(0.5)
    rng = op.state(1)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert op.forward(x, rng).shape == (0, 64)
    dn = TTDropNorm(64, 0.5)
    dn.forward(x, rng)
    _, _, dg, _ = dn.backward(x, x, rng, None, torch.empty(0, 2, device="cuda"))
    assert float(dg.abs().max()) == 0
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(x=x.float()), dict(x=x.t()), dict(rng=rng.int()), dict(rng=rng[:1]),
                dict(rng=None), dict(rng=rng.cpu()), dict(res=x[:2])):
        with pytest.raises(ValueError):
            op.forward(**{"x": x, "rng": rng, **bad})
        with pytest.raises(ValueError):
            dn.forward(**{"x": x, "rng": rng, **bad})

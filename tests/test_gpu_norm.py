"""Layer normalisation on the GPU against the fp64 oracle."""

import numpy as np
import pytest

from block_util import NORM_TOL, assert_near
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from tensor_train_compressed_tt_gb300 import _build
    _build.build()


def _rand(r, shape, act, mean=0.0, scale=1.0):
    x = torch.from_numpy((mean + scale * r.standard_normal(shape)).astype(np.float32))
    return x.to(DT[act]).cuda()


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _case(T, N, act, res=True, affine=True, eps=1e-5, mean=0.5, seed=0, stream=None,
          accumulate=False):
    from tensor_train_compressed_tt_gb300.layer import TTNorm
    r = np.random.default_rng(seed)
    op = TTNorm(N, DT[act], eps=eps, accumulate=accumulate)
    x = _rand(r, (T, N), act, mean)
    rs = _rand(r, (T, N), act) if res else None
    gamma = _rand(r, N, "f32", 1.0, 0.3) if affine else None
    beta = _rand(r, N, "f32", 0.0, 0.3) if affine else None
    nan = lambda *s, dt=DT[act]: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    y, s, st = op.forward(x, gamma, beta, res=rs, y=nan(T, N), sum=nan(T, N) if res else None,
                          stats=nan(T, 2, dt=torch.float32), stream=stream)
    ry, rsum, rst = B.norm_forward(_np(x), _np(gamma), _np(beta), _np(rs), eps)
    assert_near(_np(y), ry, NORM_TOL[act], "y")
    # means near zero are held to the statistics' own scale
    assert_near(_np(st), rst, 1e-5, "stats")
    if res:
        assert_near(_np(s), rsum, NORM_TOL[act], "sum")
    else:
        assert s is None
        s = x
    dy = _rand(r, (T, N), act)
    dsum = _rand(r, (T, N), act) if res else None
    old = _rand(r, (2, N), "f32")
    dg, db = (old[0].clone(), old[1].clone()) if accumulate else \
        (nan(N, dt=torch.float32), nan(N, dt=torch.float32))
    # the backward's own statistics: what was stored of s, rounded
    _, _, st = op.forward(s)
    dx, dg, db = op.backward(s, dy, gamma, st, dsum=dsum, dx=nan(T, N), dgamma=dg, dbeta=db,
                             stream=stream)
    rx, rg, rb = B.norm_backward(_np(s), _np(dy), _np(gamma), _np(dsum), eps)
    if accumulate:
        rg, rb = rg + _np(old[0]), rb + _np(old[1])
    assert_near(_np(dx), rx, NORM_TOL[act], "dx")
    assert_near(_np(dg), rg, 1e-5, "dgamma")
    assert_near(_np(db), rb, 1e-5, "dbeta")
    return op, s, dy, gamma, st, dsum, (dx, dg, db)


WIDTHS = [2, 7, 8, 64, 255, 256, 257, 512, 513, 768, 769, 1000, 1023, 1024, 1030, 2048, 2049, 4096,
          4100, 8192, 8200, 16384, 16385, 20001]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("N", WIDTHS)
def test_widths(N, act):
    _case(37, N, act)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 257, 5000])
@pytest.mark.parametrize("N", [64, 768, 1023, 2048])
def test_token_counts(T, N, act):
    _case(T, N, act, seed=T)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_width_one_and_constant_rows(act):
    """A row without spread normalises to beta and has a zero-mean gradient."""
    from tensor_train_compressed_tt_gb300.layer import TTNorm
    for N in (1, 64, 1023):
        x = torch.full((5, N), 3.0, dtype=DT[act], device="cuda")
        op = TTNorm(N, DT[act])
        beta = torch.arange(N, dtype=torch.float32, device="cuda")
        y, _, st = op.forward(x, None, beta)
        assert torch.equal(y, beta.to(DT[act]).expand(5, N))
        dx, dg, db = op.backward(x, torch.ones_like(x), None, st)
        assert float(dx.float().abs().max()) == 0 and float(dg.abs().max()) == 0
        assert torch.equal(db, torch.full_like(db, 5.0))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_without_residual_and_weights(act):
    _case(100, 768, act, res=False, affine=False)
    _case(100, 768, act, res=False, affine=True)
    _case(100, 96, act, res=True, affine=False, eps=0.3)


def test_large_mean_keeps_the_variance():
    """Mean 1000 times the spread: the variance comes from the centred values."""
    _case(64, 768, "f32", res=False, mean=0.0)
    from tensor_train_compressed_tt_gb300.layer import TTNorm
    r = np.random.default_rng(3)
    x = _rand(r, (64, 768), "f32", 1000.0)
    y, _, st = TTNorm(768, torch.float32).forward(x)
    ry, _, rst = B.norm_forward(_np(x))
    # the mean is rounded to 2^-24 of 1000, 6e-5 of the spread
    assert np.abs(_np(y) - ry).max() < 4e-4 and np.abs(_np(st)[:, 1] / rst[:, 1] - 1).max() < 1e-5


@pytest.mark.parametrize("N", [64, 768, 4096, 20001])
def test_accumulate(N):
    _case(300, N, "bf16", accumulate=True)


@pytest.mark.parametrize("N", [768, 1023, 4096, 20001])
def test_gradients_are_bit_reproducible(N):
    op, s, dy, gamma, st, dsum, first = _case(3000 if N < 5000 else 100, N, "bf16")
    for _ in range(3):
        again = op.backward(s, dy, gamma, st, dsum=dsum)
        for a, b in zip(first, again):
            assert torch.equal(a, b)


def test_no_tokens():
    from tensor_train_compressed_tt_gb300.layer import TTNorm
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    for acc in (False, True):
        op = TTNorm(64, accumulate=acc)
        y, _, st = op.forward(x)
        g = torch.ones(64, device="cuda")
        dx, dg, db = op.backward(x, x, None, st, dgamma=g, dbeta=g.clone())
        assert y.shape == dx.shape == (0, 64)
        assert torch.equal(dg, torch.full_like(dg, float(acc))) and torch.equal(dg, db)


@pytest.mark.parametrize("N", [768, 1023, 4096, 20001])
def test_in_place(N):
    """sum over x, y over res, dx over dy: each row is read before it is written."""
    from tensor_train_compressed_tt_gb300.layer import TTNorm
    r = np.random.default_rng(4)
    op = TTNorm(N)
    x, res, dy = (_rand(r, (200, N), "bf16") for _ in range(3))
    y, s, st = op.forward(x, res=res)
    x2, res2 = x.clone(), res.clone()
    op.forward(x2, res=res2, sum=x2, y=res2)
    assert torch.equal(x2, s) and torch.equal(res2, y)
    dx, dg, db = op.backward(s, dy, None, st)
    d2 = dy.clone()
    _, dg2, db2 = op.backward(s, d2, None, st, dx=d2)
    assert torch.equal(d2, dx) and torch.equal(dg, dg2) and torch.equal(db, db2)


def test_only_asked_gradients():
    """Null dgamma, dbeta, stats and sum at the C entry."""
    from tensor_train_compressed_tt_gb300 import ttc
    from tensor_train_compressed_tt_gb300.layer import TTNorm
    op = TTNorm(768)
    x = _rand(np.random.default_rng(5), (300, 768), "bf16")
    y, _, st = op.forward(x)
    dx, dg, db = op.backward(x, y, None, st)
    ws, cur = op.workspace(300), torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr()  # noqa: E731
    y2, dx2, one = torch.empty_like(y), torch.empty_like(dx), torch.empty_like(dg)
    ttc.check(ttc.tt_norm_forward(op.plan, 300, p(x), p(x), 0, 0, 0, p(y2), 0, cur))
    for g, b in ((0, 0), (p(one), 0), (0, p(one))):
        ttc.check(ttc.tt_norm_backward(op.plan, 300, p(x), p(y), 0, 0, p(st), p(dx2), g, b, p(ws),
                                       ws.numel(), cur))
        assert torch.equal(dx, dx2)
        if g:
            assert torch.equal(one, dg)
        if b:
            assert torch.equal(one, db)


def test_another_stream_and_graph():
    from tensor_train_compressed_tt_gb300.layer import TTNorm
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _case(500, 768, "bf16")
    r = np.random.default_rng(6)
    op, x, dy = TTNorm(768), _rand(r, (999, 768), "bf16"), _rand(r, (999, 768), "bf16")
    y, _, st = op.forward(x)
    dx, dg, db = op.backward(x, dy, None, st)
    bufs = [torch.zeros_like(t) for t in (y, st, dx, dg, db)]
    ws = op.workspace(999)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.forward(x, y=bufs[0], stats=bufs[1])
        op.backward(x, dy, None, bufs[1], dx=bufs[2], dgamma=bufs[3], dbeta=bufs[4], ws=ws)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(bufs, (y, st, dx, dg, db)):
        assert torch.equal(a, b)


def test_wrapper_refuses():
    from tensor_train_compressed_tt_gb300.layer import TTNorm
    op = TTNorm(64)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x[:, :32], x.t(), x.cpu(), torch.zeros(4, 128, dtype=x.dtype, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            op.forward(bad)
    with pytest.raises(ValueError):
        op.forward(x, gamma=torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        op.forward(x, res=x[:2])


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1028, 2048, 4096, 8192])
@pytest.mark.parametrize("T", [2432, 2433, 5001])
def test_many_rows_without_a_residual(T, N, act):
    """Two rows at a time, and the last row of a block alone (from 16 rows an SM)."""
    _case(T, N, act, res=False, seed=T + N)


@pytest.mark.parametrize("accumulate", [False, True])
def test_default_gradients_on_a_given_stream(accumulate):
    """stream= another one than the current, which is busy: the weight gradients
    that the call makes are the kernel's."""
    from tensor_train_compressed_tt_gb300.layer import TTNorm
    r = np.random.default_rng(8)
    op = TTNorm(768, accumulate=accumulate)
    x, dy = _rand(r, (300, 768), "bf16"), _rand(r, (300, 768), "bf16")
    _, _, st = op.forward(x)
    dx, dg, db = op.backward(x, dy, None, st)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)   # some 10 ms
        got = op.backward(x, dy, None, st, stream=side)
        torch.cuda.synchronize()
        for a, b in zip((dx, dg, db), got):
            assert torch.equal(a, b)

"""Refusals of the layer normalisation and attention entry points (host only:
every call here returns before anything is enqueued)."""

import ctypes

import pytest

from tensor_train_compressed_tt_gb300 import ttc

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
F32, BF16, E4M3 = ttc.TT_DT_F32, ttc.TT_DT_BF16, ttc.TT_DT_E4M3


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tensor_train_compressed_tt_gb300 import _build
    _build.build()
    return ttc.lib()


def _code(fn, *a):
    with pytest.raises(ttc.TTError) as e:
        fn(*a)
    return e.value.code


@pytest.mark.parametrize("args,code", [
    ((0, 1e-5, BF16), INVALID), ((8, 0.0, BF16), INVALID), ((8, float("nan"), BF16), INVALID),
    ((8, float("inf"), BF16), INVALID), ((8, 1e-5, 7), INVALID),
    ((8, 1e-5, BF16, ttc.TT_REUSE_Z), INVALID), ((8, 1e-5, E4M3), UNSUPPORTED),
    (((1 << 20) + 1, 1e-5, F32), UNSUPPORTED)])
def test_norm_plan_refuses(args, code):
    assert _code(ttc.tt_norm_plan, *args) == code


def _attn(heads=4, kv=2, dim=64, left=-1, right=0, sinks=0, scale=0.0, act=BF16, flags=0):
    return ttc.tt_attn_plan(heads, kv, dim, left, right, sinks, scale, act, flags)


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), INVALID), (dict(heads=1025, kv=1), INVALID), (dict(kv=3), INVALID),
    (dict(kv=0), INVALID), (dict(dim=0), INVALID), (dict(sinks=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(act=9), INVALID), (dict(flags=1), INVALID),
    (dict(dim=257), UNSUPPORTED), (dict(act=E4M3), UNSUPPORTED)])
def test_attn_plan_refuses(kw, code):
    with pytest.raises(ttc.TTError) as e:
        _attn(**kw)
    assert e.value.code == code


def test_plans_of_another_kind_are_refused():
    norm, attn = ttc.tt_norm_plan(64, 1e-5, F32), _attn()
    lin = ttc.tt_plan(ttc.make_desc((4, 4), (4, 4), (1, 4, 4, 4, 1), F32))
    s = ttc.tt_attn_seqs()
    h = ttc.tt_heads()
    for p in (attn, lin):
        assert ttc.tt_norm_forward(p, 1, 256, 0, 0, 0, 0, 256, 0) == INVALID
        assert ttc.tt_norm_backward(p, 1, 256, 256, 0, 0, 256, 256, 0, 0, 256, 1 << 20) == INVALID
    for p in (norm, lin):
        assert ttc.tt_attn_forward(p, s, h, h, h, h, 0, 0, 0) == INVALID
        assert ttc.tt_attn_backward(p, s, h, h, h, h, 0, h, h, h, h, 0, 0) == INVALID
        assert _code(ttc.tt_attn_workspace_size, p, s, True) == INVALID
    for p in (norm, attn):
        assert ttc.tt_forward(p, 1, 256, 256, 256, 256, 1 << 20) == INVALID
        n = ctypes.c_size_t()
        buf = (ctypes.c_size_t * 8)()
        assert ttc.lib().tt_param_layout(p.handle, buf, buf, ctypes.byref(n)) == INVALID
    assert _code(ttc.tt_workspace_size, attn, 4) == INVALID


def test_norm_arguments():
    p = ttc.tt_norm_plan(64, 1e-5, F32)
    ok = 4096   # an address that passes the alignment checks; never dereferenced here
    assert ttc.tt_norm_forward(p, -1, ok, 0, 0, 0, 0, ok, 0) == INVALID
    assert ttc.tt_norm_forward(p, 0, 0, 0, 0, 0, 0, 0, 0) == 0
    for bad in ((0, 0, 0, 0, 0, ok, 0), (ok, 0, 0, 0, 0, 0, 0), (ok + 8, 0, 0, 0, 0, ok, 0),
                (ok, ok + 4, 0, 0, 0, ok, 0), (ok, 0, ok + 2, 0, 0, ok, 0),
                (ok, 0, 0, ok + 1, 0, ok, 0), (ok, 0, 0, 0, ok + 8, ok, 0),
                (ok, 0, 0, 0, 0, ok + 8, 0), (ok, 0, 0, 0, 0, ok, ok + 4)):
        assert ttc.tt_norm_forward(p, 4, *bad) == INVALID, bad
    n = ttc.tt_workspace_size(p, 4)
    good = [ok, ok, 0, 0, ok, ok, 0, 0]   # s dy dsum gamma stats dx dgamma dbeta
    for i, v in ((0, 0), (1, 0), (4, 0), (5, 0), (0, ok + 8), (2, ok + 8), (3, ok + 2),
                 (6, ok + 2), (7, ok + 1)):
        bad = list(good)
        bad[i] = v
        assert ttc.tt_norm_backward(p, 4, *bad, ok, n) == INVALID, (i, v)
    assert ttc.tt_norm_backward(p, 4, *good, 0, n) == WORKSPACE
    assert ttc.tt_norm_backward(p, 4, *good, ok + 16, n) == WORKSPACE
    assert ttc.tt_norm_backward(p, 4, *good, ok, n - 1) == WORKSPACE


def _seqs(B=1, max_q=8, max_k=8, Tq=8, Tk=8, at=4096):
    return ttc.tt_attn_seqs(B, max_q, max_k, Tq, Tk, at, at, at, at)


def test_attn_arguments():
    p = _attn(4, 2, 64)
    h = ttc.tt_heads(4096, 256, 64)
    ok, ws = _seqs(), 1 << 20
    run = lambda s, *hs: ttc.tt_attn_forward(p, s, *hs, 0, 4096, ws)  # noqa: E731
    for s in (_seqs(B=-1), _seqs(B=(1 << 20) + 1), _seqs(max_q=-1), _seqs(max_k=-1),
              _seqs(max_k=(1 << 29) + 1), _seqs(Tq=-1), _seqs(Tk=1 << 31), _seqs(at=0),
              _seqs(at=4098)):
        assert run(s, h, h, h, h) == INVALID
        assert _code(ttc.tt_attn_workspace_size, p, s, True) == INVALID
        assert ttc.tt_attn_backward(p, s, h, h, h, h, 4096, h, h, h, h, 4096, ws) == INVALID
    for bad in (ttc.tt_heads(0, 256, 64), ttc.tt_heads(4097, 256, 64), ttc.tt_heads(4096, -1, 64),
                ttc.tt_heads(4096, 256, -1)):
        for i in range(4):
            hs = [h] * 4
            hs[i] = bad
            assert run(ok, *hs) == INVALID
        for i in range(8):
            hs = [h] * 8
            hs[i] = bad
            assert ttc.tt_attn_backward(p, ok, *hs[:4], 4096, *hs[4:], 4096, ws) == INVALID
    assert ttc.tt_attn_forward(p, ok, h, h, h, h, 4098, 4096, ws) == INVALID
    assert ttc.tt_attn_backward(p, ok, h, h, h, h, 0, h, h, h, h, 4096, ws) == INVALID
    n = ttc.tt_attn_workspace_size(p, ok, True)
    assert n >= 4 * 8 * 4
    for at, size in ((0, n), (4096 + 16, n), (4096, n - 1)):
        assert ttc.tt_attn_backward(p, ok, h, h, h, h, 4096, h, h, h, h, at, size) == WORKSPACE
    # nothing to do: no launch, no pointer needed
    none = ttc.tt_heads(0, 256, 64)
    assert ttc.tt_attn_forward(p, _seqs(B=0, Tq=0, Tk=0, at=0), none, none, none, none, 0, 0, 0) == 0


def test_null_arguments():
    L = ttc.lib()
    assert L.tt_norm_plan(None, None) == INVALID
    out = ctypes.c_void_p()
    assert L.tt_norm_plan(None, ctypes.byref(out)) == INVALID
    assert L.tt_attn_plan(None, ctypes.byref(out)) == INVALID
    p = _attn()
    assert L.tt_attn_forward(p.handle, None, None, None, None, None, None, None, 0, None) == INVALID
    assert L.tt_attn_forward(None, None, None, None, None, None, None, None, 0, None) == INVALID

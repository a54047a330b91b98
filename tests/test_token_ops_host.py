"""Refusals of the entry points of rotary positions, log probabilities and dropout, and
whose memory their wrappers take (host only: nothing is enqueued)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

from tensor_train_compressed_tt_gb300 import layer, ttc  # noqa: E402
from test_wrapper_streams_host import FakeStream, made  # noqa: E402, F401

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
F32, BF16, E4M3 = ttc.TT_DT_F32, ttc.TT_DT_BF16, ttc.TT_DT_E4M3
OK = 4096  # an address that passes the alignment checks; never dereferenced here
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tensor_train_compressed_tt_gb300 import _build
    _build.build()
    return ttc.lib()


def _code(fn, *a):
    with pytest.raises(ttc.TTError) as e:
        fn(*a)
    return e.value.code


def _rope(heads=4, kv=2, dim=64, rot=64, base=1e4, freqs=None, inter=False, eps=1e-5, act=BF16,
          flags=0):
    return ttc.tt_rope_plan(heads, kv, dim, rot, base, freqs, inter, eps, act, flags)


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), INVALID), (dict(heads=1025, kv=1), INVALID), (dict(kv=3), INVALID),
    (dict(kv=0), INVALID), (dict(dim=0), INVALID), (dict(rot=-2), INVALID),
    (dict(rot=63), INVALID), (dict(rot=66), INVALID), (dict(base=0.0), INVALID),
    (dict(base=-3.0), INVALID), (dict(base=NAN), INVALID), (dict(base=INF), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=0.0, rot=0), INVALID),
    (dict(act=9), INVALID), (dict(flags=2), INVALID), (dict(dim=257, rot=2), UNSUPPORTED),
    (dict(act=E4M3), UNSUPPORTED), (dict(freqs=[NAN] * 32), INVALID),
    (dict(freqs=[INF] * 32), INVALID)])
def test_rope_plan_refuses(kw, code):
    with pytest.raises(ttc.TTError) as e:
        _rope(**kw)
    assert e.value.code == code


def test_rope_frequencies():
    with pytest.raises(ValueError):
        _rope(freqs=[1.0] * 31)
    _rope(freqs=[1.0] * 32, base=0.0)  # base is not read
    _rope(rot=0, base=NAN)


@pytest.mark.parametrize("args,code", [
    ((0, 1.0, 0, BF16), INVALID), ((8, 0.0, 0, BF16), INVALID), ((8, NAN, 0, BF16), INVALID),
    ((8, -1.0, 0, BF16), INVALID), ((8, 1e7, 0, BF16), INVALID), ((8, 1.0, -1, BF16), INVALID),
    ((8, 1.0, 9, BF16), INVALID), ((8, 1.0, 0, 5), INVALID), ((8, 1.0, 0, E4M3), UNSUPPORTED),
    (((1 << 24) + 1, 1.0, 0, F32), UNSUPPORTED), ((800, 1.0, 65, F32), UNSUPPORTED)])
def test_logp_plan_refuses(args, code):
    assert _code(ttc.tt_logp_plan, *args) == code


@pytest.mark.parametrize("args,code", [
    ((-0.1, 0, BF16), INVALID), ((1.1, 0, BF16), INVALID), ((NAN, 0, BF16), INVALID),
    ((0.5, -1, BF16), INVALID), ((0.5, 65536, BF16), INVALID), ((0.5, 0, 7), INVALID),
    ((0.5, 0, E4M3), UNSUPPORTED)])
def test_dropout_plan_refuses(args, code):
    assert _code(ttc.tt_dropout_plan, *args) == code


def test_plans_of_another_kind_are_refused():
    rope, logp = _rope(), ttc.tt_logp_plan(64, 1.0, 0, BF16)
    drop = ttc.tt_dropout_plan(0.5, 0, BF16)
    norm = ttc.tt_norm_plan(64, 1e-5, BF16)
    h = ttc.tt_heads(OK, 64, 64)
    for p in (logp, drop, norm):
        assert ttc.tt_rope_forward(p, 1, 0, h, h, 0, 0, h, h, None, None, 0, 0) == INVALID
        assert ttc.tt_rope_backward(p, 1, 0, h, h, 0, 0, h, h, h, h, 0, 0, OK, 1 << 20) == INVALID
    for p in (rope, drop, norm):
        assert ttc.tt_logp_forward(p, 1, OK, 64, OK, OK, OK, 0, 0, 0) == INVALID
        assert ttc.tt_logp_backward(p, 1, OK, 64, OK, OK, OK, 0, 0, OK, 64) == INVALID
        assert ttc.tt_logp_loss(p, 1, OK, 64, OK, OK, 0, OK, OK, 0, OK, 64) == INVALID
    for p in (rope, logp, norm):
        assert ttc.tt_dropout(p, 8, OK, OK, 0, OK) == INVALID
        assert ttc.tt_norm_dropout_forward(norm, p, 1, OK, OK, 0, 0, 0, OK, OK, OK) == INVALID
    other = ttc.tt_dropout_plan(0.5, 0, F32)  # of another activation type
    assert ttc.tt_norm_dropout_forward(norm, other, 1, OK, OK, 0, 0, 0, OK, OK, OK) == INVALID
    assert ttc.tt_norm_dropout_forward(rope, drop, 1, OK, OK, 0, 0, 0, OK, OK, OK) == INVALID
    assert ttc.tt_norm_dropout_backward(norm, other, 1, OK, OK, OK, 0, 0, OK, OK, OK + 64, 0, 0,
                                        OK, 1 << 20) == INVALID
    n = ctypes.c_size_t()
    buf = (ctypes.c_size_t * 8)()
    for p in (rope, logp, drop):
        assert ttc.tt_forward(p, 1, 256, 256, 256, 256, 1 << 20) == INVALID
        assert ttc.tt_norm_forward(p, 1, 256, 0, 0, 0, 0, 256, 0) == INVALID
        assert ttc.lib().tt_param_layout(p.handle, buf, buf, ctypes.byref(n)) == INVALID
    assert ttc.tt_workspace_size(logp, 4) == ttc.tt_workspace_size(drop, 4) == 0
    assert ttc.tt_workspace_size(_rope(eps=0.0), 4) == 0 < ttc.tt_workspace_size(rope, 4)


def test_rope_arguments():
    p, flat = _rope(), _rope(eps=0.0)
    h = ttc.tt_heads(OK, 256, 64)

    def fwd(pl=p, T=4, pos=0, hs=(h,) * 4, gq=0, gk=0, v=None, vo=None, rows=0, n=0):
        return ttc.tt_rope_forward(pl, T, pos, hs[0], hs[1], gq, gk, hs[2], hs[3], v, vo, rows, n)

    bads = (ttc.tt_heads(0, 256, 64), ttc.tt_heads(OK + 1, 256, 64), ttc.tt_heads(OK, -1, 64),
            ttc.tt_heads(OK, 256, -1))
    for kw in (dict(T=-1), dict(T=1 << 31), dict(pos=OK + 2), dict(gq=OK + 2), dict(gk=OK + 1),
               dict(rows=OK + 2, n=8), dict(rows=OK, n=-1), dict(v=h), dict(vo=h),
               dict(pl=flat, gq=OK), dict(pl=flat, gk=OK)):
        assert fwd(**kw) == INVALID, kw
    for bad in bads:
        for i in range(4):
            hs = [h] * 4
            hs[i] = bad
            assert fwd(hs=hs) == INVALID
        assert fwd(v=bad, vo=h) == INVALID and fwd(v=h, vo=bad) == INVALID
    none = ttc.tt_heads(0, 256, 64)
    assert fwd(T=0, hs=(none,) * 4) == 0
    ws = ttc.tt_workspace_size(p, 4)

    def bwd(pl=p, T=4, hs=(h,) * 6, g=(0,) * 4, at=OK, n=ws):
        return ttc.tt_rope_backward(pl, T, 0, hs[0], hs[1], g[0], g[1], hs[2], hs[3], hs[4], hs[5],
                                    g[2], g[3], at, n)

    for bad in bads:
        for i in range(6):
            hs = [h] * 6
            hs[i] = bad
            assert bwd(hs=hs) == INVALID, i
    for i in range(4):
        g = [0] * 4
        g[i] = OK + 2
        assert bwd(g=g) == INVALID
        g[i] = OK
        assert bwd(pl=flat, g=g) == INVALID
    for at, n in ((0, ws), (OK + 16, ws), (OK, ws - 1)):
        assert bwd(at=at, n=n) == WORKSPACE
    assert bwd(T=-1) == INVALID
    L = ttc.lib()
    assert L.tt_rope_forward(p.handle, 4, *([None] * 10), 0, None) == INVALID
    assert L.tt_rope_forward(None, 4, *([None] * 10), 0, None) == INVALID
    assert L.tt_rope_plan(None, None) == INVALID


def test_logp_arguments():
    p, top = ttc.tt_logp_plan(64, 1.0, 0, BF16), ttc.tt_logp_plan(64, 1.0, 4, BF16)
    good = dict(T=4, logits=OK, stride=64, targets=OK, logp=OK, lse=OK, entropy=OK, top=0,
                top_logp=0)
    for bad in (dict(T=-1), dict(T=1 << 31), dict(logits=0), dict(logits=OK + 1), dict(stride=63),
                dict(stride=-64), dict(stride=(1 << 31) + 1), dict(targets=OK + 2),
                dict(targets=0), dict(logp=OK + 2), dict(lse=OK + 1), dict(entropy=OK + 2),
                dict(top=OK), dict(top_logp=OK), dict(top=OK, top_logp=OK)):
        assert ttc.tt_logp_forward(p, **{**good, **bad}) == INVALID, bad
    for bad in (dict(top=OK), dict(top_logp=OK), dict(top=OK + 2, top_logp=OK),
                dict(top=OK, top_logp=OK + 2)):
        assert ttc.tt_logp_forward(top, **{**good, **bad}) == INVALID, bad
    good = dict(T=4, logits=OK, stride=64, targets=OK, lse=OK, dlogp=OK, entropy=OK, dentropy=OK,
                dlogits=OK, dstride=64)
    for bad in (dict(T=-1), dict(logits=0), dict(stride=63), dict(dstride=63),
                dict(dstride=(1 << 31) + 1), dict(targets=0), dict(lse=0), dict(lse=OK + 2),
                dict(dlogp=0, dentropy=0), dict(entropy=0), dict(dlogits=0), dict(dlogits=OK + 1),
                dict(dlogp=OK + 2), dict(dentropy=OK + 2), dict(entropy=OK + 2)):
        assert ttc.tt_logp_backward(p, **{**good, **bad}) == INVALID, bad
    good = dict(T=4, logits=OK, stride=64, targets=OK, dlogp=OK, dentropy=OK, logp=OK, lse=OK,
                entropy=OK, dlogits=OK, dstride=64)
    for bad in (dict(T=-1), dict(logits=0), dict(stride=63), dict(dstride=63), dict(targets=0),
                dict(dlogp=0, dentropy=0), dict(dlogits=0), dict(dlogits=OK + 1),
                dict(logp=OK + 2), dict(lse=OK + 2), dict(entropy=OK + 2), dict(dlogp=OK + 2)):
        assert ttc.tt_logp_loss(p, **{**good, **bad}) == INVALID, bad
    assert ttc.tt_logp_forward(p, 0, 0, 64, 0, 0, 0, 0, 0, 0) == 0
    out = ctypes.c_void_p()
    assert ttc.lib().tt_logp_plan(None, ctypes.byref(out)) == INVALID
    assert ttc.lib().tt_logp_plan(None, None) == INVALID


def test_dropout_arguments():
    p, norm = ttc.tt_dropout_plan(0.5, 0, BF16), ttc.tt_norm_plan(64, 1e-5, BF16)
    good = dict(n=8, rng=OK, x=OK, res=0, y=OK)
    for bad in (dict(n=-1), dict(n=1 << 48), dict(rng=0), dict(rng=OK + 4), dict(x=0),
                dict(x=OK + 8), dict(res=OK + 8), dict(y=0), dict(y=OK + 2)):
        assert ttc.tt_dropout(p, **{**good, **bad}) == INVALID, bad
    assert ttc.tt_dropout(p, 0, 0, 0, 0, 0) == 0
    for rng in (0, OK + 4):
        assert ttc.tt_norm_dropout_forward(norm, p, 4, rng, OK, 0, 0, 0, 0, OK, 0) == INVALID
    ws = ttc.tt_workspace_size(norm, 4)
    bwd = lambda rng=OK, dx=OK, dres=OK + 1024, at=OK, n=ws: ttc.tt_norm_dropout_backward(  # noqa: E731
        norm, p, 4, rng, OK, OK, 0, 0, OK, dx, dres, 0, 0, at, n)
    for bad in (dict(rng=0), dict(rng=OK + 2), dict(dx=0), dict(dres=OK + 8), dict(dres=OK)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(n=ws - 1) == WORKSPACE and bwd(at=0) == WORKSPACE


# ---- whose memory the wrappers take ---------------------------------------------------

@pytest.fixture
def fake(made, monkeypatch):  # noqa: F811
    for name in ("tt_rope_forward", "tt_rope_backward", "tt_logp_forward", "tt_logp_backward",
                 "tt_logp_loss", "tt_dropout", "tt_norm_dropout_forward",
                 "tt_norm_dropout_backward"):
        monkeypatch.setattr(ttc, name, lambda *a: 0)
    monkeypatch.setattr(layer, "_heads_of", lambda *a: None)
    monkeypatch.setattr(layer.TTLogProbs, "_rows", lambda self, t, n, name: (0, self.V))
    return made


def _run_rope(s):
    op = layer.TTRotary(2, 32, dtype=torch.float32)
    q, p = torch.ones(4, 2, 32), torch.ones(4, dtype=torch.int32)
    op.forward(q, q, p, stream=s)
    op.backward(q, q, p, q, q, stream=s)
    op.to_cache(q, q, q, p, p, q, q, stream=s)


def _run_logp(s):
    op = layer.TTLogProbs(16, torch.float32, top=3)
    x, t, g = torch.ones(4, 16), torch.ones(4, dtype=torch.int32), torch.ones(4)
    op.forward(x, t, stream=s)
    op.backward(x, t, g, g, stream=s)
    op.loss(x, t, g, stream=s)


def _run_drop(s):
    op, dn = layer.TTDropout(0.5, torch.float32), layer.TTDropNorm(16, 0.5, torch.float32)
    x, rng = torch.ones(4, 16), torch.ones(2, dtype=torch.int64)
    op.forward(x, rng, stream=s)
    op.backward(x, rng, stream=s)
    dn.forward(x, rng, stream=s)
    dn.backward(x, x, rng, None, torch.ones(4, 2), stream=s)


@pytest.mark.parametrize("run", [_run_rope, _run_logp, _run_drop])
def test_memory_is_the_calls_streams(fake, monkeypatch, run):
    log, held = fake
    real = torch.ones
    inside = FakeStream()
    run(inside)
    mine = [at for _, at in log]
    assert mine and all(at is inside for at in mine)
    assert held and all(s == "current" for _, s in held)
    del log[:], held[:]
    run(None)
    assert log and all(at is None for _, at in log) and not held
    assert real is torch.ones


def test_weight_gradients_that_are_added_to_start_at_zero(fake, monkeypatch):
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: real(*a, **k).fill_(7))
    q = torch.ones(4, 2, 32)
    for g in layer.TTRotary(2, 32, dtype=torch.float32, accumulate=True).backward(
            q, q, None, q, q)[2:]:
        assert float(g.abs().max()) == 0
    dn = layer.TTDropNorm(16, 0.5, torch.float32, accumulate=True)
    x = torch.ones(4, 16)
    for g in dn.backward(x, x, torch.ones(2, dtype=torch.int64), None, torch.ones(4, 2))[2:]:
        assert float(g.abs().max()) == 0


def test_a_tensor_of_another_device_is_refused(monkeypatch):
    class Elsewhere:
        device = torch.device("cuda:1")

        def get_device(self):
            return 1
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError):
        layer._same_device(None, Elsewhere())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    layer._same_device(Elsewhere(), None, torch.ones(1))

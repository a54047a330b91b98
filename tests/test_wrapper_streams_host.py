"""What the wrappers allocate or fill by themselves belongs to the call's stream
(host only: the library's calls and the streams are stand-ins that record)."""

import contextlib

import pytest

torch = pytest.importorskip("torch")

from tensor_train_compressed_tt_gb300 import layer, ttc  # noqa: E402


class FakeStream:
    cuda_stream = 77


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tensor_train_compressed_tt_gb300 import _build
    _build.build()


@pytest.fixture
def made(monkeypatch):
    """(function, stream current at the time) of every tensor made, and the tensors
    whose memory was held for another stream."""
    log, now = [], [None]

    @contextlib.contextmanager
    def stream(s):
        old, now[0] = now[0], s
        yield
        now[0] = old

    def recorder(name, real):
        def make(*a, **k):
            log.append((name, now[0]))
            return real(*a, **k)
        return make

    for name in ("empty", "zeros", "full"):
        monkeypatch.setattr(torch, name, recorder(name, getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "current")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    held = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: held.append((t.shape, s)))
    monkeypatch.setattr(layer, "_dense", lambda t, *a: 0 if t is None else t.data_ptr())
    for name in ("tt_norm_forward", "tt_norm_backward", "tt_attn_forward", "tt_attn_backward",
                 "tt_forward", "tt_backward", "tt_ffn_forward", "tt_ffn_backward",
                 "tt_multi_forward", "tt_multi_backward", "tt_ttm_lookup",
                 "tt_ttm_lookup_backward"):
        monkeypatch.setattr(ttc, name, lambda *a: 0)
    return log, held


def _norm(accumulate=False):
    op = layer.TTNorm(64, torch.float32, accumulate=accumulate)
    x, st = torch.ones(4, 64), torch.ones(4, 2)
    return op, x, st


@pytest.mark.parametrize("accumulate", [False, True])
def test_norm_weight_gradients_are_filled_on_the_calls_stream(made, accumulate):
    log, _ = made
    op, x, st = _norm(accumulate)
    s = FakeStream()
    del log[:]
    _, dg, db = op.backward(x, x, None, st, stream=s)
    fills = [at for name, at in log if name in ("zeros", "full")]
    assert fills == ([s, s] if accumulate else [])   # overwritten unless added to
    if accumulate:
        assert float(dg.abs().max()) == 0 and float(db.abs().max()) == 0

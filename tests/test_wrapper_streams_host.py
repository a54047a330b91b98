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


def _attn():
    op = layer.TTAttention(2, 32, dtype=torch.float32)
    off = torch.tensor([0, 4], dtype=torch.int32)
    return op, torch.ones(4, 2, 32), layer.TTSeqs.packed(off, 4, 4)


def _run_norm(s):
    op, x, st = _norm()
    op.forward(x, res=x, stream=s)
    op.backward(x, x, None, st, stream=s)


def _run_attn(s):
    op, q, seqs = _attn()
    o, lse = op.forward(q, q, q, seqs, stream=s)
    op.backward(q, q, q, o, lse, q, seqs, stream=s)


def _run_linear(s):
    op = layer.TTLinear((4, 4), (4, 4), (1, 4, 4, 4, 1), torch.float32)
    x, p = torch.ones(3, 16), torch.ones(op.n_params)
    op.forward(x, p, stream=s)
    op.backward(x, x, p, stream=s)


def _run_ffn(s):
    m = ((4, 4), (4, 4), (1, 4, 4, 4, 1))
    op = layer.TTFFN(m, m, torch.float32)
    x, p = torch.ones(3, 16), torch.ones(200)
    op.forward(x, p, p, stream=s)
    op.backward(x, x, p, p, stream=s)


def _run_multi(s):
    m = ((4, 4), (4, 4), (1, 4, 4, 4, 1))
    op = layer.TTMulti([m, m], torch.float32)
    x, p = torch.ones(3, 16), torch.ones(200)
    op.forward(x, [p, p], stream=s)
    op.backward(x, [x, x], [p, p], stream=s)


def _run_ttm(s):
    op = layer.TTMEmbedding((4, 4), (4, 4), (1, 4, 1))
    idx, p = torch.ones(3, dtype=torch.int32), torch.ones(op.n_params)
    out = op.lookup(idx, p, stream=s)
    op.backward(idx, out, p, stream=s)


RUNS = [_run_norm, _run_attn, _run_linear, _run_ffn, _run_multi, _run_ttm]


@pytest.mark.parametrize("run", RUNS)
def test_memory_is_the_calls_streams(made, monkeypatch, run):
    """Outputs and workspaces that the caller does not give: from the memory of the
    stream that the kernels run on, where a workspace that is dropped at the call's
    end is next used after them; outputs are held for the caller's stream too."""
    log, held = made
    monkeypatch.setattr(layer.TTAttention, "_heads", lambda *a: None)
    inside = FakeStream()
    run(inside)
    mine = [at for _, at in log]
    assert mine and all(at is inside for at in mine)
    assert held and all(s == "current" for _, s in held)
    del log[:], held[:]
    run(None)
    assert log and all(at is None for _, at in log) and not held


def _linear():
    op = layer.TTLinear((4, 4), (4, 4), (1, 4, 4, 4, 1), torch.float32, accumulate=True)
    x = torch.ones(3, 16)
    return [op.backward(x, x, torch.ones(op.n_params))[1]]


def _ffn():
    m = ((4, 4), (4, 4), (1, 4, 4, 4, 1))
    x, p = torch.ones(3, 16), torch.ones(200)
    return list(layer.TTFFN(m, m, torch.float32, accumulate=True).backward(x, x, p, p)[1:])


def _multi():
    m = ((4, 4), (4, 4), (1, 4, 4, 4, 1))
    x, p = torch.ones(3, 16), torch.ones(200)
    return list(layer.TTMulti([m, m], torch.float32, accumulate=True).backward(
        x, [x, x], [p, p])[1])


def _ttm():
    op = layer.TTMEmbedding((4, 4), (4, 4), (1, 4, 1), accumulate=True)
    out = torch.ones(3, 16)
    return [op.backward(torch.ones(3, dtype=torch.int32), out, torch.ones(op.n_params))]


@pytest.mark.parametrize("run", [_linear, _ffn, _multi, _ttm])
def test_gradients_that_are_added_to_start_at_zero(made, monkeypatch, run):
    """accumulate=True and no gradient given: the kernel adds to what the call makes."""
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: real(*a, **k).fill_(7))
    for g in run():
        assert float(g.abs().max()) == 0

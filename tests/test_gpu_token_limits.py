"""Ends of the ranges of rotary positions, log probabilities and dropout on the GPU against the
fp64 oracle, at the bounds of their other tests (test_gpu_rope, test_gpu_logp)."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tensor_train_compressed_tt_gb300.layer import TTLogProbs  # noqa: E402
from test_gpu_logp import _check_grad, _f32, _i32, _rows, _status  # noqa: E402
from token_util import DT, nan, rand  # noqa: E402


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

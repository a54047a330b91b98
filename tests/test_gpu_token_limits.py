"""Ends of the ranges of rotary positions, log probabilities and dropout on the GPU."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from token_util import rand  # noqa: E402


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

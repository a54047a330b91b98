"""Ends of the ranges of rotary positions, log probabilities and dropout (host only: nothing is
enqueued)."""

import pytest

torch = pytest.importorskip("torch")

from tensor_train_compressed_tt_gb300 import ttc  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tensor_train_compressed_tt_gb300 import _build
    _build.build()
    return ttc.lib()


def _rope(heads, kv, dim=64, act=ttc.TT_DT_BF16):
    return ttc.tt_rope_plan(heads, kv, dim, dim, 1e4, None, False, 1e-5, act, 0)


@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 2), (8, 1), (12, 12), (71, 71), (1024, 1024)])
def test_rope_workspace_of_no_tokens(heads, kv):
    """An empty batch has a workspace of a size, whatever the number of heads."""
    assert 0 < ttc.tt_workspace_size(_rope(heads, kv), 0) <= \
        ttc.tt_workspace_size(_rope(heads, kv), 1)

"""Ends of the ranges of rotary positions, log probabilities and dropout (host only: nothing is
enqueued)."""

import pytest

torch = pytest.importorskip("torch")

from tensor_train_compressed_tt_gb300 import layer, ttc  # noqa: E402
from tensor_train_compressed_tt_gb300.encoder import TTTokenHead, TTTransformerBlock  # noqa: E402
from tensor_train_compressed_tt_gb300.layer import TTRotary, TTSeqs  # noqa: E402


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


def test_a_block_with_an_accumulating_rotary_starts_at_zero(monkeypatch):
    """The block's buffers of gradients that are added to hold zeros, the others' nothing."""
    real = torch.empty
    monkeypatch.setattr(layer, "_dense", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(torch, "empty", lambda *a, **k: real(*a, **k).fill_(7))
    seqs = TTSeqs.packed(torch.tensor([0, 4], dtype=torch.int32), 4, 4)
    for accumulate in (True, False):
        block = TTTransformerBlock(12, rotary=TTRotary(12, 64, accumulate=accumulate))
        b = block.buffers(4, seqs, device="cpu")
        for nm in ("dgq", "dgk"):
            assert b[nm].shape == (64,) and (b[nm] == (0 if accumulate else 7)).all()


def _block(**kw):
    return TTTransformerBlock(12, **kw)


def _head(**kw):
    return TTTokenHead((12, 8, 8), (16, 16, 20), ttc.tt_default_ranks((12, 8, 8), (16, 16, 20), 30),
                       **kw)


@pytest.mark.parametrize("make", [_block, _head])
def test_a_share_that_is_none_is_refused(make):
    """Not taken as no dropout."""
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(ValueError, match="dropout"):
            make(dropout=p, site=0)
    for p in (0.0, 0.1, 1.0):
        make(dropout=p, site=0)


@pytest.mark.parametrize("make", [_block, _head])
def test_dropout_in_a_model_has_places_of_its_own(make):
    """Blocks and a head that all took the same site would drop the same elements."""
    for p in (0.1, 1.0):
        with pytest.raises(ValueError, match="site"):
            make(dropout=p)
        make(dropout=p, site=7)
    make(dropout=0.0)
    make()
    for site in (-1, 65536):
        with pytest.raises(ttc.TTError):
            make(dropout=0.1, site=site)

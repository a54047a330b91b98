"""The oracle of layer normalisation and attention, pinned by differences and closed forms."""

import numpy as np
import pytest

from oracle import block_oracle as B


def _diff(f, x, w, eps=1e-6):
    """Central differences of <w, f(x)> in every element of x."""
    g = np.zeros_like(x)
    for at in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[at] += eps
        b[at] -= eps
        g[at] = ((w * (f(a) - f(b))).sum()) / (2 * eps)
    return g


def test_norm_forward_rows_have_the_asked_mean_and_spread():
    r = np.random.default_rng(0)
    x, res = r.normal(3, 2, (7, 33)), r.normal(0, 1, (7, 33))
    y, s, st = B.norm_forward(x, res=res, eps=1e-12)
    assert np.allclose(s, x + res)
    assert np.allclose(y.mean(1), 0) and np.allclose(y.std(1), 1)
    y2, _, _ = B.norm_forward(x, np.full(33, 2.0), np.full(33, -1.0), res=res, eps=1e-12)
    assert np.allclose(y2, 2 * y - 1)


def test_norm_backward_against_differences():
    r = np.random.default_rng(1)
    s, dy, dsum = (r.normal(0, 1, (3, 6)) for _ in range(3))
    gamma, beta = r.normal(1, 0.3, 6), r.normal(0, 1, 6)
    dx, dg, db = B.norm_backward(s, dy, gamma, dsum)
    f = lambda a: B.norm_forward(a, gamma, beta)[0]  # noqa: E731
    assert np.allclose(dx, _diff(f, s, dy) + dsum, atol=1e-7)
    assert np.allclose(dg, _diff(lambda a: B.norm_forward(s, a, beta)[0], gamma, dy), atol=1e-7)
    assert np.allclose(db, _diff(lambda a: B.norm_forward(s, gamma, a)[0], beta, dy), atol=1e-7)


def test_attn_mask_closed_forms():
    assert B.attn_mask(3, 3, -1, 0, 0).tolist() == np.tril(np.ones((3, 3), bool)).tolist()
    m = B.attn_mask(1, 6, 1, 0, 2)   # the last token: itself, one before it, two first ones
    assert m.tolist() == [[True, True, False, False, True, True]]
    assert not B.attn_mask(4, 2, -1, 0, 0)[:2].any()   # positions -2 and -1 see no key


def test_attn_uniform_when_scores_are_equal():
    q, k = np.zeros((4, 1, 3)), np.ones((4, 1, 3))
    v = np.arange(12.0).reshape(4, 1, 3)
    o, lse = B.attn_forward(q, k, v, [(0, 4, 0, 4)], right=0)
    assert np.allclose(o[2, 0], v[:3, 0].mean(0)) and np.allclose(lse[0, 2], np.log(3))


@pytest.mark.parametrize("left,right,sinks", [(-1, -1, 0), (1, 0, 1), (1, 1, 0), (0, 0, 0)])
def test_attn_backward_against_differences(left, right, sinks):
    r = np.random.default_rng(2)
    q, k, v = r.normal(0, 1, (5, 4, 2)), r.normal(0, 1, (6, 2, 2)), r.normal(0, 1, (6, 2, 2))
    do = r.normal(0, 1, q.shape)
    seqs = [(0, 2, 0, 3), (2, 5, 3, 6)]
    kw = dict(left=left, right=right, sinks=sinks)
    dq, dk, dv = B.attn_backward(q, k, v, do, seqs, **kw)
    assert np.allclose(dq, _diff(lambda a: B.attn_forward(a, k, v, seqs, **kw)[0], q, do), atol=1e-7)
    assert np.allclose(dk, _diff(lambda a: B.attn_forward(q, a, v, seqs, **kw)[0], k, do), atol=1e-7)
    assert np.allclose(dv, _diff(lambda a: B.attn_forward(q, k, a, seqs, **kw)[0], v, do), atol=1e-7)

"""Pins of the oracle of rotary positions, log probabilities and dropout (CPU)."""

import numpy as np
import pytest

from oracle import token_oracle as K


@pytest.mark.parametrize("counter,key,words", [
    ([0] * 4, [0] * 2, [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
    ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
     [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1])])
def test_philox_known_answers(counter, key, words):
    """The published known-answer vectors of Philox 4x32 with ten rounds."""
    assert K.philox(counter, key) == words


def test_drop_bits_are_uniform_and_split_by_site_and_offset():
    a = K.drop_bits(4096, 7, 0, 0)
    # mean of n uniform values: standard deviation 65536 / sqrt(12 n) = 296
    assert abs(a.mean() - 32767.5) < 6 * 296
    for other in (K.drop_bits(4096, 8, 0, 0), K.drop_bits(4096, 7, 1, 0),
                  K.drop_bits(4096, 7, 0, 1), K.drop_bits(4096, 7, 1 << 32, 0)):
        assert (a != other).mean() > 0.99
    assert np.array_equal(K.drop_bits(10, 7, 0, 0, first=3), a[3:13])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(6, 6), (7, 4), (8, 0)])
def test_rope_gradient_by_differences(dim, rot, inter):
    r = np.random.default_rng(dim)
    x, w = r.standard_normal((3, 2, dim)), r.standard_normal((3, 2, dim))
    g, pos, f = r.uniform(0.5, 1.5, dim), np.array([0, 5, -3]), K.rope_freqs(rot, 100.0)
    args = dict(pos=pos, freqs=f, rot=rot, eps=1e-3, interleaved=inter)
    L = lambda x, g: (w * K.rope_forward(x, g=g, **args)).sum()  # noqa: E731
    dx, dg = K.rope_backward(x, w, g=g, **args)
    h = 1e-6
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((L(x + e, g) - L(x - e, g)) / (2 * h) - dx[at]) < 1e-7
    for c in range(dim):
        e = np.zeros(dim)
        e[c] = h
        assert abs((L(x, g + e) - L(x, g - e)) / (2 * h) - dg[c]) < 1e-7


def test_rotation_depends_on_the_distance_alone():
    r = np.random.default_rng(1)
    q, k, f = r.standard_normal((1, 1, 8)), r.standard_normal((1, 1, 8)), K.rope_freqs(8)
    turn = lambda x, p: K.rope_forward(x, np.array([p]), f, 8)  # noqa: E731
    a = (turn(q, 11) * turn(k, 4)).sum()
    assert abs(a - (turn(q, 1007) * turn(k, 1000)).sum()) < 1e-10
    assert np.allclose(K.rope_forward(q, np.array([0]), f, 8), q)


def test_logp_gradient_by_differences():
    r = np.random.default_rng(2)
    x = r.standard_normal((4, 9))
    x[1, 3] = -np.inf
    t = np.array([2, 0, -1, 8])
    a, b = r.standard_normal(4), r.standard_normal(4)

    def L(x):
        logp, _, ent, _, _ = K.logp_forward(x, t, 1.3)
        return (a * logp + b * ent).sum()

    d, _ = K.logp_backward(x, t, a, b, 1.3)
    h = 1e-6
    for at in np.ndindex(x.shape):
        if np.isinf(x[at]):
            assert d[at] == 0
            continue
        e = np.zeros_like(x)
        e[at] = h
        assert abs((L(x + e) - L(x - e)) / (2 * h) - d[at]) < 1e-7


def test_logp_special_rows():
    x = np.array([[0.0, 0.0, 0.0, 0.0], [-np.inf] * 4, [3.0, -np.inf, 3.0, 1.0]])
    logp, lse, ent, ids, tops = K.logp_forward(x, np.array([1, 2, 1]), top=4)
    assert np.allclose(lse[0], np.log(4)) and np.allclose(ent[0], np.log(4))
    assert lse[1] == -np.inf and logp[1] == -np.inf and ent[1] == 0 and logp[2] == -np.inf
    assert ids.tolist() == [[0, 1, 2, 3], [0, 1, 2, 3], [0, 2, 3, 1]]
    assert np.all(tops[1] == -np.inf) and tops[2, 3] == -np.inf

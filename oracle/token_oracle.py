"""fp64 oracle of the operators around attention and loss: norm of heads with rotation
by position, log probabilities with entropy and top alternatives and their gradient,
and dropout from Philox 4x32.  Plain definitions; shares no code with the library."""

from __future__ import annotations

import numpy as np


# ---- norm of heads and rotation by position -----------------------------------------

def rope_freqs(rot, base=10000.0):
    return np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _turn(u, pos, freqs, rot, interleaved, sign):
    a, b = _pairs(rot, interleaved)
    ang = np.asarray(pos, np.float64)[:, None, None] * freqs
    c, s = np.cos(ang), sign * np.sin(ang)
    y = u.copy()
    y[..., a] = u[..., a] * c - u[..., b] * s
    y[..., b] = u[..., a] * s + u[..., b] * c
    return y


def rope_forward(x, pos, freqs, rot, g=None, eps=0.0, interleaved=False):
    """x (T, heads, dim); eps == 0: no norm."""
    u = np.asarray(x, np.float64)
    if eps > 0:
        u = u / np.sqrt((u * u).mean(axis=2, keepdims=True) + eps)
        if g is not None:
            u = u * np.asarray(g, np.float64)
    return _turn(u, pos, freqs, rot, interleaved, 1.0)


def rope_backward(x, dy, pos, freqs, rot, g=None, eps=0.0, interleaved=False):
    """(dx, dg) for L = <dy, y>; dg is None without a norm."""
    du = _turn(np.asarray(dy, np.float64), pos, freqs, rot, interleaved, -1.0)
    if eps == 0:
        return du, None
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps)
    h = x * r
    gx = du if g is None else du * np.asarray(g, np.float64)
    return r * (gx - h * (gx * h).mean(axis=2, keepdims=True)), (du * h).sum(axis=(0, 1))


# ---- log probabilities ------------------------------------------------------------------

def log_p(z):
    """(log p, lse) of a row.  The maximum comes off first: beside logits of 1e38 the
    logarithm of the sum would be lost in lse, in 64 bits too."""
    with np.errstate(over="ignore"):
        d = z - z.max()
    logs = np.log(np.exp(d).sum())
    return d - logs, z.max() + logs


def logp_forward(x, targets=None, scale=1.0, top=0):
    """(logp, lse, entropy, top indices, their log probabilities), row by row."""
    x = np.asarray(x, np.float64)
    T, V = x.shape
    lse, ent = np.full(T, -np.inf), np.zeros(T)
    logp = np.zeros(T)
    ids = np.zeros((T, top), np.int64)
    tops = np.full((T, top), -np.inf)
    for t in range(T):
        z = scale * x[t]
        m = z.max()
        if m > -np.inf:
            lp, lse[t] = log_p(z)
            live = lp > -np.inf
            ent[t] = -(np.exp(lp[live]) * lp[live]).sum()
        else:
            lp = z
        if targets is not None and targets[t] >= 0:
            logp[t] = lp[targets[t]]
        order = sorted(range(V), key=lambda v: (-x[t, v], v)) if top and V <= 64 else \
            np.lexsort((np.arange(V), -x[t]))
        for k in range(top):
            ids[t, k] = order[k]
            tops[t, k] = lp[order[k]]
    return logp, lse, ent, ids, tops


def logp_backward(x, targets, dlogp=None, dentropy=None, scale=1.0):
    """(dlogits, size): size bounds the terms that meet in each element."""
    x = np.asarray(x, np.float64)
    _, lse, ent, _, _ = logp_forward(x, scale=scale)
    d, size = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[0]):
        if lse[t] == -np.inf:
            continue
        lp = log_p(scale * x[t])[0]
        p = np.exp(lp)
        if dlogp is not None and targets[t] >= 0:
            d[t] -= dlogp[t] * p
            d[t, targets[t]] += dlogp[t]
            size[t] += abs(dlogp[t]) * p
            size[t, targets[t]] += abs(dlogp[t])
        if dentropy is not None:
            live = p > 0
            plp = np.zeros_like(p)
            plp[live] = p[live] * (lp[live] + ent[t])
            d[t] -= dentropy[t] * plp
            # lp + ent is a sum of two numbers of errors of their own, which stay where it is 0
            size[t, live] += abs(dentropy[t]) * p[live] * (1 + np.abs(lp[live]) + ent[t])
    return scale * d, scale * size


# ---- dropout ----------------------------------------------------------------------------

def philox(counter, key, rounds=10):
    """Philox 4x32 (Salmon et al., 2011): four words of Python integers."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def drop_bits(n, seed, offset, site, first=0):
    """The 16 bits of elements first .. first + n."""
    seed, offset = seed & (1 << 64) - 1, offset & (1 << 64) - 1
    low = (1 << 32) - 1
    out = np.empty(n, np.int64)
    words, group = None, -1
    for j in range(n):
        i = first + j
        if i >> 3 != group:
            group = i >> 3
            words = philox([group & low, (group >> 32) + (site << 16), offset & low, offset >> 32],
                           [seed & low, seed >> 32])
        w = words[(i & 7) >> 1]
        out[j] = w >> 16 if i & 1 else w & 0xFFFF
    return out


def drop_factor(shape, p, seed, offset=0, site=0):
    """What each element is multiplied by: 0 or 1 / (1 - p)."""
    cut = int(np.floor(65536 * p + 0.5))
    keep = drop_bits(int(np.prod(shape)), seed, offset, site) >= cut
    return keep.reshape(shape) * (65536.0 / (65536 - cut) if cut < 65536 else 0.0)

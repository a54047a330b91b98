"""fp64 oracle of the operators between an encoder block's TT layers: layer
normalisation with a residual sum, and attention with a sliding window and
first tokens that stay visible.  Plain definitions with explicit masks, one
sequence and head at a time; shares no code with the library."""

from __future__ import annotations

import numpy as np


def norm_forward(x, gamma=None, beta=None, res=None, eps=1e-5):
    """(y, s, stats): stats[:, 0] = mean, stats[:, 1] = 1 / sqrt(var + eps)."""
    s = np.asarray(x, np.float64) + (0.0 if res is None else np.asarray(res, np.float64))
    mean = s.mean(axis=1, keepdims=True)
    rstd = 1.0 / np.sqrt(((s - mean) ** 2).mean(axis=1, keepdims=True) + eps)
    y = (s - mean) * rstd
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, s, np.concatenate([mean, rstd], axis=1)


def norm_backward(s, dy, gamma=None, dsum=None, eps=1e-5):
    """(dx, dgamma, dbeta) for L = <dy, y> + <dsum, s>."""
    s, dy = np.asarray(s, np.float64), np.asarray(dy, np.float64)
    _, _, st = norm_forward(s, eps=eps)
    h = (s - st[:, :1]) * st[:, 1:]
    g = dy if gamma is None else dy * gamma
    dx = st[:, 1:] * (g - g.mean(axis=1, keepdims=True) -
                      h * (g * h).mean(axis=1, keepdims=True))
    if dsum is not None:
        dx = dx + dsum
    return dx, (dy * h).sum(axis=0), dy.sum(axis=0)


def attn_mask(lq, lk, left, right, sinks):
    """(lq, lk) truth values: key j visible to query row t at position t + lk - lq."""
    i = np.arange(lq)[:, None] + (lk - lq)
    j = np.arange(lk)[None, :]
    ok = np.ones((lq, lk), bool)
    if right >= 0:
        ok &= j <= i + right
    if left >= 0:
        ok &= (j >= i - left) | (j < sinks)
    return ok


def _one(q, k, mask, scale):
    """Softmax weights (0 where masked) and row log-sums of one head."""
    z = np.full((q.shape[0], k.shape[0]), -np.inf)
    for t in range(q.shape[0]):
        j = np.nonzero(mask[t])[0]
        z[t, j] = scale * (k[j] @ q[t])
    p = np.zeros_like(z)
    lse = np.full(q.shape[0], -np.inf)
    for t in range(q.shape[0]):
        j = np.nonzero(mask[t])[0]
        if len(j):
            m = z[t, j].max()
            e = np.exp(z[t, j] - m)
            p[t, j] = e / e.sum()
            lse[t] = m + np.log(e.sum())
    return p, lse


def _product(w, v):
    """sum_j w[t, j] v[j] over the j with a weight: a masked row of v is not touched."""
    out = np.zeros((w.shape[0], v.shape[1]))
    for t in range(w.shape[0]):
        j = np.nonzero(w[t])[0]
        out[t] = w[t, j] @ v[j]
    return out


def attn_forward(q, k, v, seqs, left=-1, right=-1, sinks=0, scale=None):
    """q (Tq, H, D), k and v (Tk, KV, D), seqs: (q0, q1, k0, k1) of each
    sequence.  (o, lse (H, Tq)); rows of no sequence are NaN."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    H, KV, D = q.shape[1], k.shape[1], q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    o, lse = np.full(q.shape, np.nan), np.full((H, q.shape[0]), np.nan)
    for q0, q1, k0, k1 in seqs:
        mask = attn_mask(q1 - q0, k1 - k0, left, right, sinks)
        for h in range(H):
            g = h // (H // KV)
            p, ls = _one(q[q0:q1, h], k[k0:k1, g], mask, scale)
            o[q0:q1, h] = _product(p, v[k0:k1, g])
            lse[h, q0:q1] = ls
    return o, lse


def attn_backward(q, k, v, do, seqs, left=-1, right=-1, sinks=0, scale=None):
    """(dq, dk, dv) for L = <do, o>; rows of no sequence are NaN."""
    q, k, v, do = (np.asarray(a, np.float64) for a in (q, k, v, do))
    H, KV, D = q.shape[1], k.shape[1], q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    dq = np.full(q.shape, np.nan)
    dk, dv = np.full(k.shape, np.nan), np.full(v.shape, np.nan)
    for q0, q1, k0, k1 in seqs:
        mask = attn_mask(q1 - q0, k1 - k0, left, right, sinks)
        dk[k0:k1] = 0.0
        dv[k0:k1] = 0.0
        for h in range(H):
            g = h // (H // KV)
            qs, ks, vs, ds_o = q[q0:q1, h], k[k0:k1, g], v[k0:k1, g], do[q0:q1, h]
            p, _ = _one(qs, ks, mask, scale)
            dp = np.where(mask, ds_o @ np.where(mask.any(0)[:, None], vs, 0.0).T, 0.0)
            ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
            dq[q0:q1, h] = scale * _product(ds, ks)
            dk[k0:k1, g] += scale * ds.T @ qs
            dv[k0:k1, g] += p.T @ ds_o
    return dq, dk, dv

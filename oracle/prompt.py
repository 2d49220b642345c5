"""Oracle of causal attention over packed prompts and of its gradient, in 64 bits, from the
definitions in include/spec_prompt.h."""
from __future__ import annotations

import numpy as np


def sequences(cu, N):
    """(first, end) of each sequence, cut to the rows that are there."""
    for a, e in zip(cu[:-1], cu[1:]):
        a, e = min(max(int(a), 0), N), min(max(int(e), 0), N)
        if a < e:
            yield a, e


def seen(t, window=0):
    i = np.arange(t)
    see = i[:, None] >= i[None, :]
    return see & (i[:, None] - i[None, :] < window) if window else see


def attend(q, k, v, cu, scale, window=0):
    """(out, lse) in float64 of q [N, Hq, D], k and v [N, Hkv, D]."""
    N, H, D = q.shape
    G = H // k.shape[1]
    out, lse = np.zeros((N, H, D)), np.full((N, H), -np.inf)
    for a, e in sequences(cu, N):
        see = seen(e - a, window)
        for h in range(H):
            z = np.where(see, q[a:e, h] @ k[a:e, h // G].T * scale, -np.inf)
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            total = p.sum(1, keepdims=True)
            lse[a:e, h] = (m + np.log(total))[:, 0]
            out[a:e, h] = (p / total) @ v[a:e, h // G]
    return out, lse


def gradient(go, q, k, v, out, lse, cu, scale, window=0):
    """(grad_q, grad_k, grad_v) in float64, from the given out and lse."""
    N, H, D = q.shape
    G = H // k.shape[1]
    gq, gk, gv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for a, e in sequences(cu, N):
        see = seen(e - a, window)
        for h in range(H):
            y = h // G
            z = np.where(see, q[a:e, h] @ k[a:e, y].T * scale, -np.inf)
            p = np.exp(z - lse[a:e, h, None])
            delta = (go[a:e, h] * out[a:e, h]).sum(1, keepdims=True)
            ds = p * (go[a:e, h] @ v[a:e, y].T - delta) * scale
            gq[a:e, h] = ds @ k[a:e, y]
            gk[a:e, y] += ds.T @ q[a:e, h]
            gv[a:e, y] += p.T @ go[a:e, h]
    return gq, gk, gv

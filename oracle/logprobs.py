"""Float64 oracle of token log-probabilities and their gradient (one row at a time,
from the definitions in include/spec_logprobs.h)."""
from __future__ import annotations

import numpy as np


def row(x, token, temperature=1.0, top_n=0):
    """(logprob, rank, entropy, lse, ids, logprobs of ids) of one row of float64 logits;
    None for a data error. A negative token skips the row."""
    x = np.asarray(x, dtype=np.float64)
    V = x.size
    if token < 0:
        return 0.0, -1, 0.0, 0.0, [-1] * top_n, [0.0] * top_n
    t = 1.0 if temperature == 0 else float(temperature)
    if token >= V or not t > 0 or np.isinf(t) or np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
        return None
    z = x / t
    m = z.max()
    lsum = np.log(np.exp(z - m).sum())     # relative to the maximum: logits may be as large as 1e38
    lse, lp = m + lsum, (z - m) - lsum
    p = np.exp(lp)
    live = p > 0
    H = -float((p[live] * lp[live]).sum())
    rank = int((x > x[token]).sum() + (x[:token] == x[token]).sum())
    order = np.lexsort((np.arange(V), -x))[:top_n]
    order = [int(j) for j in order if x[j] > -np.inf]
    pad = top_n - len(order)
    return (float(lp[token]), rank, H, float(lse), order + [-1] * pad,
            [float(lp[j]) for j in order] + [-np.inf] * pad)


def row_gradient(x, token, temperature, lse, entropy, g_lp, g_h, ids=(), g_top=()):
    """d loss / d x of one row, from the forward's lse and entropy as they are given."""
    x = np.asarray(x, dtype=np.float64)
    if token < 0:
        return np.zeros_like(x)
    t = 1.0 if temperature == 0 else float(temperature)
    lp = x / t - lse
    p = np.exp(lp)
    up = np.zeros_like(x)
    up[token] += g_lp
    for j, g in zip(ids, g_top):
        if 0 <= j < x.size:
            up[j] += g
    plogp = np.zeros_like(x)
    live = p > 0
    plogp[live] = p[live] * (lp[live] + entropy)
    return (up - p * up.sum() - g_h * plogp) / t

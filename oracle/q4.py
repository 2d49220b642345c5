"""Oracle of the LM head in 4 bits, in 64 bits, from the definition in include/spec_lm_head.h."""
from __future__ import annotations

import numpy as np


def weight(codes, scale, bias):
    """The weight [V, d] of codes [V, d / 2] uint8, scale and bias [V, d / group]."""
    V, half = codes.shape
    q = np.empty((V, 2 * half))
    q[:, 0::2], q[:, 1::2] = codes % 16, codes // 16
    group = 2 * half // scale.shape[1]
    return q * np.repeat(scale.astype(np.float64), group, 1) + np.repeat(bias.astype(np.float64), group, 1)


def logits(hidden, codes, scale, bias):
    return hidden.astype(np.float64) @ weight(codes, scale, bias).T


def error_bound(hidden, codes, scale, bias):
    """How far fp32 sums may be off, in any order and truncated (u = 2^-23): a group's exact products
    (code - 8) hidden and hidden are summed (group steps), scaled (two roundings, one of bias + 8 scale)
    and added to the other groups (d / group steps)."""
    h = np.abs(hidden.astype(np.float64))
    V, half = codes.shape
    per = scale.shape[1]
    group = 2 * half // per
    q = np.empty((V, 2 * half))
    q[:, 0::2], q[:, 1::2] = codes % 16, codes // 16
    s, b = np.abs(scale.astype(np.float64)), np.abs(bias.astype(np.float64))
    size = np.repeat(s, group, 1) * np.abs(q - 8) + np.repeat(b + 8 * s, group, 1)
    return 2.0 ** -23 * (group + per + 4) * (h @ size.T)

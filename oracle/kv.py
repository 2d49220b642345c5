"""Oracle of the paged e4m3 key/value cache: the append (bit for bit, in fp32 steps) and the
attention of a window over it (in 64 bits), from the definitions in include/spec_kv.h."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -60, 119


def decode_table():
    """The 256 values of e4m3 (codes 0x7F and 0xFF are NaN)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (e == 15 and m == 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if c & 128 else v
    return out


TABLE = decode_table()
_POS = TABLE[:127]                       # ascending finite magnitudes


def encode(x):
    """Codes of float32 values: nearest, ties to the even code, beyond 448 to 448, NaN to NaN."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    a = np.minimum(np.abs(x), E4M3_MAX)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code) | np.where(np.signbit(x) & ~np.isnan(x), 128, 0)
    return code.astype(np.uint8)


def scale_of(x):
    """Smallest power of two s with max finite |x| <= 448 s, in range."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    a = a[np.isfinite(a)]
    top = a.max() if a.size else 0.0
    e = MIN_EXP
    while e < MAX_EXP and top > E4M3_MAX * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def rotate(x, cos, sin, interleaved):
    """Rotates [..., dim] by one position's float32 tables [rot / 2], each step rounded to float32."""
    x = np.asarray(x, dtype=np.float32).copy()
    h = cos.shape[-1]
    i = np.arange(0, 2 * h, 2) if interleaved else np.arange(h)
    j = i + (1 if interleaved else h)
    a, b = x[..., i], x[..., j]
    with np.errstate(invalid="ignore", over="ignore"):
        x[..., i], x[..., j] = a * cos - b * sin, b * cos + a * sin
    return x


def append(k, v, cache, seq_len, cu, table, page, tables=None, interleaved=False):
    """Appends in place: cache = [k codes, k scales, v codes, v scales] (numpy, uint8 and
    float32); k, v float32 [N, H, D]. Returns whether a token could not be stored."""
    kc, ks, vc, vs = cache
    dropped = False
    for b in range(len(seq_len)):
        n, L = cu[b + 1] - cu[b], int(seq_len[b])
        if L < 0:
            continue
        for j in range(L // page, (L + n - 1) // page + 1) if n else ():
            lo, hi = max(L, j * page), min(L + n, (j + 1) * page)
            pg = int(table[b][j]) if j < table.shape[1] else -1
            end = hi if tables is None else min(hi, tables[0].shape[0])
            if not 0 <= pg < kc.shape[0] or end < hi:
                dropped = True
            if not 0 <= pg < kc.shape[0] or end <= lo:
                continue
            keep = lo - j * page
            for h in range(kc.shape[1]):
                for is_v, (x, codes, scales) in enumerate(((k, kc, ks), (v, vc, vs))):
                    y = np.stack([x[cu[b] + p - L, h] if is_v or tables is None else
                                  rotate(x[cu[b] + p - L, h], tables[0][p], tables[1][p], interleaved)
                                  for p in range(lo, end)])
                    s = scale_of(y)
                    if keep:
                        old = scales[pg, h]
                        s = max(s, old)
                        if s > old:
                            codes[pg, h, :keep] = encode((TABLE[codes[pg, h, :keep]] * np.float64(old / s)).astype(np.float32))
                    codes[pg, h, keep:keep + end - lo] = encode(y / s)
                    scales[pg, h] = s
    return dropped


def attend(q, cache, seq_len, cu, table, page, scale, window=0):
    """(out, lse) in float64 of q [N, Hq, D]; keys of unmapped pages are not seen."""
    kc, ks, vc, vs = cache
    N, Hq, D = q.shape
    Hkv = kc.shape[1]
    out, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    for b in range(len(seq_len)):
        L, n = int(seq_len[b]), cu[b + 1] - cu[b]
        if L < 0 or n == 0:
            continue
        pos = np.arange(L + n)
        pg = np.array([int(table[b][p // page]) if p // page < table.shape[1] else -1 for p in pos])
        mapped = (pg >= 0) & (pg < kc.shape[0])
        for h in range(Hkv):
            at = pos[mapped], pg[mapped]
            key = TABLE[kc[at[1], h, at[0] % page]] * ks[at[1], h].astype(np.float64)[:, None]
            val = TABLE[vc[at[1], h, at[0] % page]] * vs[at[1], h].astype(np.float64)[:, None]
            for i in range(n):
                see = at[0] <= L + i
                if window:
                    see &= at[0] > L + i - window
                if not see.any():
                    continue
                for g in range(Hq // Hkv):
                    qh = h * (Hq // Hkv) + g
                    a = (key[see] @ q[cu[b] + i, qh].astype(np.float64)) * scale
                    m = a.max()
                    p = np.exp(a - m)
                    out[cu[b] + i, qh] = p @ val[see] / p.sum()
                    lse[cu[b] + i, qh] = m + np.log(p.sum())
    return out, lse

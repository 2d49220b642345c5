"""GPU: attention of a window over the paged e4m3 cache against the float64 oracle.

Tolerances, from the kernel's arithmetic (u = 2^-24): with A the largest scale * sum |q_d k_d|
of the visible keys and E the largest |log2| of their value scales, a logit is off by at most
(head_dim + 8) u A (sum of exact products), its exponent by 8 u (1.45 A + E + 8) more and the
exponential by 2^-21: d together. Weights w = p (value scale) are rounded to fp16 for the value
product: by 2^-11 of themselves, or by half the subnormal spacing 2^-25 in a frame in which the
largest weight is at least 2^7. So, with c the codes' values,
  |out - ref| <= (2^-11 + 2 d) sum p |v| + 2^-32 max(w) sum |c| + half an ulp of bf16 |ref|,
  |lse - ref| <= d + (keys / 8 + 80) u + 4 u |lse|."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from oracle import kv as okv
from tests.test_gpu_kv import _i32, make, to_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def compare(out, lse, q, cache, sl, cu, table, page, scale, window, seqs=None, nan_ok=False):
    N, H, D = q.shape
    out, lse, q = out.cpu().double().numpy(), lse.cpu().double().numpy(), q.cpu().double().numpy()
    kc, ks, vc, vs = cache
    kh = kc.shape[1]
    for b in range(len(sl)) if seqs is None else seqs:
        L, n = int(sl[b]), int(cu[b + 1] - cu[b])
        pos = np.arange(max(L, 0) + n if L >= 0 else 0)
        pg = np.array([int(table[b][p // page]) if p // page < table.shape[1] else -1 for p in pos], dtype=int)
        ok = (pg >= 0) & (pg < kc.shape[0])
        pos, pg = pos[ok], pg[ok]
        for h in range(kh):
            key = okv.TABLE[kc[pg, h, pos % page]] * ks[pg, h].astype(np.float64)[:, None]
            val = okv.TABLE[vc[pg, h, pos % page]] * vs[pg, h].astype(np.float64)[:, None]
            for i in range(n):
                see = pos <= L + i
                if window:
                    see &= pos > L + i - window
                for g in range(H // kh):
                    r, qh = int(cu[b]) + i, h * (H // kh) + g
                    if not see.any():
                        assert (out[r, qh] == 0).all() and lse[r, qh] == -np.inf, (b, i, qh)
                        continue
                    a = key[see] @ q[r, qh] * scale
                    m = a.max()
                    p = np.exp(a - m)
                    ref_lse, p = m + np.log(p.sum()), p / p.sum()
                    ref = p @ val[see]
                    if np.isnan(ref).any():
                        assert nan_ok
                        assert (np.isnan(out[r, qh]) == np.isnan(ref)).all(), (b, i, qh)
                        continue
                    A = (np.abs(key[see]) @ np.abs(q[r, qh])).max() * abs(scale)
                    sc = vs[pg, h].astype(np.float64)[see]
                    d = (D + 8) * U * A + 8 * U * (1.45 * A + np.abs(np.log2(sc)).max() + 8) + 2.0 ** -21
                    tol = ((2.0 ** -11 + 2 * d) * (p @ np.abs(val[see])) + 2.0 ** -8 * np.abs(ref) + 1e-30
                           + 2.0 ** -32 * (p * sc).max() * np.abs(val[see] / sc[:, None]).sum(0))
                    err = np.abs(out[r, qh] - ref)
                    k = (err / tol).argmax()
                    assert (err <= tol).all(), (b, i, qh, k, err[k], tol[k], ref[k])
                    assert abs(lse[r, qh] - ref_lse) <= d + (see.sum() / 8 + 80) * U + 4 * U * abs(ref_lse), (b, i, qh)


def check(lens, new, heads=4, kv_heads=2, dim=64, page=16, window=0, seed=0, scale=None, gain=1.0, edit=None, q_edit=None,
          garbage=True, seqs=None, nan_ok=False, spread=1.0, max_tokens=None):
    g, cache, sl, cu, table = make(lens, new, heads, kv_heads, dim, page, seed, spread=spread)
    if garbage:                    # what lies past the end: NaN codes and odd scales in pages not in use
        for b, (L, n) in enumerate(zip(lens, new)):
            end = max(L, 0) + n
            if end % page:
                cache[0][table[b][end // page], :, end % page:] = 0x7F
                cache[2][table[b][end // page], :, end % page:] = 0xFF
        used = set(table[table >= 0].tolist())
        for pg in range(cache[0].shape[0]):
            if pg not in used:
                cache[0][pg], cache[2][pg], cache[1][pg], cache[3][pg] = 0x7F, 0x7F, np.nan, np.nan
    if edit:
        edit(cache, table)
    N = int(cu[-1])
    wide = torch.randn(N, heads + 3, dim, generator=g) * gain
    q = wide.to(torch.bfloat16)[:, :heads]
    if q_edit:
        q_edit(q)
    qd = q.to(DEV) if heads % 2 else wide.to(torch.bfloat16).to(DEV)[:, :heads]
    if q_edit:
        qd = q.to(DEV)
    scale = dim ** -0.5 if scale is None else scale
    kvc = to_cache(cache)
    win = (_i32(sl.tolist()), _i32(cu.tolist()), _i32(table.tolist()), max_tokens or max(new))
    out, lse = sv.spec_kv_attention(qd, kvc, *win, scale=scale, window=window)
    again, lse2 = sv.spec_kv_attention(qd, kvc, *win, scale=scale, window=window)
    torch.cuda.synchronize()
    if not nan_ok:
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    compare(out, lse, q, cache, sl, cu, table, page, scale, window, seqs, nan_ok)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,new", [(1, 1, 1), (8, 8, 2), (6, 2, 5), (14, 2, 3), (16, 1, 2), (32, 4, 4)])
def test_windows(heads, kv_heads, new, dim, page):
    check([0, 1, 31, 32, 33, 130, 517], [new] * 7, heads, kv_heads, dim, page, seed=dim + page + heads)


@pytest.mark.parametrize("dim", [64, 128])
def test_ragged_lengths_and_empty_places(dim):
    check([0, 700, 40, -1, 5, 0, 63], [1, 0, 37, 3, 70, 0, 6], 8, 2, dim, 32, seed=dim)
    check([3, 3], [0, 1], 8, 8, dim, 16, seed=dim + 1)


@pytest.mark.parametrize("window", [1, 7, 32, 100])
def test_sliding_windows(window):
    check([0, 10, 250, 64, 1000], [5, 1, 40, 6, 3], 4, 2, 64, 16, window=window, seed=window)
    check([300], [2], 8, 1, 128, 64, window=window, seed=window)


def test_long_contexts_split_over_warps():
    check([9000, 100, 5000], [3, 2, 1], 8, 2, 128, 64, seed=1)
    check([20000], [1], 2, 1, 64, 16, seed=2)
    check([50] * 300, [2] * 300, 2, 1, 64, 16, seed=3, seqs=range(0, 300, 29))


def test_long_windows_of_new_tokens():
    check([100, 0], [150, 33], 8, 2, 64, 32, seed=4)
    check([65], [70], 6, 1, 128, 128, seed=5)


@pytest.mark.parametrize("gain,spread", [(1e-20, 1.0), (60.0, 1.0), (1.0, 2.0 ** 40), (1.0, 2.0 ** -40), (1e20, 2.0 ** -60)])
def test_magnitudes(gain, spread):
    # the logits stay of order 1 to 1000 through `scale`
    check([40, 300], [3, 2], 4, 2, 64, 32, seed=7, gain=gain, spread=spread,
          scale=0.125 if gain in (1e-20, 60.0) else 0.125 / (gain * spread))


def test_scales_that_differ_from_page_to_page():
    def edit(c, t):
        r = np.random.default_rng(1)
        for k in (1, 3):
            c[k][:] = np.exp(r.normal(size=c[k].shape) * (2 if k == 1 else 8) - 4).astype(np.float32)   # not powers of two
    check([700, 90], [4, 4], 8, 2, 128, 16, seed=8, edit=edit, garbage=False)


def test_unmapped_pages_are_not_seen():
    def edit(c, t):
        t[0, 2:5] = -1
        t[1, :] = -1
        t[2, 0] = 1 << 20
        t[3, 6] = -7
    check([200, 60, 5, 97], [3, 2, 4, 4], 4, 2, 64, 16, seed=9, edit=edit)


def test_nan_stays_where_it_is_seen():
    inf, nan = float("inf"), float("nan")

    def edit(c, t):                # tokens 52 and 54 of sequence 0 are new: query i sees up to 50 + i
        c[2][t[0][52 // 16], 0, 52 % 16, 9] = 0x7F
        c[2][t[0][54 // 16], 1, 54 % 16, 40] = 0xFF
        c[0][t[0][53 // 16], 1, 53 % 16, 3] = 0x7F
    for dim in (64, 128):
        check([50, 20], [6, 2], 8, 2, dim, 16, seed=10, edit=edit, nan_ok=True)

    def q_edit(q):
        q[0, 1, 5] = nan
    check([50, 20], [6, 2], 8, 2, 64, 16, seed=11, q_edit=q_edit, nan_ok=True)


def test_extreme_logits():
    check([400], [2], 2, 2, 64, 16, seed=12, scale=30.0)          # one key takes all
    check([400], [2], 2, 2, 64, 16, seed=13, scale=0.0)           # all keys alike
    check([400], [2], 2, 2, 64, 16, seed=14, scale=-0.125)


def test_offsets_past_32_bits():
    # 70,000 pages of 8 heads x 64 tokens x 128 bytes: the last pages lie past 4 GB
    page, kh, D, pool = 64, 8, 128, 70_000
    k = torch.zeros(pool, kh, page, D, dtype=torch.uint8, device=DEV)
    v = torch.zeros(pool, kh, page, D, dtype=torch.uint8, device=DEV)
    one = torch.ones(pool, kh, device=DEV)
    g = torch.Generator().manual_seed(5)
    table = np.array([[pool - 1, 3, pool - 2]], np.int32)
    small = [np.zeros((3, kh, page, D), np.uint8), np.ones((3, kh), np.float32) / 64, np.zeros((3, kh, page, D), np.uint8),
             np.ones((3, kh), np.float32) / 64]
    for x in (small[0], small[2]):
        x[:] = torch.randint(0, 120, x.shape, generator=g, dtype=torch.uint8).numpy()
    for j, p in enumerate(table[0]):
        k[p], v[p] = torch.from_numpy(small[0][j]).to(DEV), torch.from_numpy(small[2][j]).to(DEV)
    q = torch.randn(2, 16, D, generator=g).to(torch.bfloat16)
    kvc = sv.KVCache(k, one / 64, v, one / 64)
    out, lse = sv.spec_kv_attention(q.to(DEV), kvc, _i32([150]), _i32([0, 2]), _i32(table.tolist()), 2)
    compare(out, lse, q, small, [150], [0, 2], np.array([[0, 1, 2]]), page, D ** -0.5, 0)
    new = torch.randn(2, kh, D, generator=g).to(DEV)
    sv.spec_kv_append(new, new, kvc, _i32([150]), _i32([0, 2]), _i32(table.tolist()), 2)
    okv.append(new.cpu().numpy(), new.cpu().numpy(), small, [150], [0, 2], np.array([[0, 1, 2]]), page)
    assert np.array_equal(k[pool - 2].cpu().numpy(), small[0][2]) and np.array_equal(v[pool - 2].cpu().numpy(), small[2][2])


def test_workspace_stream_and_graph():
    g, cache, sl, cu, table = make([300, 64], [3, 2], 8, 2, 64, 16, 3)
    q = torch.randn(5, 8, 64, generator=g).to(torch.bfloat16).to(DEV)
    kvc, win = to_cache(cache), (_i32(sl.tolist()), _i32(cu.tolist()), _i32(table.tolist()), 3)
    ref = sv.spec_kv_attention(q, kvc, *win)
    ws = torch.full((sv.spec_kv_attention_workspace_bytes(2, 3, 8, 2, 64),), 0xFF, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.spec_kv_attention(q, kvc, *win, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    out, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_kv_attention(q, kvc, *win, out=out, lse=lse, workspace=ws)
    win[0][0] = 200
    graph.replay()
    torch.cuda.synchronize()
    fresh = sv.spec_kv_attention(q, kvc, *win)
    assert torch.equal(out, fresh[0]) and torch.equal(lse, fresh[1]) and not torch.equal(out, ref[0])


def test_append_then_attend():
    # one window through both operators against the oracle's append and attention
    g, cache, sl, cu, table = make([45, 10], [4, 4], 8, 2, 64, 16, 21)
    x = torch.randn(8, 12, 64, generator=g).to(torch.bfloat16)
    q, k, v = x.to(DEV).split([8, 2, 2], 1)
    cos, sin = sv.rope_tables(128, 64, device=DEV)
    kvc, win = to_cache(cache), (_i32(sl.tolist()), _i32(cu.tolist()), _i32(table.tolist()), 4)
    qr = sv.spec_kv_append(k, v, kvc, *win, q=q, cos=cos, sin=sin)
    out, lse = sv.spec_kv_attention(qr, kvc, *win)
    f = x.float().numpy()
    okv.append(f[:, 8:10], f[:, 10:], cache, sl, cu, table, 16, (cos.cpu().numpy(), sin.cpu().numpy()))
    compare(out, lse, qr, cache, sl, cu, table, 16, 0.125, 0)


def test_attention_refusals():
    cache = sv.KVCache.empty(8, 16, 2, 64, device=DEV)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device=DEV)
    win = (_i32([0]), _i32([0, 4]), _i32([[0, 1]]), 4)
    for bad in (lambda: sv.spec_kv_attention(q.float(), cache, *win), lambda: sv.spec_kv_attention(q[:, :3], cache, *win),
                lambda: sv.spec_kv_attention(q[..., :32], cache, *win), lambda: sv.spec_kv_attention(q, cache, *win, window=-1),
                lambda: sv.spec_kv_attention(q, cache, *win[:3], 9), lambda: sv.spec_kv_attention(q, cache, *win, scale=float("inf")),
                lambda: sv.spec_kv_attention(q, cache, *win, workspace=torch.empty(64, dtype=torch.uint8, device=DEV)),
                lambda: sv.spec_kv_attention(q, cache, *win, out=q.float()), lambda: sv.spec_kv_attention(q, cache, *win, lse=q)):
        with pytest.raises(sv.SpecVerifyError):
            bad()


# --- many query rows (new tokens x query heads of a kv head, head_dim 128): the wide kernel

@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kv_heads,new", [(4, 1, 64), (8, 1, 130), (7, 1, 37), (2, 2, 257), (64, 1, 4)])
def test_many_rows(heads, kv_heads, new, page):
    check([0, 1, 127, 128, 300], [new] * 5, heads, kv_heads, 128, page, seed=heads + page, seqs=(0, 2, 4))


def test_many_rows_ragged_and_empty_places():
    check([0, 1500, -1, 5, 64, 700], [90, 1, 3, 0, 200, 33], 8, 2, 128, 32, seed=30)
    check([12000, 40], [70, 50], 4, 1, 128, 64, seed=31)            # items cut between blocks


@pytest.mark.parametrize("window", [1, 50, 128, 1000])
def test_many_rows_in_sliding_windows(window):
    check([0, 500, 2000], [100, 60, 128], 4, 1, 128, 16, window=window, seed=window)


def test_many_rows_unmapped_pages_and_scales():
    def edit(c, t):
        t[0, 2:5] = -1
        t[1, :] = -1
        t[2, 0] = 1 << 20
        t[2, 9] = -7
        r = np.random.default_rng(1)
        for k in (1, 3):
            c[k][:] = np.exp(r.normal(size=c[k].shape) * (2 if k == 1 else 6) - 4).astype(np.float32)
    check([200, 60, 97], [70, 64, 80], 4, 1, 128, 16, seed=32, edit=edit, garbage=False)


@pytest.mark.parametrize("gain,spread", [(1e-20, 1.0), (60.0, 1.0), (1.0, 2.0 ** 40), (1.0, 2.0 ** -40)])
def test_many_rows_magnitudes(gain, spread):
    check([40, 300], [100, 90], 4, 2, 128, 32, seed=33, gain=gain, spread=spread,
          scale=0.09 if gain != 1.0 else 0.09 / (gain * spread))
    check([400], [100], 2, 1, 128, 16, seed=34, scale=0.0)


def test_many_rows_negative_scale():
    check([400, 20], [100, 70], 4, 2, 128, 16, seed=37, scale=-0.09)


def test_many_rows_nan_stays_where_it_is_seen():
    nan = float("nan")

    def edit(c, t):                # tokens 52, 75 and 100 of sequence 0 are new: query i sees up to 50 + i
        c[2][t[0][52 // 16], 0, 52 % 16, 9] = 0x7F
        c[2][t[0][75 // 16], 1, 75 % 16, 120] = 0xFF
        c[0][t[0][100 // 16], 1, 100 % 16, 3] = 0x7F
        c[2][t[1][3 // 16], 0, 3, 77] = 0x7F          # seen by every query of sequence 1

    def q_edit(q):
        q[70, 1, 5] = nan
    check([50, 200], [60, 50], 8, 2, 128, 16, seed=35, edit=edit, q_edit=q_edit, nan_ok=True)


@pytest.mark.parametrize("window", [0, 40])
def test_many_rows_many_nan(window):
    def edit(c, t):                # a NaN in every element of four in five of the new tokens, some in all
        for p in range(50, 110):
            for h in range(2):
                if p % 5:
                    c[2][t[0][p // 16], h, p % 16, (p * 7 + h) % 128] = 0x7F
                if p == 100 + h:
                    c[2][t[0][p // 16], h, p % 16] = 0xFF
        for p in range(240, 250):
            c[2][t[1][p // 16], 1, p % 16, ::p % 4 + 2] = 0x7F
    check([50, 200], [60, 50], 8, 2, 128, 16, seed=36, edit=edit, window=window, nan_ok=True)


def test_many_rows_repeat_and_streams():
    g, cache, sl, cu, table = make([1000, 300], [128, 65], 4, 1, 128, 64, 36)
    q = torch.randn(193, 4, 128, generator=g).to(torch.bfloat16).to(DEV)
    kvc, win = to_cache(cache), (_i32(sl.tolist()), _i32(cu.tolist()), _i32(table.tolist()), 128)
    ref = sv.spec_kv_attention(q, kvc, *win)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = sv.spec_kv_attention(q, kvc, *win, stream=side)
        side.synchronize()
        assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])

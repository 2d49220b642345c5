"""GPU: the paged e4m3 cache: appended codes and scales bit for bit against the oracle,
queries within one rounding of the type."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from oracle import kv as okv

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(lens, new, heads, kv_heads, dim, page, seed, extra=2, spread=1.0):
    """A cache with random codes and power-of-two scales, and the window's tables."""
    g = torch.Generator().manual_seed(seed)
    need = [max(-(-(max(c, 0) + t) // page), 1) for c, t in zip(lens, new)]
    pool = sum(need) + extra
    order = torch.randperm(pool, generator=g).tolist()
    table = np.full((len(lens), max(need) + 1), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    cache = []
    for _ in range(2):
        codes = torch.randint(0, 256, (pool, kv_heads, page, dim), generator=g, dtype=torch.uint8).numpy()
        codes[(codes & 127) == 127] ^= 1              # no NaN among the values in use
        cache += [codes, (2.0 ** torch.randint(-9, -3, (pool, kv_heads), generator=g)).float().numpy() * np.float32(spread)]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return g, cache, np.array(lens, np.int32), cu, table


def to_cache(c):
    t = [torch.from_numpy(x.copy()).to(DEV) for x in c]
    return sv.KVCache(t[0].view(torch.float8_e4m3fn), t[1], t[2].view(torch.float8_e4m3fn), t[3])


def check_append(lens, new, heads=4, kv_heads=2, dim=64, page=16, dtype="bf16", rot=32, interleaved=False, seed=0, packed=True,
                 gain=1.0, poison=None, max_pos=None, calls=1, table_edit=None, max_tokens=None):
    g, cache, sl, cu, table = make(lens, new, heads, kv_heads, dim, page, seed)
    if table_edit:
        table_edit(table)
    N = max(int(cu[-1]), 1)
    wide = heads + 2 * kv_heads
    qkv = (torch.randn(N, wide, dim, generator=g) * gain).to(TYPES[dtype])
    if poison is not None:
        for at, val in poison:
            qkv[at] = val
    q, k, v = qkv.to(DEV).split([heads, kv_heads, kv_heads], 1)
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    mp = max_pos or table.shape[1] * page
    tabs = sv.rope_tables(mp, rot, device=DEV) if rot else (None, None)
    kvc, flag = to_cache(cache), torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(calls):
        qo = sv.spec_kv_append(k, v, kvc, _i32(sl.tolist()), _i32(cu.tolist()), _i32(table.tolist()),
                               max_tokens or max(max(new), 1), q=q, cos=tabs[0], sin=tabs[1], interleaved=interleaved, flag=flag)
    torch.cuda.synchronize()
    np_tabs = None if not rot else [t.cpu().numpy() for t in tabs]
    host = qkv.float().numpy()
    dropped = okv.append(host[:, heads:heads + kv_heads], host[:, heads + kv_heads:], cache, sl, cu, table, page, np_tabs, interleaved)
    assert int(flag.item()) == int(dropped)
    for name, got, ref in zip(("k codes", "k scale", "v codes", "v scale"), kvc, cache):
        got = got.view(torch.uint8).cpu().numpy() if got.dtype != torch.float32 else got.cpu().numpy()
        if ref.dtype == np.uint8:                      # NaN codes of either sign are NaN
            nan = ((got & 127) == 127) & ((ref & 127) == 127)
            assert ((got == ref) | nan).all(), (name, int((got != ref).sum()))
        else:
            assert np.array_equal(got, ref), name
    for b in range(len(lens)):
        for i in range(int(cu[b + 1] - cu[b])):
            r, p = int(cu[b]) + i, int(sl[b]) + i
            if sl[b] < 0:
                assert (qo[r] == 0).all()
                continue
            if rot and p >= mp:
                assert torch.isnan(qo[r]).all()
                continue
            ref = host[r, :heads] if not rot else okv.rotate(host[r, :heads], np_tabs[0][p], np_tabs[1][p], interleaved)
            ref = torch.from_numpy(ref).to(TYPES[dtype])
            assert torch.equal(torch.nan_to_num(qo[r].cpu(), 7.0), torch.nan_to_num(ref, 7.0))
    return kvc


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
def test_windows(page, dim, dtype):
    check_append([0, 1, page - 1, page, 3 * page + 5, 2 * page - 2], [5] * 6, dim=dim, page=page, dtype=dtype, rot=dim, seed=page + dim)


@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, False), (48, True), (64, False), (128, True)])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 3), (16, 2), (8, 8)])
def test_rotations_and_heads(heads, kv_heads, rot, interleaved):
    check_append([7, 30], [3, 1], heads=heads, kv_heads=kv_heads, dim=128, page=32, rot=rot, interleaved=interleaved, seed=rot + heads)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ragged_lengths_from_none_to_long(dtype):
    check_append([0, 5, 200, -1, 33, 64], [300, 0, 1, 4, 31, 129], page=64, dtype=dtype, rot=32, seed=5, packed=False)
    check_append([3], [0], page=16, seed=6)


@pytest.mark.parametrize("gain", [1e-30, 1e-4, 300.0, 1e30])
def test_scales_that_grow_stay_or_start_again(gain):
    check_append([10, 16, 31, 3], [9, 9, 2, 1], page=16, dtype="fp32", gain=gain, seed=3, rot=64)


def test_appending_again_changes_nothing():
    check_append([10, 16, 31, 3], [9, 9, 2, 1], page=16, gain=40.0, seed=4, calls=3)


def test_infinities_and_nan():
    inf, nan = float("inf"), float("nan")
    # wide is 4 query heads, 2 key heads, 2 value heads
    check_append([10, 40], [4, 3], dtype="fp32", rot=0, seed=2,
                 poison=[((0, 4, 3), inf), ((1, 5, 0), -inf), ((2, 6, 9), nan), ((5, 7), inf), ((6, 7, 2), nan)])


def test_unmapped_pages_and_positions_past_the_tables_are_reported():
    def edit(t):
        t[0, 1] = -1
        t[1, 0] = 10_000
    check_append([10, 3, 0], [30, 2, 2], page=16, seed=1, table_edit=edit)
    check_append([10, 3], [30, 2], page=16, seed=1, max_pos=25)
    check_append([100, 3], [3, 2], page=16, seed=1, max_pos=64)


def test_a_sequence_past_max_tokens_is_reported():
    g, cache, sl, cu, table = make([0, 0], [6, 2], 2, 1, 64, 16, 1)
    k = torch.randn(8, 1, 64, generator=g).to(DEV)
    kvc, flag = to_cache(cache), torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.spec_kv_append(k, k, kvc, _i32([0, 0]), _i32([0, 6, 8]), _i32(table.tolist()), 4, flag=flag)
    assert int(flag.item()) == 1
    ref = [c.copy() for c in cache]
    kk = k.cpu().numpy()
    okv.append(kk[[0, 1, 2, 3, 6, 7]], kk[[0, 1, 2, 3, 6, 7]], ref, sl, np.array([0, 4, 6]), table, 16)
    assert np.array_equal(kvc.k_codes.view(torch.uint8).cpu().numpy(), ref[0])


def test_queries_in_place_and_another_stream():
    g, cache, sl, cu, table = make([5, 20], [3, 3], 4, 2, 64, 16, 9)
    q, k = torch.randn(6, 4, 64, generator=g).to(DEV), torch.randn(6, 2, 64, generator=g).to(DEV)
    cos, sin = sv.rope_tables(100, 64, device=DEV)
    win = (_i32(sl.tolist()), _i32(cu.tolist()), _i32(table.tolist()), 3)
    a, b = to_cache(cache), to_cache(cache)
    ref = sv.spec_kv_append(k, k, a, *win, q=q, cos=cos, sin=sin)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q2 = q.clone()
    side.wait_stream(torch.cuda.current_stream())
    assert sv.spec_kv_append(k, k, b, *win, q=q2, cos=cos, sin=sin, q_out=q2, stream=side) is q2
    side.synchronize()
    assert torch.equal(ref, q2)
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8) if x.dtype != torch.float32 else x, y.view(torch.uint8) if y.dtype != torch.float32 else y)


def test_append_refusals():
    cache = sv.KVCache.empty(8, 16, 2, 64, device=DEV)
    k = torch.zeros(4, 2, 64, device=DEV)
    win = (_i32([0]), _i32([0, 4]), _i32([[0, 1]]), 4)
    for bad in (lambda: sv.spec_kv_append(k.half(), k.half(), cache, *win), lambda: sv.spec_kv_append(k, k[:, :1], cache, *win),
                lambda: sv.spec_kv_append(k[..., :32], k[..., :32], cache, *win), lambda: sv.spec_kv_append(k, k, cache, *win, q_out=k),
                lambda: sv.spec_kv_append(k, k, cache, *win, cos=torch.zeros(9, 32, device=DEV)),
                lambda: sv.spec_kv_append(k, k, cache, _i32([0, 1]), *win[1:]), lambda: sv.spec_kv_append(k, k, cache, *win[:3], 5),
                lambda: sv.spec_kv_append(k, k, cache._replace(v_scale=cache.v_scale[:1]), *win),
                lambda: sv.spec_kv_append(k.transpose(0, 1).contiguous().transpose(0, 1), k, cache, *win)):
        with pytest.raises(sv.SpecVerifyError):
            bad()

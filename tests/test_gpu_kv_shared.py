"""GPU: attention of a batch on shared prefixes against the float64 oracle over each sequence's own row
of the page table, with the tolerances of test_gpu_kv_attention (the join of two parts adds a few
units of 2^-24, which its bounds leave room for: 80 of them for lse, 2^-21 for the weights)."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from tests.test_gpu_kv import _i32, make, to_cache
from tests.test_gpu_kv_attention import compare

pytestmark = pytest.mark.gpu
DEV = "cuda"


# Two passes are made where the page table has room for this many bytes of keys and values that are read again
TWO_PASSES = 320 << 20


def build(groups, heads, kv_heads, dim, page, seed=0, spread=1.0, two=True):
    """groups: a list of (shared tokens, [(own cached tokens or None for an empty place, new tokens), ...]).
    two: the page table's rows are so long (unmapped at their ends) that the shared tokens are a pass of their own."""
    lens, new, of = [], [], []
    for i, (shared, members) in enumerate(groups):
        for own, t in members:
            lens.append(-1 if own is None else shared + own)
            new.append(t)
            of.append(i)
    g, cache, sl, cu, table = make(lens, new, heads, kv_heads, dim, page, seed, spread=spread)
    cg = np.concatenate([[0], np.cumsum([len(m) for _, m in groups])])
    again = (len(lens) - len(groups)) * kv_heads * 2 * dim * page
    if two and again:
        table = np.pad(table, ((0, 0), (0, max(0, TWO_PASSES // again + 1 - table.shape[1]))), constant_values=-1)
    if not two:
        assert again * table.shape[1] < TWO_PASSES
    shared = np.array([s for s, _ in groups], np.int32)
    for i, (s, _) in enumerate(groups):            # the members' rows name one member's pages for the whole pages shared
        live = [b for b in range(cg[i], cg[i + 1]) if lens[b] >= 0]
        for b in live[1:]:
            table[b, :s // page] = table[live[0], :s // page]
    # what lies past the end: NaN codes, also in pages that no table names
    named = set(table[table >= 0].tolist())
    for pg in range(cache[0].shape[0]):
        if pg not in named:
            cache[0][pg], cache[2][pg], cache[1][pg], cache[3][pg] = 0x7F, 0x7F, np.nan, np.nan
    for b, (L, t) in enumerate(zip(lens, new)):
        end = max(L, 0) + t
        if end % page and L >= 0:
            cache[0][table[b][end // page], :, end % page:] = 0x7F
            cache[2][table[b][end // page], :, end % page:] = 0xFF
    return g, cache, sl, cu, table, cg, shared


def check(groups, heads=8, kv_heads=2, dim=64, page=16, seed=0, told=None, scale=None, spread=1.0, edit=None, seqs=None, max_tokens=None,
          q_edit=None, two=True):
    """told: what the call is told of shared_len, where that differs."""
    g, cache, sl, cu, table, cg, shared = build(groups, heads, kv_heads, dim, page, seed, spread, two)
    if edit:
        edit(cache, table)
    N = int(cu[-1])
    q = torch.randn(N, heads + 1, dim, generator=g).to(torch.bfloat16)[:, :heads]
    if q_edit:
        q_edit(q)
    kvc = to_cache(cache)
    new = np.diff(cu)
    win = (_i32(sl.tolist()), _i32(cu.tolist()), _i32(table.tolist()), max_tokens or int(new.max()))
    sh = _i32((shared if told is None else told).tolist() if not isinstance(told, list) else told)
    args = dict(cu_groups=_i32(cg.tolist()), shared_len=sh, scale=scale)
    out, lse = sv.spec_kv_attention_shared(q.to(DEV), kvc, *win, **args)
    again = sv.spec_kv_attention_shared(q.to(DEV), kvc, *win, **args)
    torch.cuda.synchronize()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    compare(out, lse, q, cache, sl, cu, table, page, dim ** -0.5 if scale is None else scale, 0, seqs)
    return out, lse


@pytest.mark.parametrize("dim,page", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("heads,kv_heads,new", [(2, 2, 1), (8, 2, 3), (14, 2, 2), (32, 4, 5)])
def test_one_prefix(heads, kv_heads, new, dim, page):
    check([(640, [(0, new), (1, new), (50, new), (300, new), (127, new)])], heads, kv_heads, dim, page, seed=dim + page + heads)


def test_little_that_is_shared_is_one_pass():
    g = [(640, [(0, 2), (50, 2), (300, 1)]), (100, [(None, 1), (4, 2)])]
    a, b = (check(g, 4, 2, 64, 16, seed=20, two=two) for two in (False, True))
    assert ((a[1] - b[1]).abs().nan_to_num(0) <= 1e-4).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_many_rows_on_a_prefix(dim):
    check([(1024, [(10 * i, 2) for i in range(40)])], 8, 1, dim, 64, seed=1, seqs=range(0, 40, 7))
    check([(300, [(7 * i, 1) for i in range(70)]), (2000, [(3 * i, 1) for i in range(33)])], 4, 2, dim, 16, seed=2, seqs=range(0, 103, 9))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shared", [0, 1, 63, 64, 127, 128, 129, 255, 384, 1000])
def test_prefix_lengths(shared, dim):
    check([(shared, [(20, 2), (0, 1), (150, 3)])], 4, 2, dim, 16, seed=shared)


@pytest.mark.parametrize("dim", [64, 128])
def test_groups_of_many_kinds(dim):
    check([(0, [(30, 2), (5, 0)]), (512, [(3, 0)]), (256, [(0, 1)]), (700, [(1, 2), (None, 2), (90, 0), (400, 5)]), (128, [(None, 1)]),
           (130, [(None, 3), (2, 1), (0, 4)])], 6, 2, dim, 32, seed=3)


def test_long_windows_and_a_tight_bound():
    check([(512, [(10, 40), (100, 1), (0, 17)])], 4, 1, 128, 64, seed=4)
    check([(512, [(10, 40), (100, 1), (0, 17)])], 4, 1, 64, 64, seed=5)


def test_shared_len_is_cut_to_what_every_sequence_holds():
    # told more than is shared by the shortest: the cut is the shortest's seq_len
    g = [(256, [(0, 2), (300, 1), (40, 2)])]
    ref = check(g, 4, 2, 64, 16, seed=6)
    got = check(g, 4, 2, 64, 16, seed=6, told=[1 << 20])
    # (256 + 0 cached in the first: units below 256 in both calls)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    check(g, 4, 2, 64, 16, seed=6, told=[-5])
    check(g, 4, 2, 64, 16, seed=6, told=[-(1 << 31)])
    check(g, 4, 2, 64, 16, seed=6, told=[(1 << 31) - 1])


@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (32, 2)])
def test_it_is_the_attention_of_each_sequence(heads, kv_heads):
    # as spec_kv_attention on the same tables, within both calls' rounding (2^-11 of weights, bf16 results)
    g, cache, sl, cu, table, cg, shared = build([(2048, [(30 * i, 3) for i in range(12)])], heads, kv_heads, 128, 64, seed=7)
    q = torch.randn(int(cu[-1]), heads, 128, generator=g).to(torch.bfloat16).to(DEV)
    kvc, win = to_cache(cache), (_i32(sl.tolist()), _i32(cu.tolist()), _i32(table.tolist()), 3)
    a = sv.spec_kv_attention(q, kvc, *win)
    b = sv.spec_kv_attention_shared(q, kvc, *win, _i32(cg.tolist()), _i32(shared.tolist()))
    assert ((a[1] - b[1]).abs() <= 1e-4).all()
    size = a[0].float().abs().amax()
    assert ((a[0].float() - b[0].float()).abs() <= 2.0 ** -7 * a[0].float().abs() + 2.0 ** -8 * size).all()


def test_unmapped_pages_and_nan_values():
    def edit(c, t):
        t[:, 3] = -1                   # a page of the prefix
        t[1, 25:] = 1 << 20            # the second's own
    check([(384, [(60, 2), (30, 2), (0, 1)])], 4, 2, 64, 16, seed=8, edit=edit)
    g, cache, sl, cu, table, cg, shared = build([(384, [(60, 2), (30, 2)])], 4, 2, 64, 16, seed=9)
    cache[2][table[0, 2], 1, 5, 7] = 0x7F          # a value of the prefix: every row of kv head 1
    cache[2][table[1, 24], 0, 3, 9] = 0x7F         # one of the second's own: its rows of kv head 0
    q = torch.randn(4, 4, 64, generator=g).to(torch.bfloat16).to(DEV)
    out, _ = sv.spec_kv_attention_shared(q, to_cache(cache), _i32(sl.tolist()), _i32(cu.tolist()), _i32(table.tolist()), 2, _i32(cg.tolist()),
                                         _i32(shared.tolist()))
    nan = torch.isnan(out)
    expect = torch.zeros_like(nan)
    expect[:, 2:, 7] = True
    expect[2:, :2, 9] = True
    assert torch.equal(nan, expect)


def test_magnitudes():
    check([(300, [(60, 2), (30, 2), (0, 1)])], 4, 2, 64, 16, seed=10, spread=2.0 ** 30, scale=0.125 * 2.0 ** -30)
    check([(300, [(60, 2), (30, 2), (0, 1)])], 4, 2, 128, 16, seed=11, scale=-0.1)
    check([(300, [(60, 2), (30, 2), (0, 1)])], 4, 2, 128, 16, seed=12, scale=0.0)

    def far(q):
        q[::2] *= 300
    check([(900, [(20 * i, 2) for i in range(9)])], 16, 2, 128, 32, seed=13, q_edit=far)


def test_rows_past_max_tokens_and_behind_the_last_sequence_stay():
    g, cache, sl, cu, table, cg, shared = build([(256, [(20, 5), (3, 2)])], 4, 2, 64, 16, seed=14)
    q = torch.randn(12, 4, 64, generator=g).to(torch.bfloat16).to(DEV)
    out, lse = torch.full((12, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((12, 4), 7.0, device=DEV)
    sv.spec_kv_attention_shared(q, to_cache(cache), _i32(sl.tolist()), _i32(cu.tolist()), _i32(table.tolist()), 3, _i32(cg.tolist()),
                                _i32(shared.tolist()), out=out, lse=lse)
    stay = torch.tensor([False] * 3 + [True] * 2 + [False] * 2 + [True] * 5, device=DEV)
    assert (out[stay] == 7).all() and (lse[stay] == 7).all() and not (out[~stay] == 7).all(2).any()


def test_captured_replayed_and_on_a_stream():
    g, cache, sl, cu, table, cg, shared = build([(640, [(20 * i, 2) for i in range(20)])], 8, 2, 128, 32, seed=15)
    q = torch.randn(40, 8, 128, generator=g).to(torch.bfloat16).to(DEV)
    kvc, sld, shd = to_cache(cache), _i32(sl.tolist()), _i32(shared.tolist())
    args = (kvc, sld, _i32(cu.tolist()), _i32(table.tolist()), 2, _i32(cg.tolist()), shd)
    size = sv.spec_kv_attention_shared_workspace_bytes(20, 1, 40, 2, 8, 2, 128)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    ref = sv.spec_kv_attention_shared(q, *args, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = sv.spec_kv_attention_shared(q, *args, workspace=ws)
    graph.replay()
    assert torch.equal(kept[0], ref[0]) and torch.equal(kept[1], ref[1])
    shd.fill_(128)
    sld -= 5
    graph.replay()
    now = sv.spec_kv_attention_shared(q, *args)
    assert torch.equal(kept[0], now[0]) and torch.equal(kept[1], now[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sv.spec_kv_attention_shared(q, *args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other[0], now[0])


def test_refusals():
    g, cache, sl, cu, table, cg, shared = build([(64, [(20, 2), (3, 2)])], 4, 2, 64, 16, seed=16)
    q = torch.randn(4, 4, 64, generator=g).to(torch.bfloat16).to(DEV)
    kvc = to_cache(cache)
    a = dict(seq_len=_i32(sl.tolist()), cu_tokens=_i32(cu.tolist()), page_table=_i32(table.tolist()), max_tokens=2,
             cu_groups=_i32(cg.tolist()), shared_len=_i32(shared.tolist()))
    sv.spec_kv_attention_shared(q, kvc, **a)
    for kw in (dict(cu_groups=a["cu_groups"][:1]), dict(cu_groups=a["cu_groups"].long()), dict(shared_len=a["shared_len"].cpu()),
               dict(shared_len=a["shared_len"][:0], cu_groups=a["cu_groups"][:1]), dict(shared_len=_i32([1, 1, 1]), cu_groups=_i32([0, 1, 2, 2])),
               dict(max_tokens=0), dict(max_tokens=5), dict(seq_len=a["seq_len"][:1]), dict(page_table=a["page_table"][0]),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV)), dict(out=q[:2]), dict(lse=q[..., 0]), dict(scale=float("inf"))):
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_kv_attention_shared(q, kvc, **{**a, **kw})
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_kv_attention_shared(q.float(), kvc, **a)
    q.requires_grad_()
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_kv_attention_shared(q, kvc, **a)[0].sum().backward()

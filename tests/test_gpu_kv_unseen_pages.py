"""GPU: pages that no query of the window sees are never looked at, whatever their codes and
scales hold: pages reserved past a sequence's last token, and pages before a sliding window.
Tolerances as in tests/test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv_attention import check

pytestmark = pytest.mark.gpu
# query rows for a kv head: 4 (head_dim 64), 12, 32 (units of 128 tokens), 160 (tensor-core kernel)
SHAPES = [(64, 4, 2, 2), (128, 8, 2, 3), (128, 32, 4, 4), (128, 4, 1, 40)]


def _poison(cache, pages, bad):
    for codes, scale in ((0, 1), (2, 3)):
        cache[codes][pages] = 0x7F
        cache[scale][pages] = bad


@pytest.mark.parametrize("bad", [0.0, float("inf"), float("nan")])
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("dim,heads,kv_heads,new", SHAPES)
def test_reserved_pages_past_the_end(dim, heads, kv_heads, new, page, bad):
    def edit(cache, table):            # every free entry of the table names a page never written
        pool = cache[0].shape[0]
        free = int((table < 0).sum())
        for i in range(4):
            cache[i] = np.concatenate([cache[i], np.ones((free, *cache[i].shape[1:]), cache[i].dtype)])
        _poison(cache, slice(pool, None), bad)
        table[table < 0] = np.arange(pool, pool + free)
    check([5, 17, 64, 100, 130, 0], [new] * 6, heads, kv_heads, dim, page, seed=page + dim, edit=edit)


@pytest.mark.parametrize("bad", [0.0, float("inf"), float("nan")])
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("dim,heads,kv_heads,new", SHAPES)
def test_pages_before_a_sliding_window(dim, heads, kv_heads, new, page, bad):
    lens, window = [100, 250, 371, 3], 20

    def edit(cache, table):
        for b, n in enumerate(lens):
            for j in range(len(table[b])):
                if (j + 1) * page <= n - window + 1:       # its last token lies before query 0's window
                    _poison(cache, table[b][j], bad)
    check(lens, [new] * 4, heads, kv_heads, dim, page, window=window, seed=page + dim, edit=edit)


@pytest.mark.parametrize("heads,kv_heads,new", [(8, 2, 3), (4, 1, 40)])
def test_long_gaps_of_unmapped_pages(heads, kv_heads, new):
    """Units of which nothing is copied, between units that are: what a unit's facts say must be
    there when it is announced, also when no copy has to be waited for."""
    def edit(cache, table):
        for j in range(table.shape[1]):
            if (j // 12) % 2:                        # 192 tokens mapped, 192 not
                table[:, j] = -1
    for seed in range(6):
        check([3000, 700, 2050], [new] * 3, heads, kv_heads, 128, 16, seed=seed, edit=edit, garbage=False)

"""GPU: single tokens, verify windows and long chunks of prompts in one call of spec_kv_attention,
in sizes where items of all kinds share blocks. Tolerances as in tests/test_gpu_kv_attention.py."""
import pytest

from tests.test_gpu_kv_attention import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 8, 2), (128, 8, 2), (128, 64, 8)])
def test_chunks_beside_single_tokens(dim, heads, kv_heads, page):
    lens = [1200, 0, 300, 5, 2500, 700, 64, 129, 0, 1, -1, 900, 33, 2000, 80, 17]
    new = [1, 150, 1, 5, 1, 97, 1, 5, 1, 5, 4, 0, 1, 65, 1, 5]
    check(lens, new, heads, kv_heads, dim, page, seed=dim + heads + page, seqs=None if heads < 64 else range(0, 16, 3))


@pytest.mark.parametrize("window", [40, 700])
def test_in_a_sliding_window(window):
    check([1200, 0, 300, 5, 2500], [1, 150, 5, 1, 90], 4, 1, 128, 32, window=window, seed=window)

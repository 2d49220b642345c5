"""GPU: value scales at the ends of the range that include/spec_kv.h states: 2^-100 and 2^100, and
a factor of 2^96 between the pages of a sequence. Tolerances as in
tests/test_gpu_kv_attention.py: a key that weighs less than 2^-37 of the largest may be lost
there, which for n keys is n 2^-37 of the sum, below the n / 8 2^-24 of its additions."""
import numpy as np
import pytest

from tests.test_gpu_kv_attention import check

pytestmark = pytest.mark.gpu
SHAPES = [(64, 4, 2, 2), (128, 8, 2, 3), (128, 32, 4, 4), (128, 4, 1, 40)]


@pytest.mark.parametrize("exponents", [(-48, 48), (48, -48), (-60, 36), (-100, -100), (100, 100), (-100, -4), (100, 4)])
@pytest.mark.parametrize("dim,heads,kv_heads,new", SHAPES)
def test_ends_of_the_range(dim, heads, kv_heads, new, exponents):
    def edit(cache, table):
        for b in range(table.shape[0]):
            for j, p in enumerate(table[b]):
                if p >= 0:
                    cache[3][p] = np.float32(2.0) ** exponents[j % 2]
                    if exponents == (-60, 36) and j % 2 == 0:
                        cache[2][p] = 0                      # pages of zeros, as the append scales them
    check([90, 700, 31], [new] * 3, heads, kv_heads, dim, 16, seed=dim + new, edit=edit, garbage=False)

"""GPU: queries whose elements differ by orders of magnitude (a few strong channels) are scored
as exactly by every kernel of spec_kv_attention: the bound is the one of
tests/test_gpu_kv_attention.py, with keys that are 0 in the strong channel, so that the logits
come from the small elements alone."""
import pytest
import torch

from tests.test_gpu_kv_attention import check

pytestmark = pytest.mark.gpu


def _run(lens, new, heads, kv_heads, dim, ratio, seed):
    strong = 5

    def edit(cache, table):
        cache[0][..., strong] = 0

    def q_edit(q):
        q[..., strong] = ratio
        q[::2, :, strong] = -ratio
    check(lens, new, heads, kv_heads, dim, 32, seed=seed, edit=edit, q_edit=q_edit, garbage=False)


@pytest.mark.parametrize("ratio", [30.0, 300.0, 1000.0, 30000.0])
@pytest.mark.parametrize("lens,new,heads,kv_heads,dim", [
    ([40, 300], [3, 2], 8, 2, 64), ([40, 300], [3, 2], 8, 2, 128), ([40, 300], [8, 8], 16, 2, 128),
    ([40, 300, 0], [70, 50, 130], 4, 1, 128), ([200, 1000], [3, 90], 8, 2, 128)])
def test_strong_channels(lens, new, heads, kv_heads, dim, ratio):
    _run(lens, new, heads, kv_heads, dim, ratio, seed=int(ratio) + dim + heads)


@pytest.mark.parametrize("new", [[3, 2], [80, 40]])
def test_an_infinite_element_makes_its_row_nan(new):
    def q_edit(q):
        q[1, 1, 5] = float("inf")
        q[4, 0, 77] = -float("inf")
    check([50, 200], new, 8, 2, 128, 16, seed=3, q_edit=q_edit, nan_ok=True)


def test_a_long_window_in_the_batch_changes_no_other_precision():
    # one short window alone and beside a long one: both within the bound, whatever kernel runs
    for new in ([4], [4, 100]):
        _run([700, 90][:len(new)], new, 4, 1, 128, 3000.0, seed=9)


def test_every_element_of_another_size():
    # from 1 down to 2^-24 of the row's largest; keys grow the other way as far as e4m3 goes
    def q_edit(q):
        q.mul_(2.0 ** -torch.linspace(0, 24, q.shape[-1]))

    def edit(cache, table):
        d = cache[0].shape[-1]
        for c in range(d):
            cache[0][..., c] = (cache[0][..., c] & 0x87) | (min(c * 15 // d, 14) << 3)
    for new in ([6], [90]):
        check([300], new, 4, 1, 128, 32, seed=4, q_edit=q_edit, edit=edit, garbage=False, scale=1.0)

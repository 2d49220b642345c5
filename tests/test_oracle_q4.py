"""CPU: the oracle of the 4-bit LM head against closed forms, its bound against fp32 sums in several
orders, and the quantiser."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from oracle import q4


def test_codes_lie_low_half_first():
    codes = np.array([[0x21, 0x43]], np.uint8)
    w = q4.weight(codes, np.array([[2.0, 0.5]]), np.array([[-1.0, 3.0]]))
    assert w.tolist() == [[1.0, 3.0, 4.5, 5.0]]
    assert q4.logits(np.array([[1.0, 0, 0, 2.0]]), codes, np.array([[2.0, 0.5]]), np.array([[-1.0, 3.0]])).tolist() == [[11.0]]


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantise_and_back(group):
    g = torch.Generator().manual_seed(group)
    w = torch.randn(40, 256, generator=g) * torch.exp(torch.randn(40, 1, generator=g))
    w[3] = 0.25                                   # a constant row
    q = sv.Q4Weight.quantize(w, group)
    ref = q4.weight(q.codes.numpy(), q.scale.float().numpy(), q.bias.float().numpy())
    assert np.abs(q.dequantize().double().numpy() - ref).max() <= 2.0 ** -23 * np.abs(ref).max()
    # half a step, and what the bf16 rounding of step and bias (2^-8 of each) moves the ends by
    span = (w.unflatten(1, (-1, group)).amax(2) - w.unflatten(1, (-1, group)).amin(2)).repeat_interleave(group, 1)
    low = w.unflatten(1, (-1, group)).amin(2).abs().repeat_interleave(group, 1)
    err = (q.dequantize() - w).abs()
    assert (err <= span / 30 * (1 + 2.0 ** -7) + 2.0 ** -8 * (span + low) + 1e-7).all()
    assert (q.codes[3] == 0).all()


def test_quantise_refuses():
    for w, group in ((torch.zeros(4, 96), 64), (torch.zeros(4, 128), 48), (torch.zeros(128), 64), (torch.zeros(4, 128).int(), 64)):
        with pytest.raises(sv.SpecVerifyError):
            sv.Q4Weight.quantize(w, group)


def test_bound_holds_for_fp32_sums():
    r = np.random.default_rng(0)
    d, group, V = 512, 64, 20
    h = r.normal(size=(3, d)).astype(np.float32)
    h = torch.from_numpy(h).to(torch.bfloat16).float().numpy()
    codes = r.integers(0, 256, (V, d // 2), dtype=np.uint8)
    scale = torch.from_numpy(r.uniform(0.01, 0.1, (V, d // group)).astype(np.float32)).to(torch.bfloat16).float().numpy()
    bias = torch.from_numpy(r.normal(size=(V, d // group)).astype(np.float32)).to(torch.bfloat16).float().numpy()
    ref, bound = q4.logits(h, codes, scale, bias), q4.error_bound(h, codes, scale, bias)
    q = np.empty((V, d), np.float32)
    q[:, 0::2], q[:, 1::2] = codes % 16, codes // 16
    for order in (np.arange(d), np.arange(d)[::-1]):
        got = np.zeros((3, V), np.float32)
        for g in range(d // group):
            a, x = np.zeros((3, V), np.float32), np.zeros((3, 1), np.float32)
            for j in order[(order // group) == g]:
                a += h[:, j:j + 1] * (q[:, j] - 8)
                x += h[:, j:j + 1]
            got += scale[:, g] * a + (bias[:, g] + 8 * scale[:, g]) * x
        assert (np.abs(got - ref) <= bound).all()
    assert (np.abs(q4.logits(h, codes, scale, bias * 1.01) - ref) > bound).any()      # a planted mistake

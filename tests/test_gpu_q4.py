"""GPU: the LM head in 4 bits against the float64 oracle, within its bound for fp32 sums."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from oracle import q4

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(M, V, d, group, seed=0, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    h = (torch.randn(M, d, generator=g) * gain).to(torch.bfloat16)
    codes = torch.randint(0, 256, (V, d // 2), generator=g, dtype=torch.uint8)
    scale = torch.exp(torch.randn(V, d // group, generator=g) - 4).to(torch.bfloat16)
    bias = (scale.float() * (-7.5 + torch.randn(V, d // group, generator=g))).to(torch.bfloat16)
    return h, codes, scale, bias


def check(M, V, d, group, seed=0, gain=1.0):
    host = make(M, V, d, group, seed, gain)
    h, *w = (t.to(DEV) for t in host)
    got = sv.spec_lm_head_logits_q4(h, sv.Q4Weight(*w))
    again = sv.spec_lm_head_logits_q4(h, sv.Q4Weight(*w))
    torch.cuda.synchronize()
    assert got.shape == (M, V) and torch.equal(got, again)
    args = [t.double().numpy() if t.dtype != torch.uint8 else t.numpy() for t in host]
    err = np.abs(got.double().cpu().numpy() - q4.logits(*args))
    bound = q4.error_bound(*args)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 5, 8, 9, 16, 17, 33, 64, 65, 130])
def test_rows(M, group):
    check(M, 700, 384, group, seed=M + group)


@pytest.mark.parametrize("V", [1, 15, 16, 17, 31, 127, 128, 129, 2501])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 128), (320, 64), (1024, 64), (4096, 128), (8192, 32)])
def test_vocabularies_and_widths(V, d, group):
    check(3, V, d, group, seed=V + d)
    check(1, V, d, group, seed=V + d + 1)


@pytest.mark.parametrize("gain", [1e-30, 1e30])
def test_magnitudes(gain):
    check(4, 300, 256, 64, gain=gain)


def test_a_wide_hidden_dimension():
    check(2, 40, 65536, 128)
    check(20, 40, 65536, 32)


def test_the_whole_vocabulary():
    h, codes, scale, bias = make(4, 151936, 256, 64, seed=3)
    got = sv.spec_lm_head_logits_q4(h.to(DEV), sv.Q4Weight(codes.to(DEV), scale.to(DEV), bias.to(DEV))).double().cpu().numpy()
    at = np.r_[0:300, 75000:75300, 151636:151936]
    args = [h.double().numpy(), codes[at].numpy(), scale[at].double().numpy(), bias[at].double().numpy()]
    assert (np.abs(got[:, at] - q4.logits(*args)) <= q4.error_bound(*args)).all()


@pytest.mark.parametrize("M", [1, 12])
def test_non_finite_values_stay_in_their_rows_and_columns(M):
    h, codes, scale, bias = make(M, 200, 256, 64, seed=4)
    ref = sv.spec_lm_head_logits_q4(h.to(DEV), sv.Q4Weight(codes.to(DEV), scale.to(DEV), bias.to(DEV)))
    for bad in (float("nan"), float("inf")):
        h2, s2, b2 = h.clone(), scale.clone(), bias.clone()
        h2[M - 1, 77], s2[50, 1], b2[120, 3] = bad, bad, bad
        got = sv.spec_lm_head_logits_q4(h2.to(DEV), sv.Q4Weight(codes.to(DEV), s2.to(DEV), b2.to(DEV)))
        hit = torch.zeros(M, 200, dtype=torch.bool, device=DEV)
        hit[M - 1], hit[:, 50], hit[:, 120] = True, True, True
        assert not torch.isfinite(got[hit]).any() and torch.equal(got[~hit], ref[~hit])


def test_shapes_outputs_and_streams():
    h, codes, scale, bias = make(6, 333, 128, 64, seed=5)
    w = sv.Q4Weight(codes.to(DEV), scale.to(DEV), bias.to(DEV))
    ref = sv.spec_lm_head_logits_q4(h.to(DEV), w)
    x = h.to(DEV).view(2, 3, 128)
    assert torch.equal(sv.spec_lm_head_logits_q4(x, w), ref.view(2, 3, 333))
    assert torch.equal(sv.spec_lm_head_logits_q4(x[1, 2], w), ref[5])
    out = torch.empty(6, 333, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert sv.spec_lm_head_logits_q4(h.to(DEV), w, out=out, stream=side) is out
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    hd = h.to(DEV)
    with torch.cuda.graph(graph):
        kept = sv.spec_lm_head_logits_q4(hd, w)
    hd.copy_(h.flip(0))
    graph.replay()
    assert torch.equal(kept, ref.flip(0))


def test_refusals():
    h, codes, scale, bias = make(6, 333, 128, 64, seed=6)
    hd, w = h.to(DEV), sv.Q4Weight(codes.to(DEV), scale.to(DEV), bias.to(DEV))
    for x, y in ((hd.float(), w), (hd[:, :64], w), (hd.T, w), (hd, w._replace(codes=w.codes.int())), (hd, w._replace(scale=w.scale.float())),
                 (hd, w._replace(bias=w.bias[:, :1])), (hd, w._replace(scale=w.scale[:100])), (hd, w._replace(codes=codes)), (hd, w.codes),
                 (hd[:0], w), (hd, w._replace(scale=w.scale[:, :1].contiguous(), bias=w.bias[:, :0])), (hd.t().contiguous().t(), w),
                 (hd, w._replace(scale=w.scale.repeat(1, 4), bias=w.bias.repeat(1, 4)))):     # groups of 16
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_lm_head_logits_q4(x, y)
    for out in (torch.empty(6, 332, device=DEV), torch.empty(6, 333, device=DEV, dtype=torch.bfloat16), torch.empty(6, 333)):
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_lm_head_logits_q4(hd, w, out=out)
    hd.requires_grad_()
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_lm_head_logits_q4(hd, w).sum().backward()


def test_a_quantised_head_chooses_the_tokens_of_its_own_weights():
    g = torch.Generator().manual_seed(7)
    W = torch.randn(3000, 256, generator=g).to(DEV)
    w = sv.Q4Weight.quantize(W, 64)
    h = torch.randn(9, 256, generator=g).to(torch.bfloat16).to(DEV)
    z = h.double() @ w.dequantize().double().T
    got = sv.spec_lm_head_logits_q4(h, w)
    top = z.topk(2).values
    clear = (top[:, 0] - top[:, 1]) > 1e-3
    assert clear.sum() > 5 and torch.equal(got.argmax(1)[clear], z.argmax(1)[clear])

"""GPU: the gradient of rows whose log-sum-exp is far from zero (low temperatures, shifted
logits) against a float64 gradient that forms its own log-sum-exp.

Tolerances (u = 2^-24): a probability's exponent is off by 16 u of itself, the sum of
exponentials by 2^-22 and at most 93 additions (64 logits of a thread, 29 to join threads, warps
and blocks), each exponential by 2^-22 more, and log2 of the sum by 2^-23 of itself; then the
rounding of the output type. Probabilities below 2^-126 count as 0."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from oracle import logprobs

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# (factor of normal logits, shift, temperature): |lse| from about 30 to 10^6
ROWS = [(2, 20, 1.0), (10, 0, 0.05), (2, 60, 1.0), (2, -95, 0.5), (12, 0, 0.05), (2, 500, 1.0), (2, -900, 1.0), (30, 0, 0.15),
        (10, 0, 0.01), (2, 1500, 1.0), (2, 40, 0.05), (2, -1e6, 1.0)]


def _case(V, dtype, in_place, off=0, n=3):
    R = len(ROWS)
    g = torch.Generator().manual_seed(V)
    x = torch.randn(R, V + off, generator=g)
    for r, (f, s, _) in enumerate(ROWS):
        x[r] = x[r] * f + s
    x[7, off::2] = -float("inf")
    x[6, off::3] = torch.finfo(TYPES[dtype]).min
    x = x.to(TYPES[dtype])
    temp = torch.tensor([t for _, _, t in ROWS])
    tok = torch.randint(0, V, (R,), generator=g, dtype=torch.int32)
    best = x[:, off:].float().argmax(1).to(torch.int32)
    tok[::2] = best[::2]                                   # confident rows among them
    tok[3] = -1
    glp, gh, gt = torch.randn(R, generator=g), torch.randn(R, generator=g), torch.randn(R, n, generator=g)
    xd = x.to(DEV)[:, off:]
    z = x[:, off:].double().numpy()
    f = sv.spec_token_logprobs(xd, tok.to(DEV), temp.to(DEV), n)
    out = xd if in_place else None if off == 0 else torch.empty(R, V, dtype=xd.dtype, device=DEV)
    d = sv.spec_token_logprobs_backward(xd, tok.to(DEV), f.lse, f.entropy, temp.to(DEV), glp.to(DEV), gh.to(DEV), f.top_ids,
                                        gt.to(DEV), out=out).cpu().double().numpy()
    half = torch.finfo(TYPES[dtype]).eps / 2
    for r in range(R):
        T, t = float(temp[r]), int(tok[r])
        if t < 0:
            assert (d[r] == 0).all()
            continue
        _, _, H, _, ids, _ = logprobs.row(z[r], t, T, n)
        assert f.top_ids[r].tolist() == ids
        y = (z[r] - z[r].max()) / T
        lsum = np.log(np.exp(y).sum())
        lp = np.maximum(y - lsum, -700.0)
        up = np.zeros(V)
        up[t] += float(glp[r])
        for j, v in zip(ids, gt[r].tolist()):
            up[j] += v
        ref = (up - np.exp(lp) * (up.sum() + float(gh[r]) * (lp + H))) / T
        size = abs(float(glp[r])) + float(gt[r].abs().sum()) + abs(float(gh[r])) * (np.abs(lp) + H)
        rel = 2.0 ** -21 + (93 + 16 + 16 * np.abs(lp)) * U + lsum * 2.0 ** -23
        if abs(float(f.lse[r])) <= 64:                     # formed from the given lse of 32 bits
            rel = rel + 2.0 ** -19
        tol = np.exp(lp) * size / T * rel + half * np.abs(ref) * 1.01
        tol = tol + 8 * U * np.abs(up) / T + 8 * U * size / T * (up != 0) + 2.0 ** -126 * size / T + 1e-37
        # the entropy is the forward's, good to (V / 512 + 320) u of 1 + 2 sum p |z - m|
        spread = 1 + 2 * (np.exp(lp) * np.abs(np.maximum(y, -700.0))).sum()
        tol = tol + np.exp(lp) * abs(float(gh[r])) / T * ((V / 512 + 320) * U + 2.0 ** -22) * spread
        err = np.abs(d[r] - ref)
        k = int((err / tol).argmax())
        assert (err <= tol).all(), (r, k, err[k], tol[k], ref[k])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [2051, 40003, 151936, 262144])
def test_far_rows(V, dtype, in_place):
    _case(V, dtype, in_place)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,off", [(33000, 8), (20001, 1), (140001, 3)])
def test_far_rows_off_alignment(V, off, dtype):
    _case(V, dtype, False, off)


def test_a_confident_row_has_no_spurious_gradient():
    # p of the best token is 1 - 2^-40 or nearer: its gradient is 0 to a rounding, not to that of lse
    V = 5000
    x = torch.zeros(4, V, device=DEV)
    x[:, 17] = torch.tensor([40.3, 45.7, 50.1, 48.9], device=DEV)
    temp = torch.tensor([0.05, 0.05, 0.06, 0.09], device=DEV)
    tok = torch.full((4,), 17, dtype=torch.int32, device=DEV)
    f = sv.spec_token_logprobs(x, tok, temp)
    d = sv.spec_token_logprobs_backward(x, tok, f.lse, f.entropy, temp, grad_logprob=torch.ones(4, device=DEV))
    assert float((d * temp[:, None]).abs().max()) <= 2.0 ** -21

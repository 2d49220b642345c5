"""GPU: token log-probabilities and their gradient against the float64 oracle.

Tolerances, from the kernels' arithmetic (u = 2^-24 the fp32 rounding):
* the softmax sum: at most V / 512 + 16 additions in one thread and 40 more to merge,
  each u; 2^-22 for the exponential and 4 u for its argument's rounding for each
  unit of the exponent (64 units are taken): e = (V / 512 + 56) u + 2^-22 + 256 u;
* lse, logprob: e + 4 u (|z_t - m| + |lse|);  entropy: e (1 + 2 sum p |z - m|);
* gradient: relative 2^-22 + (16 + 8 |log2 p|) u on each product with p, then the
  rounding of the output type.
Ranks and ids are integers of the logits as given: exact."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from oracle import logprobs

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _check(x, tok, temp, n, rows=None):
    """x [R, V] on the device (any stride); compares `rows` (all by default)."""
    got = sv.spec_token_logprobs(x, tok.to(DEV), None if temp is None else temp.to(DEV), n)
    torch.cuda.synchronize()
    got = [g.cpu().double().numpy() if g.is_floating_point() else g.cpu().numpy() for g in got]
    lp, rank, H, lse, ids, lps = got
    for r in range(x.shape[0]) if rows is None else rows:
        z = x[r].cpu().double().numpy()
        T = 1.0 if temp is None else float(temp[r])
        ref = logprobs.row(z, int(tok[r]), T, n)
        if ref is None:
            assert np.isnan(lp[r]) and np.isnan(H[r]) and np.isnan(lse[r]) and rank[r] == -1, r
            assert (ids[r] == -1).all() and np.isnan(lps[r]).all()
            continue
        assert rank[r] == ref[1], (r, rank[r], ref[1])
        assert list(ids[r]) == ref[4], (r, list(ids[r]), ref[4])
        if int(tok[r]) < 0:
            assert lp[r] == 0 and H[r] == 0 and lse[r] == 0 and (lps[r] == 0).all()
            continue
        T = T or 1.0
        e = (z.size / 512 + 56 + 256) * U + 2.0 ** -22
        y = z[z > -np.inf] / T
        p = np.exp(y - y.max())
        p /= p.sum()

        def near(a, b, m):
            if np.isinf(np.float32(b)):            # past the output type's range
                return a == np.float32(b)
            if np.isinf(b):
                return a == b
            return abs(a - b) <= e + 4 * U * (abs(m) + abs(ref[3]))
        assert near(lse[r], ref[3], y.max()), (r, lse[r], ref[3])
        assert near(lp[r], ref[0], z[int(tok[r])] / T - y.max()), (r, lp[r], ref[0])
        assert abs(H[r] - ref[2]) <= e * (1 + 2 * (p * np.abs(y - y.max())).sum()), (r, H[r], ref[2])
        for a, b in zip(lps[r], ref[5]):
            assert near(a, b, b), (r, a, b)


def _rows(R, V, dtype, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(R, V, generator=g) * scale).to(TYPES[dtype])
    tok = torch.randint(0, V, (R,), generator=g, dtype=torch.int32)
    temp = 0.4 + torch.rand(R, generator=g)
    return x, tok, temp, g


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,V,n", [(1, 2, 2), (3, 7, 5), (2, 15, 1), (5, 255, 20), (2, 257, 32), (1, 4097, 20),
                                   (7, 32003, 10), (1, 151936, 20), (400, 1000, 4), (2, 262144, 32), (40, 50257, 0)])
def test_matches_oracle(R, V, n, dtype):
    x, tok, temp, g = _rows(R, V, dtype, R * 7 + V)
    temp[0] = 0.0
    if R > 2:
        tok[1] = -1
    tok[-1] = V - 1
    _check(x.to(DEV), tok, temp, n, None if R < 50 else range(0, R, 17))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("off,pad", [(0, 0), (1, 0), (3, 5), (5, 1), (7, 8)])
def test_offsets_and_row_strides(off, pad, dtype):
    R, V = 6, 3001
    x, tok, temp, _ = _rows(R, V + off + pad, dtype, 11 + off)
    tok = tok % V
    tok[0], tok[1], tok[2] = 0, V - 1, min(off, V - 1)
    _check(x.to(DEV)[:, off:off + V], tok, None, 9)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ties_runs_and_bans(dtype):
    V, n = 20011, 32
    rows = [torch.zeros(V),                                        # all equal
            torch.full((V,), -float("inf")).index_fill(0, torch.tensor([77, 19000]), 1.5),   # two finite logits
            torch.arange(V).float() / 64,                          # rising: the best lie in one group
            -torch.arange(V).float() / 64,                         # falling
            (torch.arange(V) % 5).float(),                         # long ties across groups
            torch.randn(V, generator=torch.Generator().manual_seed(1)),
            torch.randn(V, generator=torch.Generator().manual_seed(2)) * 60]
    rows[5][1000:] = -float("inf")
    rows.append(torch.zeros(V))                                    # -0 and +0 are equal
    rows[7][::2] = -0.0
    rows.append(torch.randn(V, generator=torch.Generator().manual_seed(3)))
    rows[8][torch.rand(V, generator=torch.Generator().manual_seed(4)) < 0.95] = -float("inf")
    x = torch.stack(rows).to(TYPES[dtype])
    for tok in (torch.tensor([5, 77, 3, 3, 14, 10, 6, 9, 2]), torch.tensor([V - 1, 0, V - 1, V - 1, V - 1, V - 1, 0, V - 2, 0])):
        _check(x.to(DEV), tok.to(torch.int32), torch.tensor([1, 1, .5, 2, 1, 1, 1, 1, 0.7]), n)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_data_errors_stay_in_their_row(dtype):
    V = 9001
    x, tok, temp, _ = _rows(12, V, dtype, 5)
    x[0, 8999] = float("nan")
    x[2, 0] = float("inf")
    x[3] = -float("inf")
    tok[4] = V
    temp[5], temp[6], temp[7] = -1.0, float("nan"), float("inf")
    x[8, V - 1] = float("nan")
    temp[9] = 1e-39
    tok[10] = -5
    got = sv.spec_token_logprobs(x.to(DEV), tok.to(DEV), temp.to(DEV), 3)
    bad = torch.isnan(got.logprob).cpu()
    assert bad.tolist() == [i in (0, 2, 3, 4, 5, 6, 7, 8, 9) for i in range(12)]
    _check(x.to(DEV), tok, torch.where(torch.arange(12) == 9, torch.tensor(1.0), temp), 3)


def test_emitted_tokens_of_a_verify_step():
    B, K, V = 6, 3, 4000
    g = torch.Generator().manual_seed(8)
    tgt = (torch.randn(B, K + 1, V, generator=g) * 3).to(DEV)
    drf = tgt[:, :K] + 0.5 * torch.randn(B, K, V, generator=g).to(DEV)
    dtok = drf.argmax(-1).to(torch.int32)
    par = (torch.ones(B, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV), torch.ones(B, device=DEV))
    out, n = sv.spec_verify(tgt, drf, dtok, *par, seed=3, offset=0)
    r = sv.spec_token_logprobs(tgt, out, top_n=2)
    assert r.logprob.shape == (B, K + 1) and r.top_ids.shape == (B, K + 1, 2)
    lp = torch.log_softmax(tgt.double(), -1)
    for b in range(B):
        for i in range(K + 1):
            t = int(out[b, i])
            if i <= int(n[b]):
                assert abs(float(r.logprob[b, i]) - float(lp[b, i, t])) < 1e-5
            else:
                assert t == -1 and float(r.logprob[b, i]) == 0 and int(r.rank[b, i]) == -1


def test_repeated_calls_give_the_same_bits_on_any_stream():
    x, tok, temp, _ = _rows(37, 60001, "bf16", 3)
    x, tok, temp = x.to(DEV), tok.to(DEV), temp.to(DEV)
    a = sv.spec_token_logprobs(x, tok, temp, 7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = sv.spec_token_logprobs(x, tok, temp, 7, stream=side)
    side.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def _grad_case(R, V, dtype, n, seed, in_place=False, off=0, same=True):
    x, tok, temp, g = _rows(R, V + off, dtype, seed)
    x, tok = x.to(DEV)[:, off:], tok % V
    temp[0] = 0.0
    if R > 3:
        tok[1] = -1
        x[2, ::3] = -float("inf")
        tok[2] = 1
    glp, gh, gt = torch.randn(R, generator=g), torch.randn(R, generator=g), torch.randn(R, n, generator=g)
    f = sv.spec_token_logprobs(x, tok.to(DEV), temp.to(DEV), n)
    z = x.cpu().double().numpy()
    out = x if in_place else None if same else torch.empty_like(x.contiguous())
    d = sv.spec_token_logprobs_backward(x, tok.to(DEV), f.lse, f.entropy, temp.to(DEV), glp.to(DEV), gh.to(DEV),
                                        f.top_ids, gt.to(DEV), out=out)
    torch.cuda.synchronize()
    d = d.cpu().double().numpy()
    half = torch.finfo(TYPES[dtype]).eps / 2          # unit roundoff of the output type
    for r in range(R):
        T = float(temp[r]) or 1.0
        lse, H = float(f.lse[r]), float(f.entropy[r])
        a = (z[r], int(tok[r]), T, lse, H, float(glp[r]), float(gh[r]), f.top_ids[r].tolist(), gt[r].double().tolist())
        ref = logprobs.row_gradient(*a)
        if int(tok[r]) < 0:
            assert (d[r] == 0).all()
            continue
        lp = np.maximum(z[r] / T - lse, -700.0)
        big = abs(float(glp[r])) + float(gt[r].abs().sum()) + abs(float(gh[r])) * (np.abs(lp) + H)
        tol = np.exp(lp) * big / T * (2.0 ** -22 + (16 + 8 * np.abs(lp) / np.log(2)) * U)
        tol = tol + half * np.abs(ref) * 1.01 + 8 * U * big / T * np.isin(np.arange(V), [int(tok[r])] + f.top_ids[r].tolist())
        assert (np.abs(d[r] - ref) <= tol + 1e-37).all(), (r, np.abs(d[r] - ref).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,V,n", [(1, 2, 0), (5, 9, 3), (4, 1001, 5), (6, 32003, 20), (2, 151936, 32), (5, 8192, 1)])
def test_gradient_matches_oracle(R, V, n, dtype):
    _grad_case(R, V, dtype, n, V + n)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_in_place_and_misaligned(dtype):
    _grad_case(5, 5003, dtype, 4, 1, in_place=True)
    _grad_case(5, 5003, dtype, 4, 2, off=1, same=False)      # logits and gradient sit differently to 16 bytes
    _grad_case(5, 5000, dtype, 4, 3, off=8)


def test_gradient_through_autograd_and_differences():
    V, n = 300, 3
    x, tok, temp, g = _rows(2, V, "fp32", 9)
    x, temp = x.to(DEV).requires_grad_(), temp.to(DEV)
    w = torch.randn(2, 2 + n, generator=g)
    r = sv.spec_token_logprobs(x, tok.to(DEV), temp, n)
    wd = w.to(DEV)
    loss = (wd[:, 0] * r.logprob + wd[:, 1] * r.entropy).sum() + (wd[:, 2:] * r.top_logprobs).sum()
    loss.backward()
    ids = r.top_ids.cpu()
    x64, w = x.detach().cpu().double().numpy(), w.double().numpy()

    def value(i, z):
        lp, _, H, lse, _, _ = logprobs.row(z, int(tok[i]), float(temp[i]))
        return w[i, 0] * lp + w[i, 1] * H + sum(w[i, 2 + k] * (z[j] / float(temp[i]) - lse) for k, j in enumerate(ids[i].tolist()))
    for i in range(2):
        for j in list(range(0, V, 23)) + [int(tok[i])] + ids[i].tolist():
            e = np.zeros(V)
            e[j] = 1e-4
            diff = (value(i, x64[i] + e) - value(i, x64[i] - e)) / 2e-4
            # the second-order term of the difference is below 1e-7 here; fp32 gives 1e-6
            assert abs(float(x.grad[i, j]) - diff) < 5e-6 * (1 + abs(diff))


def test_gradient_of_parts_and_errors():
    x, tok, temp, _ = _rows(3, 500, "fp32", 4)
    x = x.to(DEV).requires_grad_()
    r = sv.spec_token_logprobs(x, tok.to(DEV))
    r.logprob.sum().backward()
    p = torch.softmax(x.detach().double(), -1)
    ref = -p
    ref[torch.arange(3), tok.long()] += 1
    assert float((x.grad - ref).abs().max()) < 2e-6
    y = x.detach().clone()
    y[1, 3] = float("nan")
    f = sv.spec_token_logprobs(y, tok.to(DEV))
    d = sv.spec_token_logprobs_backward(y, tok.to(DEV), f.lse, f.entropy, grad_logprob=torch.ones(3, device=DEV))
    assert torch.isnan(d[1]).all() and not torch.isnan(d[0]).any() and not torch.isnan(d[2]).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [0.5, 1.3, 2.0])
def test_lowest_values_at_temperatures(T, dtype):
    V, low = 9001, torch.finfo(TYPES[dtype]).min
    g = torch.Generator().manual_seed(8)
    x = (torch.randn(5, V, generator=g) * 2)
    x[0] = low
    x[1][torch.rand(V, generator=g) < 0.9] = low
    x[1, 17] = low
    x[2, 5:] = low
    x[3] = low
    x[3, 40] = -1e30
    x = x.to(TYPES[dtype])
    _check(x.to(DEV), torch.tensor([4, 17, 9000, 40, 3], dtype=torch.int32), torch.full((5,), T), 7)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_of_logits_far_from_zero(dtype, in_place):
    # p is formed from the row: its exponents are off by 2^-23 of themselves (those that matter are
    # below 150), the sum by V / 256 + 16 roundings
    V, low = 40003, torch.finfo(TYPES[dtype]).min
    g = torch.Generator().manual_seed(12)
    x = torch.randn(6, V, generator=g) * 2
    x[0] = low
    x[1] += 30000.0
    x[2] -= 30000.0
    x[3, 2:] = low
    x[3, :2] = 5e4
    x[4] *= 1e30
    x = x.to(TYPES[dtype])
    tok = torch.tensor([3, 40002, 7, 1, int(x[4].float().argmax()), 9], dtype=torch.int32)
    temp, n = torch.tensor([0.5, 1.0, 2.0, 1.0, 1.0, 1.0]), 3
    glp, gh, gt = torch.randn(6, generator=g), torch.randn(6, generator=g), torch.randn(6, n, generator=g)
    xd = x.to(DEV)
    f = sv.spec_token_logprobs(xd, tok.to(DEV), temp.to(DEV), n)
    d = sv.spec_token_logprobs_backward(xd, tok.to(DEV), f.lse, f.entropy, temp.to(DEV), glp.to(DEV), gh.to(DEV), f.top_ids,
                                        gt.to(DEV), out=xd if in_place else None).cpu().double().numpy()
    for r in range(6):
        z, T = x[r].double().numpy(), float(temp[r])
        _, _, H, _, ids, _ = logprobs.row(z, int(tok[r]), T, n)
        assert f.top_ids[r].tolist() == ids
        lp = (z - z.max()) / T
        lp = np.maximum(lp - np.log(np.exp(lp).sum()), -700.0)
        up = np.zeros(V)
        up[int(tok[r])] += float(glp[r])
        for j, v in zip(ids, gt[r].tolist()):
            up[j] += v
        ref = (up - np.exp(lp) * (up.sum() + float(gh[r]) * (lp + H))) / T
        size = abs(float(glp[r])) + float(gt[r].abs().sum()) + abs(float(gh[r])) * (np.abs(lp) + H)
        half = torch.finfo(TYPES[dtype]).eps / 2
        tol = np.exp(lp) * size / T * (2.0 ** -20 + (V / 256 + 64 + 16 * np.abs(lp)) * U) + half * np.abs(ref) * 1.01
        tol = tol + 8 * U * np.abs(up) / T + 8 * U * size / T * (up != 0) + 1e-37
        assert (np.abs(d[r] - ref) <= tol).all(), (r, np.abs(d[r] - ref).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_one_row_for_many_tokens(dtype):
    x, tok, temp, _ = _rows(1, 5008, dtype, 21)
    tok = torch.arange(0, 5000, 700, dtype=torch.int32, device=DEV)
    R = tok.numel()
    x = x.to(DEV).requires_grad_()
    wide = x.expand(R, -1)
    r = sv.spec_token_logprobs(wide, tok, top_n=3)
    ref = sv.spec_token_logprobs(x.detach().repeat(R, 1), tok, top_n=3)
    for a, b in zip(r, ref):
        assert torch.equal(a.detach(), b)
    r.logprob.sum().backward()
    d = sv.spec_token_logprobs_backward(x.detach().repeat(R, 1), tok, ref.lse, ref.entropy, grad_logprob=torch.ones(R, device=DEV))
    assert torch.equal(x.grad, d.sum(0, keepdim=True))
    with pytest.raises(sv.SpecVerifyError):        # the gradient's rows are each their own
        sv.spec_token_logprobs_backward(wide.detach(), tok, ref.lse, ref.entropy, out=wide.detach())


def test_refusals():
    x, tok = torch.zeros(4, 64, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    E = sv.SpecVerifyError
    for bad in (lambda: sv.spec_token_logprobs(x.half(), tok), lambda: sv.spec_token_logprobs(x, tok.long()),
                lambda: sv.spec_token_logprobs(x, tok[:3]), lambda: sv.spec_token_logprobs(x.t(), tok),
                lambda: sv.spec_token_logprobs(x[0], tok[:1]), lambda: sv.spec_token_logprobs(x, tok, tok),
                lambda: sv.spec_token_logprobs(x, tok, top_n=40), lambda: sv.spec_token_logprobs(x[:, :1], tok),
                lambda: sv.spec_token_logprobs_backward(x, tok, x[:, 0], x[:, 0]),
                lambda: sv.spec_token_logprobs_backward(x, tok, torch.zeros(4, device=DEV), torch.zeros(4, device=DEV),
                                                        grad_top=torch.zeros(4, 2, device=DEV))):
        with pytest.raises(E):
            bad()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masks_of_the_lowest_value(dtype):
    # finite masks count as logits: alone they are all alike, beside others they weigh nothing
    V = 5003
    low = torch.finfo(TYPES[dtype]).min
    g = torch.Generator().manual_seed(6)
    x = torch.full((6, V), low)
    x[1, ::2] = -float("inf")                     # -inf beside the lowest value
    x[2, 7] = 3.0
    x[3] = torch.randn(V, generator=g) * 2
    x[3, 100:4000] = low
    x[4] = torch.randn(V, generator=g) * 1e36     # logits so large that one takes all
    x[5] = -torch.rand(V, generator=g) * 1e36 - 1e37
    x = x.to(TYPES[dtype])
    tok = torch.tensor([5, 1, 7, 4500, 11, 13], dtype=torch.int32)
    for n in (0, 6):
        _check(x.to(DEV), tok, torch.tensor([1.0, 1.0, 0.5, 1.0, 1.0, 1.0]), n)

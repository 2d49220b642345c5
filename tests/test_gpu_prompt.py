"""GPU: causal attention over packed prompts and its gradient against the float64 oracle.

Tolerances, from the arithmetic in include/spec_prompt.h (u = 2^-24; sums on the tensor cores may be
truncated: n terms are off by 2 n u of their absolute sum). With A the largest scale * sum |q_d k_d| of
the keys that a row sees, a logit is off by 2 (D + 8) u A and its exponential, formed in base 2, by
8 u (1.45 (A + |lse|) + 8) + 2^-21 more: d together, of itself. Weights are rounded to bf16 (2^-8) for the
products, and the result is rounded to bf16 (2^-8):
  |out - ref|  <= (2^-8 + 2 d + 2 n u) sum P |v| + 2^-8 |ref|,      |lse - ref| <= d + (n + 80) u + 4 u |lse|
  |grad_v - ref| <= (2^-8 + d + 2 n u) sum P |go| + 2^-8 |ref|
dP and delta are off by 2 (D + 8) u of their absolute sums, e together; dS by P e + (d + 4 u) (P (|dP| + |delta|))
and 2^-8 |dS| by its rounding; its sums with k and q as above. n: keys or rows that are summed."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_30_gb300 as sv
from oracle import prompt as op

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF = torch.bfloat16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(lens, heads, kv_heads, dim, seed=0, gain=1.0, before=0, behind=0):
    """qkv [N, heads + 2 kv_heads, dim] bf16 on the host, and cu."""
    g = torch.Generator().manual_seed(seed)
    N = before + sum(lens) + behind
    qkv = torch.randn(max(N, 1), heads + 2 * kv_heads, dim, generator=g)
    qkv[:, :heads + kv_heads] *= gain
    return qkv.to(BF), np.concatenate([[before], before + np.cumsum(lens)]).astype(np.int32)


def _errors(q, k, lse, a, e, h, y, see, scale, D):
    """Logits and d (a factor for each row) of head h of rows a .. e - 1."""
    z = q[a:e, h] @ k[a:e, y].T * scale
    A = np.where(see, np.abs(q[a:e, h]) @ np.abs(k[a:e, y]).T * scale, 0).max(1, keepdims=True)
    d = 2 * (D + 8) * U * A + 8 * U * (1.45 * (A + np.abs(lse[a:e, h, None])) + 8) + 2.0 ** -21
    return z, d


def check_forward(out, lse, q, k, v, cu, scale, window):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ref, ref_lse = op.attend(q, k, v, cu, scale, window)
    N, H, D = q.shape
    G = H // k.shape[1]
    inside = np.zeros(N, bool)
    for a, e in op.sequences(cu, N):
        inside[a:e] = True
        see = op.seen(e - a, window)
        n = see.sum(1, keepdims=True)
        for h in range(H):
            z, d = _errors(q, k, ref_lse, a, e, h, h // G, see, scale, D)
            p = np.where(see, np.exp(np.where(see, z, 0) - ref_lse[a:e, h, None]), 0)
            tol = (2.0 ** -8 + 2 * d + 2 * n * U) * (p @ np.abs(v[a:e, h // G])) + 2.0 ** -8 * np.abs(ref[a:e, h]) + 1e-30
            err = np.abs(out[a:e, h] - ref[a:e, h])
            assert (err <= tol).all(), (a, e, h, float((err / tol).max()), np.argwhere(~(err <= tol))[:4].tolist())
            t2 = d[:, 0] + (n[:, 0] + 80) * U + 4 * U * np.abs(ref_lse[a:e, h])
            assert (np.abs(lse[a:e, h] - ref_lse[a:e, h]) <= t2).all(), (a, e, h)
    assert (out[~inside] == 0).all() and (lse[~inside] == -np.inf).all()
    return ref, ref_lse


def check_backward(grads, go, q, k, v, out, lse, cu, scale, window):
    gq, gk, gv = (g.double().cpu().numpy() for g in grads)
    rq, rk, rv = op.gradient(go, q, k, v, out, lse, cu, scale, window)
    N, H, D = q.shape
    G = H // k.shape[1]
    tq, tk, tv = (2.0 ** -8 * np.abs(r) + 1e-30 for r in (rq, rk, rv))
    for a, e in op.sequences(cu, N):
        see = op.seen(e - a, window)
        n, rows = see.sum(1, keepdims=True), G * see.sum(0)[:, None]
        for h in range(H):
            y = h // G
            z, d = _errors(q, k, lse, a, e, h, y, see, scale, D)
            p = np.where(see, np.exp(np.where(see, z, 0) - lse[a:e, h, None]), 0)
            dp, ab = go[a:e, h] @ v[a:e, y].T, np.abs(go[a:e, h]) @ np.abs(v[a:e, y]).T
            delta = (go[a:e, h] * out[a:e, h]).sum(1, keepdims=True)
            size = (np.abs(go[a:e, h]) * np.abs(out[a:e, h])).sum(1, keepdims=True)
            ds = p * np.abs(dp - delta)
            off = p * 2 * (D + 8) * U * (ab + size) + (d + 4 * U) * p * (np.abs(dp) + np.abs(delta)) + 2.0 ** -8 * ds
            tq[a:e, h] += scale * ((off + 2 * n * U * ds) @ np.abs(k[a:e, y]))
            tk[a:e, y] += scale * ((off.T + 2 * rows * U * ds.T) @ np.abs(q[a:e, h]))
            tv[a:e, y] += ((2.0 ** -8 + d) * p).T @ np.abs(go[a:e, h]) + 2 * rows * U * (p.T @ np.abs(go[a:e, h]))
    for name, got, ref, tol in (("q", gq, rq, tq), ("k", gk, rk, tk), ("v", gv, rv, tv)):
        err = np.abs(got - ref)
        assert (err <= tol).all(), (name, float((err / tol).max()), np.argwhere(~(err <= tol))[:4].tolist())


def check(lens, heads, kv_heads, dim, window=0, seed=0, scale=None, gain=1.0, packed=True, before=0, behind=0, backward=True):
    qkv, cu = make(lens, heads, kv_heads, dim, seed, gain, before, behind)
    scale = dim ** -0.5 if scale is None else scale
    dev = qkv.to(DEV).split([heads, kv_heads, kv_heads], 1)
    if not packed:
        dev = [x.contiguous() for x in dev]
    host = [x.double().numpy() for x in qkv.split([heads, kv_heads, kv_heads], 1)]
    cud = _i32(cu.tolist())
    out, lse = sv.spec_prompt_attention(*dev, cud, scale=scale, window=window)
    again = sv.spec_prompt_attention(*dev, cud, scale=scale, window=window)
    torch.cuda.synchronize()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    ref, ref_lse = check_forward(out, lse, *host, cu, scale, window)
    if not backward:
        return
    g = torch.Generator().manual_seed(seed + 1)
    go = torch.randn(qkv.shape[0], heads, dim, generator=g).to(BF)
    ob, lb = torch.from_numpy(ref).to(BF), torch.from_numpy(ref_lse).float()
    args = (go.to(DEV), *dev, ob.to(DEV), lb.to(DEV), cud)
    grads = sv.spec_prompt_attention_backward(*args, scale=scale, window=window)
    again = sv.spec_prompt_attention_backward(*args, scale=scale, window=window)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(grads, again))
    check_backward(grads, go.double().numpy(), *host, ob.double().numpy(), lb.double().numpy(), cu, scale, window)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (2, 2), (4, 2), (3, 1), (7, 1), (8, 1)])
def test_lengths_around_the_tiles(heads, kv_heads, dim):
    check([1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257], heads, kv_heads, dim, seed=heads + dim)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 300])
def test_sliding_windows(window, dim):
    check([1, 130, 400, 513], 2, 1, dim, window=window, seed=window)
    check([300], 3, 3, dim, window=window, seed=window + 1)


@pytest.mark.parametrize("dim", [64, 128])
def test_longer_prompts(dim):
    check([1500, 3, 800], 2, 1, dim, seed=dim, packed=False)
    check([1030], 1, 1, dim, seed=dim + 1, window=700)


@pytest.mark.parametrize("before,behind", [(3, 0), (0, 5), (130, 200)])
def test_rows_outside_every_sequence(before, behind):
    check([5, 0, 130, 0, 0, 64], 4, 2, 64, before=before, behind=behind, seed=7)
    check([40, 0], 2, 2, 128, before=before, behind=behind, seed=8)


@pytest.mark.parametrize("window", [1 << 20, (1 << 31) - 2, (1 << 31) - 1])
def test_windows_longer_than_every_prompt(window):
    qkv, cu = make([130, 300], 2, 1, 64, seed=30)
    q, k, v = qkv.to(DEV).split([2, 1, 1], 1)
    cud = _i32(cu.tolist())
    a, b = (sv.spec_prompt_attention(q, k, v, cud, window=w) for w in (0, window))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = (sv.spec_prompt_attention_backward(a[0], q, k, v, *a, cud, window=w) for w in (0, window))
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))


def test_no_rows_at_all():
    qkv, _ = make([], 4, 2, 64, behind=10)
    q, k, v = qkv.to(DEV).split([4, 2, 2], 1)
    for cu in ([0, 0], [10, 10], [4, 4, 4], [0, -3], [50, 60]):
        out, lse = sv.spec_prompt_attention(q, k, v, _i32(cu))
        assert (out == 0).all() and (lse == -float("inf")).all()
        g = sv.spec_prompt_attention_backward(torch.ones_like(out), q, k, v, out, lse, _i32(cu))
        assert all((x == 0).all() for x in g)


def test_many_short_sequences():
    r = np.random.default_rng(0)
    check(r.integers(0, 12, 400).tolist(), 2, 1, 64, seed=9)
    check([1] * 300, 4, 4, 128, seed=10)


@pytest.mark.parametrize("gain,scale", [(30.0, None), (1e-18, 1e36), (1.0, 0.0), (1e15, 1e-31), (5.0, 0.3)])
def test_magnitudes(gain, scale):
    check([200, 17], 2, 1, 64, gain=gain, scale=scale, seed=11)
    check([140], 2, 2, 128, gain=gain, scale=scale, seed=12, backward=gain < 1e10)


def test_a_running_maximum_that_keeps_rising():
    # keys that grow along the prompt, so that every block of keys moves the frame
    qkv, cu = make([700], 2, 1, 64, seed=13)
    qkv[:, :2] = qkv[:, :2].abs()
    qkv[:, 2] = (torch.linspace(0, 12, 700)[:, None] * torch.ones(64)).to(BF)
    q, k, v = qkv.to(DEV).split([2, 1, 1], 1)
    out, lse = sv.spec_prompt_attention(q, k, v, _i32(cu.tolist()))
    host = [x.double().numpy() for x in qkv.split([2, 1, 1], 1)]
    check_forward(out, lse, *host, cu, 64 ** -0.5, 0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("part", ["q", "k", "v"])
@pytest.mark.parametrize("dim", [64, 128])
def test_what_is_not_finite_reaches_only_rows_that_see_it(part, bad, dim):
    lens, heads, kv = [150, 90, 40], 4, 2
    qkv, cu = make(lens, heads, kv, dim, seed=14)
    clean = qkv.to(DEV).split([heads, kv, kv], 1)
    ref, ref_lse = sv.spec_prompt_attention(*clean, _i32(cu.tolist()))
    for at in (60, 149, 150, 239, 240, 279):          # inside, and at the ends of sequences
        x = qkv.clone()
        x[at, {"q": 1, "k": heads, "v": heads + kv}[part], 5] = bad
        out, lse = sv.spec_prompt_attention(*x.to(DEV).split([heads, kv, kv], 1), _i32(cu.tolist()))
        end = next(int(e) for e in cu[1:] if at < e)
        if part == "q":
            hit = torch.zeros(len(x), heads, dtype=torch.bool)
            hit[at, 1] = True
        else:
            hit = torch.zeros(len(x), heads, dtype=torch.bool)
            hit[at:end, :2] = True
        clean_rows = ~hit.to(DEV)
        assert torch.equal(out[clean_rows], ref[clean_rows]) and torch.equal(lse[clean_rows], ref_lse[clean_rows])
        if part == "v":
            assert not torch.isfinite(out[..., 5][~clean_rows]).any()
            others = [d for d in range(dim) if d != 5]
            assert torch.equal(out[..., others], ref[..., others]) and torch.equal(lse, ref_lse)
        elif np.isnan(bad):
            assert torch.isnan(out[~clean_rows]).all() and torch.isnan(lse[~clean_rows]).all()


@pytest.mark.parametrize("part", ["q", "k", "v", "go", "out"])
@pytest.mark.parametrize("dim", [64, 128])
def test_what_is_not_finite_reaches_no_other_sequence_s_gradient(part, dim):
    lens, heads, kv = [150, 90, 40], 2, 1
    qkv, cu = make(lens, heads, kv, dim, seed=15)
    g = torch.Generator().manual_seed(1)
    go = torch.randn(qkv.shape[0], heads, dim, generator=g).to(BF).to(DEV)
    cud = _i32(cu.tolist())
    dev = [x.contiguous() for x in qkv.to(DEV).split([heads, kv, kv], 1)]
    out, lse = sv.spec_prompt_attention(*dev, cud)
    ref = sv.spec_prompt_attention_backward(go, *dev, out, lse, cud)
    for at in (149, 150, 239, 240):
        args = dict(zip(("go", "q", "k", "v", "out", "lse"), [x.clone() for x in (go, *dev, out, lse)]))
        args[part][at, 0, 7] = float("nan")
        got = sv.spec_prompt_attention_backward(*args.values(), cud)
        mine = np.zeros(len(qkv), bool)
        for a, e in op.sequences(cu, len(qkv)):
            mine[a:e] = a <= at < e
        other = torch.from_numpy(~mine).to(DEV)
        assert all(torch.equal(x[other], y[other]) for x, y in zip(got, ref))


def test_autograd():
    lens, heads, kv, dim = [70, 1, 200], 4, 2, 64
    qkv, cu = make(lens, heads, kv, dim, seed=16, behind=4)
    x = qkv.to(DEV).requires_grad_()
    q, k, v = x.split([heads, kv, kv], 1)
    out, lse = sv.spec_prompt_attention(q, k, v, _i32(cu.tolist()))
    assert out.requires_grad
    w = torch.randn(out.shape, generator=torch.Generator().manual_seed(2)).to(DEV).to(BF)
    (out * w).sum().backward()
    plain = [t.detach() for t in (q, k, v)]
    o2, l2 = sv.spec_prompt_attention(*plain, _i32(cu.tolist()))
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    ref = sv.spec_prompt_attention_backward(w, *plain, o2, l2, _i32(cu.tolist()))
    assert torch.equal(x.grad, torch.cat(ref, 1)) and (x.grad[-4:] == 0).all()
    # only the values, and a gradient that is one number, expanded
    v2 = plain[2].clone().requires_grad_()
    sv.spec_prompt_attention(plain[0], plain[1], v2, _i32(cu.tolist()))[0].sum().backward()
    ref = sv.spec_prompt_attention_backward(torch.ones_like(w), *plain, o2, l2, _i32(cu.tolist()))
    assert torch.equal(v2.grad, ref[2])
    # one tensor as keys and values: both gradients arrive
    kk = plain[1].clone().requires_grad_()
    o3, l3 = sv.spec_prompt_attention(plain[0], kk, kk, _i32(cu.tolist()))
    (o3 * w).sum().backward()
    ref = sv.spec_prompt_attention_backward(w, plain[0], plain[1], plain[1], o3.detach(), l3.detach(), _i32(cu.tolist()))
    assert torch.equal(kk.grad, ref[1] + ref[2])


def test_gradient_along_a_direction_against_differences():
    # loss(x + h t) - loss(x - h t) of the oracle; the kernel's gradients are within its tolerance of the
    # formula's, so their products with t are within that times |t|
    lens, heads, kv, dim = [50, 90], 2, 1, 64
    qkv, cu = make(lens, heads, kv, dim, seed=17)
    parts = [x.double().numpy() for x in qkv.split([heads, kv, kv], 1)]
    g = torch.Generator().manual_seed(3)
    go = torch.randn(qkv.shape[0], heads, dim, generator=g).to(BF)
    x = [t.contiguous().to(DEV).requires_grad_() for t in qkv.split([heads, kv, kv], 1)]
    out, _ = sv.spec_prompt_attention(*x, _i32(cu.tolist()))
    (out * go.to(DEV)).sum().backward()
    r, h = np.random.default_rng(4), 1e-5
    for i in range(3):
        t = np.sign(r.normal(size=parts[i].shape))
        f = []
        for s in (h, -h):
            y = list(parts)
            y[i] = parts[i] + s * t
            f.append((op.attend(*y, cu, dim ** -0.5)[0] * go.double().numpy()).sum())
        got = x[i].grad.double().cpu().numpy()
        # each element to 2^-8 of itself and, by the sums over rounded weights, of the terms' size: random in
        # sign, so that their sum over n elements grows as sqrt(n) (six of them)
        assert abs((got * t).sum() - (f[0] - f[1]) / (2 * h)) <= 6 * 2.0 ** -7 * np.sqrt((got ** 2).sum()) + 1e-3, i


def test_what_has_no_gradient_is_refused():
    qkv, cu = make([20], 2, 1, 64, seed=18)
    q, k, v = (t.contiguous().to(DEV) for t in qkv.split([2, 1, 1], 1))
    cud = _i32(cu.tolist())
    q.requires_grad_()
    out, lse = sv.spec_prompt_attention(q, k, v, cud)
    with pytest.raises(sv.SpecVerifyError):
        (out.sum() + lse.sum()).backward()
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_prompt_attention(q, k, v, cud, out=torch.empty_like(q))
    with torch.no_grad():
        given = torch.empty_like(k.expand(-1, 2, -1).contiguous())
        o, _ = sv.spec_prompt_attention(q, k, v, cud, out=given)
    assert o is given and torch.equal(o, out.detach())
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_prompt_attention(fwd.make_dual(q.detach(), torch.ones_like(q)), k, v, cud)


def test_refusals():
    qkv, cu = make([20], 2, 1, 64, seed=19)
    q, k, v = (t.contiguous().to(DEV) for t in qkv.split([2, 1, 1], 1))
    cud = _i32(cu.tolist())
    o, lse = sv.spec_prompt_attention(q, k, v, cud)
    bad = [(q.float(), k, v, cud), (q, k.half(), v, cud), (q, k[:10], v, cud), (q, k, v.expand(-1, 2, -1), cud), (q, k, v, cud.long()),
           (q, k, v, cud.cpu()), (q.cpu(), k, v, cud), (q[..., :32], k[..., :32], v[..., :32], cud), (q, k, v, cud[:1]),
           (q.transpose(0, 1), k, v, cud), (k.expand(-1, 3, -1), k, v, cud), (q, k.repeat(1, 4, 1), v.repeat(1, 4, 1), cud),
           (q[:0], k[:0], v[:0], cud)]
    for args in bad:
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_prompt_attention(*args)
    for kw in (dict(window=-1), dict(window=1 << 31), dict(window=1.5), dict(scale=float("nan")), dict(scale=-1.0), dict(scale="1"),
               dict(out=o.float()), dict(out=o[:5]), dict(lse=lse.double()), dict(lse=lse[:5])):
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_prompt_attention(q, k, v, cud, **kw)
    for args in ((o[:5], q, k, v, o, lse, cud), (o, q, k, v, o[:, :1], lse, cud), (o, q, k, v, o, lse.T, cud), (o.float(), q, k, v, o, lse, cud)):
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_prompt_attention_backward(*args)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_prompt_attention_backward(o, q, k, v, o, lse, cud, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_captured_and_replayed_with_other_lengths():
    lens, heads, kv, dim = [90, 40, 130], 4, 2, 128
    qkv, cu = make(lens, heads, kv, dim, seed=20)
    q, k, v = qkv.to(DEV).split([heads, kv, kv], 1)
    cud, go = _i32(cu.tolist()), torch.randn(qkv.shape[0], heads, dim, device=DEV).to(BF)

    def both():
        o, l = sv.spec_prompt_attention(q, k, v, cud)
        return (o, l, *sv.spec_prompt_attention_backward(go, q, k, v, o, l, cud))
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    for other in ([0, 90, 130, 260], [0, 1, 259, 260], [5, 100, 100, 240]):
        cud.copy_(_i32(other))
        graph.replay()
        got = [x.clone() for x in kept]
        assert all(torch.equal(x, y) for x, y in zip(got, both())), other


def test_two_streams_at_once_and_a_side_stream():
    qkv, cu = make([300, 200], 4, 2, 64, seed=21)
    q, k, v = qkv.to(DEV).split([4, 2, 2], 1)
    cud = _i32(cu.tolist())
    ref = sv.spec_prompt_attention(q, k, v, cud)
    go = torch.randn_like(ref[0])
    gref = sv.spec_prompt_attention_backward(go, q, k, v, *ref, cud)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [(sv.spec_prompt_attention(q, k, v, cud, stream=s), sv.spec_prompt_attention_backward(go, q, k, v, *ref, cud, stream=s))
           for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    for f, b in got:
        assert torch.equal(f[0], ref[0]) and torch.equal(f[1], ref[1]) and all(torch.equal(x, y) for x, y in zip(b, gref))
    x = [t.contiguous().requires_grad_() for t in (q, k, v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, _ = sv.spec_prompt_attention(*x, cud, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    (out * go).sum().backward()
    assert all(torch.equal(t.grad, y) for t, y in zip(x, gref))


@pytest.mark.parametrize("dim,heads,kv_heads,window", [(128, 8, 2, 0), (64, 3, 1, 0), (64, 4, 4, 900)])
def test_a_long_prompt_against_64_bits_on_the_device(dim, heads, kv_heads, window):
    # rows spread over a prompt of 9,000 tokens, formed in float64 on the device; tolerances as above with
    # |q . k| in the place of the sums of absolute products (which it bounds to a factor of 8 here: d times 8)
    T = 9000
    qkv, cu = make([17, T], heads, kv_heads, dim, seed=22)
    x = qkv.to(DEV)
    q, k, v = x.split([heads, kv_heads, kv_heads], 1)
    out, lse = sv.spec_prompt_attention(q, k, v, _i32(cu.tolist()), window=window)
    at = torch.tensor(sorted({17 + i for i in (0, 1, 127, 128, 4095, 4096, 8191, 8192, 8959, 8960, T - 1)}), device=DEV)
    j = torch.arange(17, 17 + T, device=DEV)
    for h in range(heads):
        y = h // (heads // kv_heads)
        z = q[at, h].double() @ k[17:, y].double().T * dim ** -0.5
        see = j <= at[:, None]
        if window:
            see &= j > at[:, None] - window
        z = z.masked_fill(~see, -float("inf"))
        m = torch.logsumexp(z, 1)
        p = (z - m[:, None]).exp()
        ref, size = p @ v[17:, y].double(), p @ v[17:, y].double().abs()
        A = 8 * z.masked_fill(~see, 0).abs().amax(1, keepdim=True)
        d = 2 * (dim + 8) * U * A + 8 * U * (1.45 * (A + m.abs()[:, None]) + 8) + 2.0 ** -21
        assert ((out[at, h].double() - ref).abs() <= (2.0 ** -8 + 2 * d + 2 * T * U) * size + 2.0 ** -8 * ref.abs()).all()
        assert ((lse[at, h].double() - m).abs() <= d[:, 0] + (T + 80) * U + 4 * U * m.abs()).all()


@pytest.mark.parametrize("heads,kv_heads,dim", [(64, 1, 64), (126, 2, 128), (256, 256, 64), (192, 64, 128)])
def test_many_heads(heads, kv_heads, dim):
    check([40, 1, 150], heads, kv_heads, dim, seed=31, window=0 if heads < 200 else 30)


def test_offsets_past_32_bits():
    # queries, results and gradients of 2.3e9 elements: rows at both ends against float64 on the device, with the
    # tolerances of the header (a row sees 100 keys; the keys' last row is seen by one query of each of 64 heads)
    T, H, kv, D, W = 70_000, 256, 4, 128, 100
    g = torch.Generator(device=DEV).manual_seed(32)

    def rnd(heads):
        return torch.randn(T, heads, D, generator=g, device=DEV, dtype=BF)
    q, k, v, go = rnd(H), rnd(kv), rnd(kv), rnd(H)
    cu, c = _i32([0, T]), D ** -0.5
    out, lse = sv.spec_prompt_attention(q, k, v, cu, window=W)
    gq, gk, gv = sv.spec_prompt_attention_backward(go, q, k, v, out, lse, cu, window=W)

    def d_of(A, m):
        return 2 * (D + 8) * U * A + 8 * U * (1.45 * (A + abs(m)) + 8) + 2.0 ** -21

    def ds_of(p, d, q, k, v, go, o):
        """dS and how far it may be off, of pairs in rows."""
        dp, ab = (go * v).sum(-1), (go * v).abs().sum(-1)
        delta, size = (go * o).sum(-1), (go * o).abs().sum(-1)
        ds = p * (dp - delta)
        return ds, p * 2 * (D + 8) * U * (ab + size) + (d + 4 * U) * p * (dp.abs() + delta.abs()) + 2.0 ** -8 * ds.abs()
    for r in (3, T // 2, T - 1):
        for h in (0, H - 1):
            a = max(0, r - W + 1)
            n = r + 1 - a
            kk, vv, x, y, o = (t.double() for t in (k[a:r + 1, h // 64], v[a:r + 1, h // 64], q[r, h], go[r, h], out[r, h]))
            z = kk @ x * c
            m = float(torch.logsumexp(z, 0))
            d = d_of(float((kk.abs() @ x.abs()).max()) * c, m)
            p = torch.softmax(z, 0)
            ref = p @ vv
            assert ((o - ref).abs() <= (2.0 ** -8 + 2 * d + 2 * n * U) * (p @ vv.abs()) + 2.0 ** -8 * ref.abs()).all()
            assert abs(float(lse[r, h]) - m) <= d + (n + 80) * U + 4 * U * abs(m)
            # the gradient starts from the call's own lse, which is off by as much again
            ds, off = ds_of(p, 2 * d + (n + 80) * U, x, kk, vv, y, o)
            ref = ds @ kk * c
            tol = c * ((off + 2 * n * U * ds.abs()) @ kk.abs()) + 2.0 ** -8 * ref.abs()
            assert ((gq[r, h].double() - ref).abs() <= tol).all()
    r, y, hs = T - 1, kv - 1, slice(H - 64, H)
    x, w, o, kk, vv = q[r, hs].double(), go[r, hs].double(), out[r, hs].double(), k[r, y].double(), v[r, y].double()
    p = torch.exp(x @ kk * c - lse[r, hs].double())
    d = d_of(float((x.abs() @ kk.abs()).max()) * c, float(lse[r, hs].abs().max()))
    ref = p @ w
    assert ((gv[r, y].double() - ref).abs() <= (2.0 ** -8 + d + 128 * U) * (p @ w.abs()) + 2.0 ** -8 * ref.abs()).all()
    ds, off = ds_of(p, d, x, kk, vv, w, o)
    ref = ds @ x * c
    assert ((gk[r, y].double() - ref).abs() <= c * ((off + 128 * U * ds.abs()) @ x.abs()) + 2.0 ** -8 * ref.abs()).all()

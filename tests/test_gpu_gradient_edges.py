"""GPU: what has a gradient, what refuses one, and a forward pass on another stream than its
backward pass."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import speculative_decoding_verification_30_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda"
E = sv.SpecVerifyError


def _rows():
    g = torch.Generator().manual_seed(1)
    return torch.randn(4, 500, generator=g).to(DEV), torch.tensor([1, 2, -1, 499], dtype=torch.int32, device=DEV)


def test_a_temperature_that_requires_a_gradient_is_refused():
    x, tok = _rows()
    temp = torch.ones(4, device=DEV, requires_grad=True)
    for logits in (x, x.clone().requires_grad_()):
        with pytest.raises(E):
            sv.spec_token_logprobs(logits, tok, temp)
    with torch.no_grad():
        r = sv.spec_token_logprobs(x, tok, temp)
    ref = sv.spec_token_logprobs(x, tok, temp.detach())
    assert all(torch.equal(a, b) for a, b in zip(r, ref))


def test_forward_mode_tangents_are_refused():
    x, tok = _rows()
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        with pytest.raises(E):
            sv.spec_token_logprobs(dual, tok)
        with pytest.raises(E):
            sv.spec_token_logprobs(x, tok, fwd.make_dual(torch.ones(4, device=DEV), torch.ones(4, device=DEV)))
        ok = sv.spec_token_logprobs(x, tok)
    assert torch.equal(ok.logprob, sv.spec_token_logprobs(x, tok).logprob)


def test_a_loss_on_lse_is_refused_not_lost():
    x, tok = _rows()
    x.requires_grad_()
    r = sv.spec_token_logprobs(x, tok)
    with pytest.raises(E):
        (r.logprob.sum() + r.lse.square().sum()).backward()
    r = sv.spec_token_logprobs(x, tok)
    (r.logprob.sum() + r.lse.detach().square().sum()).backward()
    assert torch.isfinite(x.grad).all()


@pytest.mark.parametrize("n", [0, 5])
def test_forward_on_a_side_stream(n):
    x, tok = _rows()
    ref = x.clone().requires_grad_()
    r = sv.spec_token_logprobs(ref, tok, top_n=n)
    (r.logprob.sum() + r.entropy.sum()).backward()
    side = torch.cuda.Stream()
    for _ in range(3):
        y = x.clone().requires_grad_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                  # the side stream is some milliseconds behind
        r = sv.spec_token_logprobs(y, tok, top_n=n, stream=side)
        one = torch.ones(4, device=DEV)
        d, = torch.autograd.grad([r.logprob, r.entropy], y, [one, one])
        del r
        # memory of the forward's outputs must not be handed out before the gradient has read it
        with torch.cuda.stream(side):
            junk = [torch.full((4,), float("nan"), device=DEV) for _ in range(8)]
        assert torch.equal(d, ref.grad)
        del junk


def test_a_graph_that_saved_what_a_call_writes_over_raises():
    x, tok = _rows()
    x = (x * 1.0).requires_grad_()
    r = sv.spec_token_logprobs(x, tok)
    one = torch.ones(4, device=DEV)
    d = x.detach()                                         # the same memory
    sv.spec_token_logprobs_backward(d, tok, r.lse.detach(), r.entropy.detach(), grad_logprob=one, out=d)
    with pytest.raises(RuntimeError, match="inplace"):
        r.logprob.sum().backward()

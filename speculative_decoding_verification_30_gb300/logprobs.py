"""Log-probabilities of given tokens over logit rows, with entropy and top alternatives,
and their gradient (include/spec_logprobs.h)."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import SpecVerifyError, _check, _dtype_code, load
from ._launch import no_tangent, on_device, ptr, wrote


class TokenLogprobs(NamedTuple):
    """Outputs of spec_token_logprobs; the leading shape is that of the tokens."""
    logprob: torch.Tensor        # float32
    rank: torch.Tensor           # int32: 0 is the argmax
    entropy: torch.Tensor        # float32, nats
    lse: torch.Tensor            # float32: ln sum exp(logits / temperature)
    top_ids: torch.Tensor        # int32 [..., top_n]
    top_logprobs: torch.Tensor   # float32 [..., top_n]


def _rows(x: torch.Tensor, name: str):
    """(R, V, row stride) of logit rows [..., V]."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise SpecVerifyError(f"{name} must be a CUDA tensor")
    V = x.shape[-1] if x.dim() else 0
    if x.dim() < 2 or (x.stride(-1) != 1 and V > 1):
        raise SpecVerifyError(f"{name} must be [..., V] with adjacent logits")
    if x.is_contiguous():
        return x.numel() // max(V, 1), V, V
    try:
        flat = x.view(-1, V)
    except RuntimeError:
        raise SpecVerifyError(f"{name}: the rows must have one stride") from None
    return flat.shape[0], V, flat.stride(0) if flat.shape[0] > 1 else V


def _per_row(t, name: str, dtype, R: int, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.numel() != R:
        raise SpecVerifyError(f"{name} must have one value for each row")
    return ptr(t, name, dtype, device)


def _forward(logits, tokens, temperature, top_n, stream):
    R, V, ld = _rows(logits, "logits")
    dev, lead = logits.device, tokens.shape
    if R == 0:
        raise SpecVerifyError("logits must have at least one row")
    tok = _per_row(tokens, "tokens", torch.int32, R, dev)
    temp = _per_row(temperature, "temperature", torch.float32, R, dev)
    with on_device(dev, stream, logits, tokens, temperature) as st:
        logprob = torch.empty(lead, dtype=torch.float32, device=dev)
        entropy = torch.empty(lead, dtype=torch.float32, device=dev)
        lse = torch.empty(lead, dtype=torch.float32, device=dev)
        rank = torch.empty(lead, dtype=torch.int32, device=dev)
        ids = torch.empty((*lead, top_n), dtype=torch.int32, device=dev)
        lps = torch.empty((*lead, top_n), dtype=torch.float32, device=dev)
        rc = load().spec_token_logprobs(logits.data_ptr(), _dtype_code(logits), R, V, ld, tok, temp, top_n,
                                        logprob.data_ptr(), rank.data_ptr(), entropy.data_ptr(), lse.data_ptr(),
                                        ids.data_ptr(), lps.data_ptr(), st)
    if rc:
        _check(rc, "spec_token_logprobs")
    return TokenLogprobs(logprob, rank, entropy, lse, ids, lps)


class _Function(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature, top_n, stream):
        r = _forward(logits, tokens, temperature, top_n, stream)
        ctx.save_for_backward(logits, tokens, temperature, r.lse, r.entropy, r.top_ids)
        ctx.done = None if stream is None else stream.record_event()
        ctx.mark_non_differentiable(r.rank, r.top_ids)
        ctx.set_materialize_grads(False)
        return tuple(r)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_lp, _rank, g_h, g_lse, _ids, g_top):
        if g_lse is not None:
            raise SpecVerifyError("lse has no gradient: use it detached in a loss")
        logits, tokens, temperature, lse, entropy, ids = ctx.saved_tensors
        if g_lp is None and g_h is None and g_top is None:
            return None, None, None, None, None
        if ctx.done is not None:
            # The forward pass ran on a stream of its own: this one comes after it, and the
            # allocator learns that what it left is in use here.
            here = torch.cuda.current_stream(logits.device)
            here.wait_event(ctx.done)
            for t in (logits, tokens, temperature, lse, entropy, ids):
                if t is not None:
                    t.record_stream(here)
        g = [None if t is None else t.contiguous() for t in (g_lp, g_h, g_top)]
        d = spec_token_logprobs_backward(logits, tokens, lse, entropy, temperature, g[0], g[1],
                                         ids if g[2] is not None else None, g[2])
        return d, None, None, None, None


def spec_token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, temperature: torch.Tensor | None = None,
                        top_n: int = 0, stream=None) -> TokenLogprobs:
    """Log-probability, rank, entropy and the top_n alternatives (0..32) of `tokens` [...]
    (int32) in the logit rows [..., V] (bf16 or fp32; the rows may have a stride, or be one
    row, expanded).

    `temperature` [...] (float32) divides the logits; 0 counts as 1. A row whose token
    is negative is skipped (outputs 0, rank and ids -1), so the out_tokens of
    spec_verify can be scored as they are. Data errors give NaN with rank and ids -1.
    When logits.requires_grad, logprob, entropy and top_logprobs are differentiable with
    respect to them. A temperature that requires a gradient is refused, and so is a backward
    pass through lse."""
    if not isinstance(tokens, torch.Tensor):
        raise SpecVerifyError("tokens must be a CUDA tensor")
    if not isinstance(top_n, int) or not 0 <= top_n <= 32:
        raise SpecVerifyError("top_n must be 0..32")
    no_tangent("spec_token_logprobs", logits, temperature)
    if torch.is_grad_enabled() and getattr(temperature, "requires_grad", False):
        raise SpecVerifyError("the temperature has no gradient: pass it detached")
    if isinstance(logits, torch.Tensor) and logits.requires_grad and torch.is_grad_enabled():
        return TokenLogprobs(*_Function.apply(logits, tokens, temperature, top_n, stream))
    return _forward(logits, tokens, temperature, top_n, stream)


def spec_token_logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor, lse: torch.Tensor,
                                 entropy: torch.Tensor, temperature: torch.Tensor | None = None,
                                 grad_logprob: torch.Tensor | None = None,
                                 grad_entropy: torch.Tensor | None = None, top_ids: torch.Tensor | None = None,
                                 grad_top: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                 stream=None) -> torch.Tensor:
    """Gradient with respect to the logits, in their type and shape, from the gradients with
    respect to logprob, entropy and top_logprobs. `lse`, `entropy` and `top_ids` are
    spec_token_logprobs's; `out` may be the logits themselves."""
    R, V, ld = _rows(logits, "logits")
    dev = logits.device
    if R == 0:
        raise SpecVerifyError("logits must have at least one row")
    if tokens is None or lse is None or entropy is None:
        raise SpecVerifyError("tokens, lse and entropy are required")
    args = [_per_row(tokens, "tokens", torch.int32, R, dev), _per_row(temperature, "temperature", torch.float32, R, dev),
            _per_row(lse, "lse", torch.float32, R, dev), _per_row(entropy, "entropy", torch.float32, R, dev),
            _per_row(grad_logprob, "grad_logprob", torch.float32, R, dev),
            _per_row(grad_entropy, "grad_entropy", torch.float32, R, dev)]
    n, ids, gt = 0, None, None
    if grad_top is not None:
        if top_ids is None or top_ids.shape != grad_top.shape or grad_top.numel() != R * grad_top.shape[-1]:
            raise SpecVerifyError("top_ids and grad_top must be [..., top_n]")
        n, ids, gt = (grad_top.shape[-1], ptr(top_ids, "top_ids", torch.int32, dev),
                      ptr(grad_top, "grad_top", torch.float32, dev))
    with on_device(dev, stream, logits, tokens, temperature, lse, entropy, grad_logprob, grad_entropy, top_ids,
                   grad_top, out) as st:
        given = out
        if out is None:
            out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        elif out.shape != logits.shape or out.dtype != logits.dtype or out.device != dev:
            raise SpecVerifyError("out must have the logits' shape, type and device")
        gld = _rows(out, "out")[2]
        rc = load().spec_token_logprobs_backward(logits.data_ptr(), _dtype_code(logits), R, V, ld, *args, n, ids, gt,
                                                 out.data_ptr(), gld, st)
    if rc:
        _check(rc, "spec_token_logprobs_backward")
    if given is not None:
        wrote(given)
    return out

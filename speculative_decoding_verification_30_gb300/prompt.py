"""Causal attention over packed prompts, with grouped heads, and its gradient
(include/spec_prompt.h)."""
from __future__ import annotations

import torch

from . import SpecVerifyError, _check, load
from ._launch import no_tangent, on_device, ptr, wrote
from .kv import _I32, _heads, _shape, _whole

_BF16 = torch.bfloat16


def _inputs(q, k, v, cu_tokens, scale, window):
    """Device, head_dim, the pointers and strides of q, k and v, and (cu, B, N, q_heads, kv_heads, head_dim, scale, window)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise SpecVerifyError("q must be a CUDA tensor")
    dev = q.device
    if q.dim() != 3 or q.shape[2] not in (64, 128):
        raise SpecVerifyError("q must be [N, q_heads, head_dim] with head_dim 64 or 128")
    dim = q.shape[2]
    qp, qs, N, qh = _heads(q, "q", _BF16, dev, dim)
    kp, ks, kn, kh = _heads(k, "k", _BF16, dev, dim)
    vp, vs, vn, vh = _heads(v, "v", _BF16, dev, dim)
    if kn != N or vn != N or kh != vh:
        raise SpecVerifyError("k and v must be [N, kv_heads, head_dim] with the rows of q")
    shape = _shape(cu_tokens)
    if shape is None or len(shape) != 1 or shape[0] < 2:
        raise SpecVerifyError("cu_tokens must be [B + 1] int32")
    _whole(window, "window", 0, _I32 - 1)
    if scale is None:
        scale = dim ** -0.5
    if not isinstance(scale, (int, float)):
        raise SpecVerifyError("scale must be a number")
    return dev, (qp, qs, kp, ks, vp, vs), (ptr(cu_tokens, "cu_tokens", torch.int32, dev), shape[0] - 1, N, qh, kh, dim,
                                           scale, window)


def _given(t, name, shape, dtype, device):
    """A tensor to write to and its address: the caller's, or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    if _shape(t) != shape:
        raise SpecVerifyError(f"{name} must be {list(shape)}")
    return t, ptr(t, name, dtype, device)


def _forward(q, k, v, cu_tokens, scale, window, out, lse, stream):
    dev, qkv, rest = _inputs(q, k, v, cu_tokens, scale, window)
    with on_device(dev, stream, q, k, v, cu_tokens, out, lse) as st:
        given = [t for t in (out, lse) if t is not None]
        out, op = _given(out, "out", tuple(q.shape), _BF16, dev)
        lse, lp = _given(lse, "lse", tuple(q.shape[:2]), torch.float32, dev)
        rc = load().spec_prompt_attention(*qkv, *rest, op, lp, st)
    if rc:
        _check(rc, "spec_prompt_attention")
    if given:
        wrote(*given)
    return out, lse


class _Function(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_tokens, scale, window, stream):
        out, lse = _forward(q, k, v, cu_tokens, scale, window, None, None, stream)
        ctx.save_for_backward(q, k, v, cu_tokens, out, lse)
        ctx.of = scale, window
        ctx.done = None if stream is None else stream.record_event()
        ctx.set_materialize_grads(False)
        return out, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_out, g_lse):
        if g_lse is not None:
            raise SpecVerifyError("lse has no gradient: use it detached in a loss")
        if g_out is None:
            return (None,) * 7
        saved = ctx.saved_tensors
        if ctx.done is not None:
            # The forward pass ran on a stream of its own: this one comes after it, and the
            # allocator learns that what it left is in use here.
            here = torch.cuda.current_stream(saved[0].device)
            here.wait_event(ctx.done)
            for t in saved:
                t.record_stream(here)
        q, k, v, cu_tokens, out, lse = saved
        g = spec_prompt_attention_backward(g_out.contiguous(), q, k, v, out, lse, cu_tokens, *ctx.of)
        return (*(x if need else None for x, need in zip(g, ctx.needs_input_grad)), None, None, None, None)


def spec_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_tokens: torch.Tensor,
                          scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
                          lse: torch.Tensor | None = None, stream=None):
    """Causal attention over packed prompts: sequence b has rows cu_tokens[b] .. cu_tokens[b + 1] - 1
    of q [N, q_heads, head_dim] and k, v [N, kv_heads, head_dim] (bf16, head_dim 64 or 128; parts of one
    projection's output as they lie); its token i sees its tokens up to i and, with window > 0, only
    the last `window` of them. Returns (out [N, q_heads, head_dim] bf16, lse [N, q_heads] float32).

    When q, k or v requires a gradient, out is differentiable with respect to them; a backward pass
    through lse raises, and so does a call that is handed out or lse then. Rows outside every
    sequence give out 0, lse -inf and gradients 0. scale (>= 0) defaults to head_dim^-1/2."""
    no_tangent("spec_prompt_attention", q, k, v)
    if torch.is_grad_enabled() and any(getattr(t, "requires_grad", False) for t in (q, k, v)):
        if out is not None or lse is not None:
            raise SpecVerifyError("out and lse cannot be given where a gradient is recorded")
        return _Function.apply(q, k, v, cu_tokens, scale, window, stream)
    return _forward(q, k, v, cu_tokens, scale, window, out, lse, stream)


def spec_prompt_attention_backward(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                   out: torch.Tensor, lse: torch.Tensor, cu_tokens: torch.Tensor,
                                   scale: float | None = None, window: int = 0,
                                   workspace: torch.Tensor | None = None, stream=None):
    """The gradients (grad_q, grad_k, grad_v) of a loss whose gradient with respect to out is grad_out
    [N, q_heads, head_dim] bf16; out and lse are what spec_prompt_attention returned for the same
    arguments. workspace: uint8, at least spec_prompt_attention_backward_workspace_bytes(...) bytes,
    not shared by calls that may overlap."""
    no_tangent("spec_prompt_attention_backward", grad_out, q, k, v, out, lse)
    dev, qkv, rest = _inputs(q, k, v, cu_tokens, scale, window)
    dim, shape = q.shape[2], tuple(q.shape)
    gp, gs, _, _ = _heads(grad_out, "grad_out", _BF16, dev, dim)
    if _shape(grad_out) != shape or _shape(out) != shape or _shape(lse) != shape[:2]:
        raise SpecVerifyError("grad_out and out must be [N, q_heads, head_dim], lse [N, q_heads]")
    op, lp = ptr(out, "out", _BF16, dev), ptr(lse, "lse", torch.float32, dev)
    with on_device(dev, stream, grad_out, q, k, v, out, lse, cu_tokens, workspace) as st:
        if workspace is None:
            size = load().spec_prompt_attention_backward_workspace_bytes(*rest[1:6])
            workspace = torch.empty(size or 16, dtype=torch.uint8, device=dev)
        wp, size = ptr(workspace, "workspace", torch.uint8, dev), workspace.numel()
        grads = [torch.empty(t.shape, dtype=_BF16, device=dev) for t in (q, k, v)]
        rc = load().spec_prompt_attention_backward(gp, gs, *qkv, op, lp, *rest, *(g.data_ptr() for g in grads), wp, size, st)
    if rc:
        _check(rc, "spec_prompt_attention_backward")
    return tuple(grads)


def spec_prompt_attention_backward_workspace_bytes(B: int, N: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace of spec_prompt_attention_backward on the current device; 0 for arguments outside its limits."""
    if not all(0 <= x < _I32 for x in (B, N, q_heads, kv_heads, head_dim)):
        return 0
    return int(load().spec_prompt_attention_backward_workspace_bytes(B, N, q_heads, kv_heads, head_dim))

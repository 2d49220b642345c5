"""Where a call runs: its device and stream, and the pointers handed to the library."""
from __future__ import annotations

import contextlib

import torch
from torch.autograd import forward_ad

from . import SpecVerifyError

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def ptr(t: torch.Tensor, name: str, dtype, device) -> int:
    """Device address of a contiguous tensor of this type on this CUDA device."""
    try:
        if t.dtype is dtype and t.device == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SpecVerifyError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise SpecVerifyError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise SpecVerifyError(f"{name} must be on {device}, got {t.device}")
    raise SpecVerifyError(f"{name} must be contiguous")


def no_tangent(call: str, *tensors):
    """Refuses forward-mode AD: the calls would drop the tangents in silence."""
    if getattr(forward_ad, "_current_level", 0) < 0:      # no dual level is open
        return
    for t in tensors:
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            raise SpecVerifyError(f"{call} carries no forward-mode tangents")


def wrote(*tensors) -> None:
    """Tells autograd that a kernel has written over a caller's tensors: a graph that saved one of
    them raises in its backward pass."""
    for t in tensors:
        torch.autograd.graph.increment_version(t)


class _NoGradient(torch.autograd.Function):
    @staticmethod
    def forward(ctx, call, n, *tensors):
        ctx.call = call
        return tensors[:n]

    @staticmethod
    def backward(ctx, *grads):
        raise SpecVerifyError(f"{ctx.call} has no gradient")


def no_gradient(call: str, outputs: tuple, *inputs):
    """The outputs of a call that has no gradient: where an input requires one, a backward pass
    through them raises instead of stopping in silence."""
    if not torch.is_grad_enabled():
        return outputs
    return _NoGradient.apply(call, len(outputs), *outputs, *inputs)


class _Here:
    """The device's current stream on the current device: nothing to set or restore."""
    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


@contextlib.contextmanager
def _there(device, stream, tensors):
    with torch.cuda.device(device):
        s = torch.cuda.current_stream() if stream is None else stream
        # Outputs made inside come from this stream's memory, and the caching
        # allocator learns that the inputs are in use on it.
        with torch.cuda.stream(s):
            if stream is not None:
                for t in tensors:
                    if isinstance(t, torch.Tensor) and t.is_cuda:
                        t.record_stream(s)
            yield int(s.cuda_stream)


def on_device(device, stream, *tensors):
    """Context in which outputs are allocated and the call is made; gives the stream's
    handle. The caller orders `stream` after the work that produces the tensors."""
    if stream is None and device.index == torch.cuda.current_device():
        return _Here(_raw_stream(device.index) if _raw_stream else int(torch.cuda.current_stream().cuda_stream))
    return _there(device, stream, tensors)

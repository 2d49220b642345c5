"""LM-head logits with weights in 4 bits and a scale and a bias for each group
(include/spec_lm_head.h)."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import SpecVerifyError, _check, load
from ._launch import no_gradient, no_tangent, on_device, ptr, wrote
from .kv import _shape


class Q4Weight(NamedTuple):
    """A weight [V, d] in 4 bits: w[v][j] = scale[v][j // group] * code[v][j] + bias[v][j // group]."""
    codes: torch.Tensor    # [V, d / 2] uint8: elements 2 j and 2 j + 1 in the low and the high half of byte j
    scale: torch.Tensor    # [V, d / group] bfloat16
    bias: torch.Tensor     # [V, d / group] bfloat16

    @classmethod
    def quantize(cls, weight: torch.Tensor, group: int = 64) -> "Q4Weight":
        """The weight [V, d] with 16 even steps from each group's smallest to its largest element."""
        if not isinstance(weight, torch.Tensor) or weight.dim() != 2 or not weight.is_floating_point():
            raise SpecVerifyError("weight must be [V, d] in floating point")
        V, d = weight.shape
        if group not in (32, 64, 128) or d < 64 or d % 64 or d % group or V < 1:
            raise SpecVerifyError("group must be 32, 64 or 128 and divide d, a multiple of 64")
        codes = torch.empty(V, d // 2, dtype=torch.uint8, device=weight.device)
        scale, bias = (torch.empty(V, d // group, dtype=torch.bfloat16, device=weight.device) for _ in range(2))
        for a in range(0, V, 16384):               # a part at a time: the fp32 copy stays small
            w = weight[a:a + 16384].detach().float().unflatten(1, (-1, group))
            lo, hi = w.amin(2), w.amax(2)
            s, b = ((hi - lo) / 15).to(torch.bfloat16), lo.to(torch.bfloat16)
            step = s.float()[..., None]
            q = torch.where(step > 0, (w - b.float()[..., None]) / step, 0.0).round_().clamp_(0, 15).to(torch.uint8).flatten(1)
            codes[a:a + 16384] = q[:, 0::2] | q[:, 1::2] << 4
            scale[a:a + 16384], bias[a:a + 16384] = s, b
        return cls(codes, scale, bias)

    def dequantize(self) -> torch.Tensor:
        """The weight [V, d] in float32."""
        q = torch.stack((self.codes & 15, self.codes >> 4), -1).flatten(1).unflatten(1, (self.scale.shape[1], -1))
        return (q.float() * self.scale.float()[..., None] + self.bias.float()[..., None]).flatten(1)


def spec_lm_head_logits_q4(hidden: torch.Tensor, weight: Q4Weight, out: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    """logits [..., V] fp32 = hidden [..., d] (bf16) . weight^T with a head in 4 bits: for a few rows,
    which are bound by the head's bytes (it is read again for every 64 rows). The call serves: a
    backward pass through the logits raises."""
    if not isinstance(hidden, torch.Tensor) or not hidden.is_cuda:
        raise SpecVerifyError("hidden must be a CUDA tensor")
    if not isinstance(weight, tuple) or len(weight) != 3:
        raise SpecVerifyError("weight must be a Q4Weight")
    no_tangent("spec_lm_head_logits_q4", hidden)
    dev = hidden.device
    codes, scale, bias = weight
    if hidden.dim() < 1 or len(_shape(codes) or ()) != 2 or codes.shape[1] * 2 != hidden.shape[-1]:
        raise SpecVerifyError("codes must be [V, d / 2] with the hidden states' d")
    V, d = codes.shape[0], hidden.shape[-1]
    groups = (_shape(scale) or (0, 0))[-1]
    if not groups or d % groups or _shape(scale) != (V, groups) or _shape(bias) != (V, groups):
        raise SpecVerifyError("scale and bias must be [V, d / group]")
    hp, cp = ptr(hidden, "hidden", torch.bfloat16, dev), ptr(codes, "codes", torch.uint8, dev)
    sp, bp = ptr(scale, "scale", torch.bfloat16, dev), ptr(bias, "bias", torch.bfloat16, dev)
    M, shape = hidden.numel() // d, (*hidden.shape[:-1], V)
    if not 1 <= M <= 65536:
        raise SpecVerifyError("hidden must have 1..65536 rows")
    with on_device(dev, stream, hidden, codes, scale, bias, out) as st:
        given = out
        if out is None:
            out = torch.empty(shape, dtype=torch.float32, device=dev)
            op = out.data_ptr()
        elif _shape(out) != shape:
            raise SpecVerifyError(f"out must be {list(shape)}")
        else:
            op = ptr(out, "out", torch.float32, dev)
        rc = load().spec_lm_head_logits_q4(hp, cp, sp, bp, M, V, d, d // groups, op, st)
    if rc:
        _check(rc, "spec_lm_head_logits_q4")
    if given is not None:
        wrote(given)
    if hidden.requires_grad or scale.requires_grad or bias.requires_grad:
        return no_gradient("spec_lm_head_logits_q4", (out,), hidden, scale, bias)[0]
    return out

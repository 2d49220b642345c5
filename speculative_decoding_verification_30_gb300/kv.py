"""The target model's paged 8-bit key/value cache around the verify step: appending a
window of tokens, and the attention of the window over it (include/spec_kv.h)."""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

from . import SpecVerifyError, _check, _dtype_code, load
from ._launch import on_device, ptr


class KVCache(NamedTuple):
    """Pages of keys and values in e4m3, with one scale for each page and kv head."""
    k_codes: torch.Tensor    # [num_pages, kv_heads, page_size, head_dim] float8_e4m3fn (or uint8)
    k_scale: torch.Tensor    # [num_pages, kv_heads] float32
    v_codes: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda") -> "KVCache":
        """A cache that holds nothing yet (its pages are written before they are read)."""
        def codes():
            return torch.zeros(num_pages, kv_heads, page_size, head_dim, dtype=torch.uint8,
                               device=device).view(torch.float8_e4m3fn)
        return cls(codes(), torch.ones(num_pages, kv_heads, device=device), codes(),
                   torch.ones(num_pages, kv_heads, device=device))


def rope_tables(max_pos: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """(cos, sin) [max_pos, rot_dim / 2] float32 of the angles pos * base^(-2 i / rot_dim),
    formed in 64 bits."""
    inv = float(base) ** (-torch.arange(rot_dim // 2, dtype=torch.float64, device=device) * 2 / rot_dim)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return a.cos().float(), a.sin().float()


def _cache(kv: KVCache, device):
    """Pointers and [num_pages, kv_heads, page_size, head_dim] of a cache."""
    k, v = kv.k_codes, kv.v_codes
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or k.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise SpecVerifyError("the codes must be [num_pages, kv_heads, page_size, head_dim] float8_e4m3fn or uint8")
    if v.shape != k.shape or kv.k_scale.shape != k.shape[:2] or kv.v_scale.shape != k.shape[:2]:
        raise SpecVerifyError("keys and values must have one shape, the scales [num_pages, kv_heads]")
    return (ptr(k, "k_codes", k.dtype, device), ptr(kv.k_scale, "k_scale", torch.float32, device),
            ptr(v, "v_codes", k.dtype, device), ptr(kv.v_scale, "v_scale", torch.float32, device)), k.shape


def _window(seq_len, cu_tokens, page_table, device):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise SpecVerifyError("page_table must be [B, max_pages]")
    B = page_table.shape[0]
    if seq_len.shape != (B,) or cu_tokens.shape != (B + 1,):
        raise SpecVerifyError("seq_len must be [B] and cu_tokens [B + 1]")
    return (ptr(seq_len, "seq_len", torch.int32, device), ptr(cu_tokens, "cu_tokens", torch.int32, device),
            ptr(page_table, "page_table", torch.int32, device)), B, page_table.shape[1]


def _heads(x, name, dtype, device, dim):
    """(address, token stride, heads) of [N, heads, dim] with adjacent heads."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.device != device:
        raise SpecVerifyError(f"{name} must be a CUDA tensor on {device}")
    if x.dim() != 3 or x.shape[2] != dim or x.dtype != dtype:
        raise SpecVerifyError(f"{name} must be [N, heads, {dim}] {dtype}")
    if x.stride(2) != 1 or (x.shape[1] > 1 and x.stride(1) != dim):
        raise SpecVerifyError(f"{name}: the heads of a token must be adjacent")
    return x.data_ptr(), x.stride(0) if x.shape[0] > 1 else x.shape[1] * dim, x.shape[1]


def spec_kv_append(k: torch.Tensor, v: torch.Tensor, kv: KVCache, seq_len: torch.Tensor, cu_tokens: torch.Tensor,
                   page_table: torch.Tensor, max_tokens: int, q: torch.Tensor | None = None,
                   cos: torch.Tensor | None = None, sin: torch.Tensor | None = None, interleaved: bool = False,
                   q_out: torch.Tensor | None = None, flag: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor | None:
    """Appends a window's keys and values [N, kv_heads, head_dim] (bf16 or fp32) to the cache
    at positions seq_len[b], seq_len[b] + 1, ... of each sequence, rotated by the tables cos
    and sin [max_pos, rot_dim / 2] when these are given. Returns the rotated queries when q
    [N, q_heads, head_dim] is given (in q_out, which may be q).

    seq_len is not advanced: spec_verify_step does that by the tokens it emits. flag [1] int32
    becomes 1 when a token could not be stored."""
    if not isinstance(k, torch.Tensor) or not k.is_cuda:
        raise SpecVerifyError("k must be a CUDA tensor")
    dev, dt = k.device, _dtype_code(k)
    cache, (pages, heads, page, dim) = _cache(kv, dev)
    win, B, max_pages = _window(seq_len, cu_tokens, page_table, dev)
    kp, ks, kh = _heads(k, "k", k.dtype, dev, dim)
    vp, vs, vh = _heads(v, "v", k.dtype, dev, dim)
    N = k.shape[0]
    if kh != heads or vh != heads or v.shape[0] != N:
        raise SpecVerifyError("k and v must be [N, kv_heads, head_dim] of the cache")
    rot = max_pos = 0
    cp = sp = None
    if (cos is None) != (sin is None):
        raise SpecVerifyError("cos and sin come together")
    if cos is not None:
        if cos.dim() != 2 or cos.shape != sin.shape:
            raise SpecVerifyError("cos and sin must be [max_pos, rot_dim / 2]")
        max_pos, rot = cos.shape[0], 2 * cos.shape[1]
        cp, sp = ptr(cos, "cos", torch.float32, dev), ptr(sin, "sin", torch.float32, dev)
    fp = None if flag is None else ptr(flag, "flag", torch.int32, dev)
    with on_device(dev, stream, k, v, *kv, seq_len, cu_tokens, page_table, q, cos, sin, q_out, flag) as st:
        qp = op = None
        qs, qh = 0, heads
        if q is not None:
            qp, qs, qh = _heads(q, "q", k.dtype, dev, dim)
            if q.shape[0] != N:
                raise SpecVerifyError("q must have the rows of k")
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            elif q_out.shape != q.shape:
                raise SpecVerifyError("q_out must have q's shape")
            op = ptr(q_out, "q_out", q.dtype, dev)
        elif q_out is not None:
            raise SpecVerifyError("q_out without q")
        rc = load().spec_kv_append(kp, ks, vp, vs, qp, qs, op, dt, cp, sp, rot, max_pos, int(interleaved), *win, B, N,
                                   max_tokens, max_pages, pages, page, qh, heads, dim, *cache, fp, st)
    _check(rc, "spec_kv_append")
    return q_out


def spec_kv_attention_workspace_bytes(B: int, max_tokens: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace of spec_kv_attention on the current device."""
    return int(load().spec_kv_attention_workspace_bytes(B, max_tokens, q_heads, kv_heads, head_dim))


def spec_kv_attention(q: torch.Tensor, kv: KVCache, seq_len: torch.Tensor, cu_tokens: torch.Tensor,
                      page_table: torch.Tensor, max_tokens: int, scale: float | None = None, window: int = 0,
                      out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None):
    """Attention of a window's queries q [N, q_heads, head_dim] (bf16) over the cache: query i
    of sequence b, at position seq_len[b] + i, sees the keys up to its own position (the window
    must have been appended) and, with window > 0, only the last `window` of them. Returns
    (out [N, q_heads, head_dim] bf16, lse [N, q_heads] float32).

    scale defaults to head_dim^-1/2. workspace: uint8, at least
    spec_kv_attention_workspace_bytes(...) bytes, not shared by calls that may overlap."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise SpecVerifyError("q must be a CUDA tensor")
    dev = q.device
    cache, (pages, heads, page, dim) = _cache(kv, dev)
    win, B, max_pages = _window(seq_len, cu_tokens, page_table, dev)
    qp, qs, qh = _heads(q, "q", torch.bfloat16, dev, dim)
    N = q.shape[0]
    if scale is None:
        scale = 1.0 / math.sqrt(dim)
    with on_device(dev, stream, q, *kv, seq_len, cu_tokens, page_table, out, lse, workspace) as st:
        need = spec_kv_attention_workspace_bytes(B, max_tokens, qh, heads, dim)
        if workspace is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        if out is None:
            out = torch.empty(N, qh, dim, dtype=torch.bfloat16, device=dev)
        elif out.shape != (N, qh, dim):
            raise SpecVerifyError("out must be [N, q_heads, head_dim]")
        if lse is None:
            lse = torch.empty(N, qh, dtype=torch.float32, device=dev)
        elif lse.shape != (N, qh):
            raise SpecVerifyError("lse must be [N, q_heads]")
        rc = load().spec_kv_attention(qp, qs, *cache, *win, B, N, max_tokens, max_pages, pages, page, qh, heads, dim,
                                      float(scale), window, ptr(out, "out", torch.bfloat16, dev),
                                      ptr(lse, "lse", torch.float32, dev),
                                      ptr(workspace, "workspace", torch.uint8, dev), workspace.numel(), st)
    _check(rc, "spec_kv_attention")
    return out, lse

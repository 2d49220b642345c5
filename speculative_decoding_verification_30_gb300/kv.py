"""The target model's paged 8-bit key/value cache around the verify step: appending a
window of tokens, and the attention of the window over it (include/spec_kv.h)."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import SpecVerifyError, _check, _dtype_code, load
from ._launch import no_gradient, no_tangent, on_device, ptr, wrote


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


_CODES = (torch.float8_e4m3fn, torch.uint8)


def _shape(t):
    return getattr(t, "shape", None)


def _cache(kv: KVCache, device):
    """Pointers and [num_pages, kv_heads, page_size, head_dim] of a cache."""
    k, ks, v, vs = kv
    shape = getattr(k, "shape", ())
    if len(shape) != 4 or k.dtype not in _CODES:
        raise SpecVerifyError("the codes must be [num_pages, kv_heads, page_size, head_dim] float8_e4m3fn or uint8")
    if _shape(v) != shape or _shape(ks) != shape[:2] or _shape(vs) != shape[:2]:
        raise SpecVerifyError("keys and values must have one shape, the scales [num_pages, kv_heads]")
    ty = k.dtype
    return (ptr(k, "k_codes", ty, device), ptr(ks, "k_scale", torch.float32, device), ptr(v, "v_codes", ty, device),
            ptr(vs, "v_scale", torch.float32, device)), shape


def _window(seq_len, cu_tokens, page_table, device):
    """Pointers, B and max_pages of a window's tables."""
    i32 = torch.int32
    try:
        B, max_pages = page_table.shape
    except (AttributeError, ValueError):
        raise SpecVerifyError("page_table must be [B, max_pages]") from None
    if _shape(seq_len) != (B,) or _shape(cu_tokens) != (B + 1,):
        raise SpecVerifyError("seq_len must be [B] and cu_tokens [B + 1]")
    return (ptr(seq_len, "seq_len", i32, device), ptr(cu_tokens, "cu_tokens", i32, device),
            ptr(page_table, "page_table", i32, device)), B, max_pages


_I32 = 2 ** 31


def _whole(x, name, lo, hi):
    """Refuses what is no whole number of lo..hi: a larger one would be cut to 32 bits."""
    if not isinstance(x, int) or not lo <= x <= hi:
        raise SpecVerifyError(f"{name} must be a whole number of {lo}..{hi}")


def _heads(x, name, dtype, device, dim):
    """(address, token stride, N, heads) of [N, heads, dim] with adjacent heads."""
    try:
        n, heads, d = x.shape
        ts, hs, ds = x.stride()
    except (AttributeError, ValueError):
        raise SpecVerifyError(f"{name} must be [N, heads, {dim}] {dtype}") from None
    if x.device != device:
        raise SpecVerifyError(f"{name} must be a CUDA tensor on {device}")
    if d != dim or x.dtype != dtype:
        raise SpecVerifyError(f"{name} must be [N, heads, {dim}] {dtype}")
    if ds != 1 or (heads > 1 and hs != dim):
        raise SpecVerifyError(f"{name}: the heads of a token must be adjacent")
    return x.data_ptr(), ts if n > 1 else heads * dim, n, heads


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
    becomes 1 when a token could not be stored. The call serves: what enters the cache has no
    gradient, and a backward pass through the rotated queries raises.

    max_tokens bounds the new tokens of a sequence. Of one with more, only the first max_tokens are
    stored (flag becomes 1) and only their rows of the result are written."""
    if not isinstance(k, torch.Tensor) or not k.is_cuda:
        raise SpecVerifyError("k must be a CUDA tensor")
    no_tangent("spec_kv_append", k, v, q)
    dev, ty = k.device, k.dtype
    dt = _dtype_code(k)
    cache, (pages, heads, page, dim) = _cache(kv, dev)
    win, B, max_pages = _window(seq_len, cu_tokens, page_table, dev)
    kp, ks, N, kh = _heads(k, "k", ty, dev, dim)
    vp, vs, vn, vh = _heads(v, "v", ty, dev, dim)
    if kh != heads or vh != heads or vn != N:
        raise SpecVerifyError("k and v must be [N, kv_heads, head_dim] of the cache")
    _whole(max_tokens, "max_tokens", 1, N)
    rot = max_pos = 0
    cp = sp = None
    if (cos is None) != (sin is None):
        raise SpecVerifyError("cos and sin come together")
    if cos is not None:
        if len(_shape(cos) or ()) != 2 or cos.shape != _shape(sin):
            raise SpecVerifyError("cos and sin must be [max_pos, rot_dim / 2]")
        max_pos, rot = cos.shape
        rot *= 2
        cp, sp = ptr(cos, "cos", torch.float32, dev), ptr(sin, "sin", torch.float32, dev)
    fp = None if flag is None else ptr(flag, "flag", torch.int32, dev)
    if fp == 0:
        raise SpecVerifyError("flag must be [1] int32")
    with on_device(dev, stream, k, v, *kv, seq_len, cu_tokens, page_table, q, cos, sin, q_out, flag) as st:
        qp = op = None
        qs, qh, given = 0, heads, q_out
        if q is not None:
            qp, qs, qn, qh = _heads(q, "q", ty, dev, dim)
            if qn != N:
                raise SpecVerifyError("q must have the rows of k")
            if q_out is None:
                q_out = torch.empty((N, qh, dim), dtype=ty, device=dev)
                op = q_out.data_ptr()
            elif _shape(q_out) != q.shape:
                raise SpecVerifyError("q_out must have q's shape")
            else:
                op = ptr(q_out, "q_out", ty, dev)
        elif q_out is not None:
            raise SpecVerifyError("q_out without q")
        rc = load().spec_kv_append(kp, ks, vp, vs, qp, qs, op, dt, cp, sp, rot, max_pos, int(interleaved), *win, B, N,
                                   max_tokens, max_pages, pages, page, qh, heads, dim, *cache, fp, st)
    if rc:
        _check(rc, "spec_kv_append")
    if given is not None:
        wrote(given)
    if q is not None and (q.requires_grad or k.requires_grad or v.requires_grad):
        return no_gradient("spec_kv_append", (q_out,), q, k, v)[0]
    return q_out


def spec_kv_attention_workspace_bytes(B: int, max_tokens: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace of spec_kv_attention on the current device; 0 for arguments outside its limits."""
    if not all(0 <= x < _I32 for x in (B, max_tokens, q_heads, kv_heads, head_dim)):
        return 0
    return int(load().spec_kv_attention_workspace_bytes(B, max_tokens, q_heads, kv_heads, head_dim))


def spec_kv_attention(q: torch.Tensor, kv: KVCache, seq_len: torch.Tensor, cu_tokens: torch.Tensor,
                      page_table: torch.Tensor, max_tokens: int, scale: float | None = None, window: int = 0,
                      out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None):
    """Attention of a window's queries q [N, q_heads, head_dim] (bf16) over the cache: query i
    of sequence b, at position seq_len[b] + i, sees the keys up to its own position (the window
    must have been appended) and, with window > 0, only the last `window` of them. Returns
    (out [N, q_heads, head_dim] bf16, lse [N, q_heads] float32).

    The call serves: a backward pass through its outputs raises. Rows of a sequence past its
    first max_tokens are not written.

    scale defaults to head_dim^-1/2. workspace: uint8, at least
    spec_kv_attention_workspace_bytes(...) bytes, not shared by calls that may overlap."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise SpecVerifyError("q must be a CUDA tensor")
    no_tangent("spec_kv_attention", q)
    dev = q.device
    cache, (pages, heads, page, dim) = _cache(kv, dev)
    win, B, max_pages = _window(seq_len, cu_tokens, page_table, dev)
    qp, qs, N, qh = _heads(q, "q", torch.bfloat16, dev, dim)
    if type(max_tokens) is not int or type(window) is not int or not (0 < max_tokens <= N and 0 <= window < _I32):
        _whole(max_tokens, "max_tokens", 1, N)
        _whole(window, "window", 0, _I32 - 1)
    if scale is None:
        scale = dim ** -0.5
    lib = load()
    with on_device(dev, stream, q, *kv, seq_len, cu_tokens, page_table, out, lse, workspace) as st:
        given = [t for t in (out, lse) if t is not None]
        if workspace is None:
            size = lib.spec_kv_attention_workspace_bytes(B, max_tokens, qh, heads, dim) or 16
            workspace = torch.empty(size, dtype=torch.uint8, device=dev)
            wp = workspace.data_ptr()
        else:
            wp = ptr(workspace, "workspace", torch.uint8, dev)
            size = workspace.numel()
        if out is None:
            out = torch.empty((N, qh, dim), dtype=torch.bfloat16, device=dev)
            op = out.data_ptr()
        elif _shape(out) != (N, qh, dim):
            raise SpecVerifyError("out must be [N, q_heads, head_dim]")
        else:
            op = ptr(out, "out", torch.bfloat16, dev)
        if lse is None:
            lse = torch.empty((N, qh), dtype=torch.float32, device=dev)
            lp = lse.data_ptr()
        elif _shape(lse) != (N, qh):
            raise SpecVerifyError("lse must be [N, q_heads]")
        else:
            lp = ptr(lse, "lse", torch.float32, dev)
        rc = lib.spec_kv_attention(qp, qs, *cache, *win, B, N, max_tokens, max_pages, pages, page, qh, heads, dim, scale,
                                   window, op, lp, wp, size, st)
    if rc:
        _check(rc, "spec_kv_attention")
    if given:
        wrote(*given)
    return no_gradient("spec_kv_attention", (out, lse), q) if q.requires_grad else (out, lse)


def spec_kv_attention_shared_workspace_bytes(B: int, groups: int, N: int, max_tokens: int, q_heads: int, kv_heads: int,
                                             head_dim: int) -> int:
    """Bytes of workspace of spec_kv_attention_shared on the current device; 0 for arguments outside its limits."""
    if not all(0 <= x < _I32 for x in (B, groups, N, max_tokens, q_heads, kv_heads, head_dim)):
        return 0
    return int(load().spec_kv_attention_shared_workspace_bytes(B, groups, N, max_tokens, q_heads, kv_heads, head_dim))


def spec_kv_attention_shared(q: torch.Tensor, kv: KVCache, seq_len: torch.Tensor, cu_tokens: torch.Tensor,
                             page_table: torch.Tensor, max_tokens: int, cu_groups: torch.Tensor,
                             shared_len: torch.Tensor, scale: float | None = None, out: torch.Tensor | None = None,
                             lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """spec_kv_attention for a batch whose sequences have leading pages in common (samples of one
    prompt, requests behind one system prompt): group g is the sequences cu_groups[g] ..
    cu_groups[g + 1] - 1 (cu_groups [G + 1] int32, from 0 to B), whose rows of page_table name the same
    pages for the positions below shared_len[g] (shared_len [G] int32). These are read once for all
    rows of the group. seq_len and page_table are those of spec_kv_attention: they count and name
    the shared tokens too. Returns (out [N, q_heads, head_dim] bf16, lse [N, q_heads] float32).

    The call serves: a backward pass through its outputs raises. workspace: uint8, at least
    spec_kv_attention_shared_workspace_bytes(...) bytes, not shared by calls that may overlap."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise SpecVerifyError("q must be a CUDA tensor")
    no_tangent("spec_kv_attention_shared", q)
    dev = q.device
    cache, (pages, heads, page, dim) = _cache(kv, dev)
    win, B, max_pages = _window(seq_len, cu_tokens, page_table, dev)
    groups = (_shape(shared_len) or (0,))[0]
    if _shape(shared_len) != (groups,) or groups < 1 or _shape(cu_groups) != (groups + 1,):
        raise SpecVerifyError("shared_len must be [G] and cu_groups [G + 1]")
    gp, sp = ptr(cu_groups, "cu_groups", torch.int32, dev), ptr(shared_len, "shared_len", torch.int32, dev)
    qp, qs, N, qh = _heads(q, "q", torch.bfloat16, dev, dim)
    _whole(max_tokens, "max_tokens", 1, N)
    if scale is None:
        scale = dim ** -0.5
    lib = load()
    with on_device(dev, stream, q, *kv, seq_len, cu_tokens, page_table, cu_groups, shared_len, out, lse, workspace) as st:
        given = [t for t in (out, lse) if t is not None]
        if workspace is None:
            size = lib.spec_kv_attention_shared_workspace_bytes(B, groups, N, max_tokens, qh, heads, dim) or 16
            workspace = torch.empty(size, dtype=torch.uint8, device=dev)
            wp = workspace.data_ptr()
        else:
            wp = ptr(workspace, "workspace", torch.uint8, dev)
            size = workspace.numel()
        if out is None:
            out = torch.empty((N, qh, dim), dtype=torch.bfloat16, device=dev)
            op = out.data_ptr()
        elif _shape(out) != (N, qh, dim):
            raise SpecVerifyError("out must be [N, q_heads, head_dim]")
        else:
            op = ptr(out, "out", torch.bfloat16, dev)
        if lse is None:
            lse = torch.empty((N, qh), dtype=torch.float32, device=dev)
            lp = lse.data_ptr()
        elif _shape(lse) != (N, qh):
            raise SpecVerifyError("lse must be [N, q_heads]")
        else:
            lp = ptr(lse, "lse", torch.float32, dev)
        rc = lib.spec_kv_attention_shared(qp, qs, *cache, *win, gp, sp, B, groups, N, max_tokens, max_pages, pages, page, qh,
                                          heads, dim, scale, op, lp, wp, size, st)
    if rc:
        _check(rc, "spec_kv_attention_shared")
    if given:
        wrote(*given)
    return no_gradient("spec_kv_attention_shared", (out, lse), q) if q.requires_grad else (out, lse)

// kv_common.cuh -- the window's and the cache's layout, shared by the append and
// attention kernels (definitions in include/spec_kv.h).
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spec_kv.h"

namespace svkv {

// Device view of one call's sequences and pages.
struct Window {
  const int32_t* seq_len;
  const int32_t* cu_tokens;
  const int32_t* page_table;
  int B, N, max_tokens, max_pages, num_pages, page_size, q_heads, kv_heads, head_dim;
};

// New tokens of sequence b: rows first .. first + count - 1 at positions len + i.
// Inconsistent cu_tokens are cut to what the arrays hold.
struct Seq {
  long long len;
  int first, count, given;   // given: before the cut to max_tokens
};
__device__ __forceinline__ Seq sequence(const Window& w, int b) {
  Seq s;
  s.len = w.seq_len[b];
  s.first = min(max(w.cu_tokens[b], 0), w.N);
  s.given = max(min(w.cu_tokens[b + 1], w.N) - s.first, 0);
  s.count = min(s.given, w.max_tokens);
  return s;
}

// Page of block j of sequence b, or -1.
__device__ __forceinline__ int page_of(const Window& w, int b, long long j) {
  if (j >= w.max_pages) return -1;
  const int p = w.page_table[(size_t)b * w.max_pages + j];
  return p >= 0 && p < w.num_pages ? p : -1;
}

// Four values as e4m3 codes: to nearest even, beyond 448 to 448, NaN stays NaN.
__device__ __forceinline__ uint32_t encode4(const float* x) {
  const uint16_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint16_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)a | ((uint32_t)b << 16);
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool bad_window(const Window& w) {
  if (w.B < 1 || w.B > 65535 || w.N < 1 || w.N > (1 << 24) || w.max_tokens < 1 || w.max_tokens > w.N) return true;
  if (w.page_size != 16 && w.page_size != 32 && w.page_size != 64 && w.page_size != 128) return true;
  if (w.head_dim != 64 && w.head_dim != 128) return true;
  if (w.kv_heads < 1 || w.kv_heads > 256 || w.q_heads < w.kv_heads || w.q_heads % w.kv_heads ||
      w.q_heads / w.kv_heads > 64)
    return true;
  return w.max_pages < 1 || w.max_pages > (1 << 20) || w.num_pages < 1 ||
         (long long)w.num_pages * w.kv_heads * w.page_size >= (1ll << 31);
}

}  // namespace svkv

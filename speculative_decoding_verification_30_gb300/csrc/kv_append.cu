// Appending a window of keys and values to the paged 8-bit cache, with the position
// rotation of keys and queries on the way (C ABI and definitions in
// include/spec_kv.h).
//
// One launch. A block owns the keys or the values of one (sequence, page, kv head):
// its new tokens are read once, rotated and kept in registers while the block agrees
// on their largest magnitude, hence on the scale, and then written as codes. The
// unit of work of a thread is 16 elements: two vectors of 8, a rotation's two halves
// when its pairs lie rot_dim / 2 apart, or 16 neighbours. The remaining blocks
// rotate the queries in the same units. Bound by latency for a verify window (a
// chain of table lookup, load, reduction, store: 64 sequences of 5 tokens 5.2 us) and by
// HBM for prompts (24 of up to 1,500 tokens, 440 MB, 87.5 us, 5,020 GB/s: loads are
// waited for with half the warps resident).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv_common.cuh"

namespace svkv {

constexpr int MIN_EXP = -60, MAX_EXP = 119;   // of a scale
// Heads of a thread in a query block, and blocks of 128 threads on an SM: the loads are
// what takes the time, so threads on the SM count more than the angles that more heads
// would save (440 MB of prompts: 88 us with 2 and 9, 91 with 2 and 8, 93 with 2 and 10,
// 108 with 4 and 8, 98 with 1 and 10).
constexpr int QI = 2, BLOCKS = 9;

struct AppendArgs {
  Window w;
  const void *k, *v, *q;
  long long k_stride, v_stride, q_stride;
  void* q_out;
  const float *cos, *sin;
  int rot, max_pos, interleaved;
  uint8_t *k_codes, *v_codes;
  float *k_scale, *v_scale;
  int32_t* flag;
  int pages_per_seq;         // pages a window can touch
  long long kv_blocks;
  int q_blocks_per_seq;
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x) {
  if (sizeof(T) == 2) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  __nv_bfloat162 b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(b);
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Where the two vectors of unit u of a head lie: elements lo and hi. A unit in the
// rotated part has its angles at pair index `pair` (8 of them).
struct Unit {
  int lo, hi, pair;
};
__device__ __forceinline__ Unit unit_at(int u, int rot, int interleaved) {
  Unit t{u * 16, u * 16 + 8, -1};
  if (t.lo < rot) {
    t.pair = u * 8;
    if (!interleaved) t = Unit{u * 8, u * 8 + rot / 2, u * 8};
  }
  return t;
}

// Pairs of floats in one 64-bit register.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Sums of two packed pairs, one by one: a packed addition after a packed
// multiplication is joined with it into one rounding.
__device__ __forceinline__ void add_each(uint64_t p, uint64_t q, float& x, float& y) {
  float a, b, c, d;
  unpair(p, a, b);
  unpair(q, c, d);
  x = __fadd_rn(a, c);
  y = __fadd_rn(b, d);
}

// The angles of a unit: cosines, sines and the sines' negatives, two at a time. Each
// product and each sum of the rotation is rounded once (no contraction), so the result
// does not depend on how the compiler groups them.
struct Angles {
  uint64_t c[4], s[4], n[4];
  __device__ __forceinline__ void load(const AppendArgs& A, int u, long long pos) {
    float x[8], y[8];
    load8(A.cos + pos * (A.rot / 2) + u, x);
    load8(A.sin + pos * (A.rot / 2) + u, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = pair(x[2 * i], x[2 * i + 1]);
      s[i] = pair(y[2 * i], y[2 * i + 1]);
      n[i] = pair(-y[2 * i], -y[2 * i + 1]);
    }
  }
  // (a, b) -> (a c - b s, b c + a s); pairs are (x[i], x[8 + i]) or (x[2 i], x[2 i + 1])
  __device__ __forceinline__ void rotate(float* x, int interleaved) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float &a0 = x[interleaved ? 4 * i : 2 * i], &a1 = x[interleaved ? 4 * i + 2 : 2 * i + 1];
      float &b0 = x[interleaved ? 4 * i + 1 : 8 + 2 * i], &b1 = x[interleaved ? 4 * i + 3 : 9 + 2 * i];
      const uint64_t a = pair(a0, a1), b = pair(b0, b1);
      add_each(mul2(a, c[i]), mul2(b, n[i]), a0, a1);
      add_each(mul2(b, c[i]), mul2(a, s[i]), b0, b1);
    }
  }
};

__device__ __forceinline__ uint2 encode8(const float* x) { return make_uint2(encode4(x), encode4(x + 4)); }

__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float r) {
  float x[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * i] = __fmul_rn(f.x, r);
    x[2 * i + 1] = __fmul_rn(f.y, r);
  }
  return encode4(x);
}

// Smallest power of two s with amax <= 448 s = 1.75 * 2^8 s, within its range.
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
  int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = min(max(e, MIN_EXP), MAX_EXP);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

template <typename T, int NT, int ITEMS, int IL>
__device__ __forceinline__ void append_page(const AppendArgs& A, long long blk) {
  const Window& w = A.w;
  __shared__ uint32_t wmax[NT / 32];
  const bool is_v = blk & 1;
  blk >>= 1;
  const int h = (int)(blk % w.kv_heads);
  blk /= w.kv_heads;
  const int jj = (int)(blk % A.pages_per_seq), b = (int)(blk / A.pages_per_seq);
  const Seq s = sequence(w, b);
  if (s.len < 0 || s.count == 0) return;
  const int P = w.page_size, D = w.head_dim, ush = D == 128 ? 3 : 2, units = 1 << ush;   // units of a head
  const long long j = (s.len >> (__ffs(P) - 1)) + jj;
  const long long lo = max(j * P, s.len), hi = min((j + 1) * P, s.len + s.count);
  const bool first = h == 0 && !is_v && threadIdx.x == 0 && A.flag;
  if (first && jj == 0 && s.given > s.count) *A.flag = 1;
  if (lo >= hi) return;
  const long long end = A.rot ? min(hi, (long long)A.max_pos) : hi;   // past max_pos: not stored
  const int keep = (int)(lo - j * P), n = (int)(max(end, lo) - lo);   // kept tokens, new tokens
  const T* x = static_cast<const T*>(is_v ? A.v : A.k) + (size_t)(s.first + (int)(lo - s.len)) *
               (size_t)(is_v ? A.v_stride : A.k_stride) + h * D;
  const long long stride = is_v ? A.v_stride : A.k_stride;
  const int rot = is_v ? 0 : A.rot;
  // the values are on their way while the page is looked up
  float y[ITEMS][16];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int it = i * NT + threadIdx.x, t = it >> ush;
    if (t < n) {
      const Unit u = unit_at(it & (units - 1), rot, IL);
      load8(x + (size_t)t * stride + u.lo, y[i]);
      load8(x + (size_t)t * stride + u.hi, y[i] + 8);
    }
  }
  const int page = page_of(w, b, j);
  if (first && (page < 0 || end < hi)) *A.flag = 1;
  if (page < 0 || n == 0) return;
  const size_t base = ((size_t)page * w.kv_heads + h) * (size_t)(P * D);
  uint8_t* codes = (is_v ? A.v_codes : A.k_codes) + base;
  float* scale = (is_v ? A.v_scale : A.k_scale) + (size_t)page * w.kv_heads + h;
  const float old = keep ? *scale : 0.f;
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int it = i * NT + threadIdx.x, t = it >> ush;
    if (t < n) {
      const Unit u = unit_at(it & (units - 1), rot, IL);
      if (u.pair >= 0) {
        Angles g;
        g.load(A, u.pair, lo + t);
        g.rotate(y[i], IL);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) big = fmaxf(big, fabsf(y[i][e]));   // passes over NaN
    }
  }
  uint32_t top = __float_as_uint(big);
  if (top == 0x7F800000u) {   // infinities do not count
    top = 0u;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if ((i * NT + threadIdx.x) >> ush < n)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t a = __float_as_uint(y[i][e]) & 0x7FFFFFFFu;
          if (a < 0x7F800000u) top = max(top, a);
        }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) top = max(top, wmax[i]);
  const float sc = fmaxf(scale_of(top), old);
  const bool pow2 = (__float_as_uint(sc) & 0x7FFFFFu) == 0u;
  const float inv = 1.f / sc;
  if (keep && sc > old) {
    const float r = __fdiv_rn(old, sc);
    for (int i = threadIdx.x; i < keep * units; i += NT) {
      uint4* p = reinterpret_cast<uint4*>(codes) + i;
      uint4 c = *p;
      c.x = rescale4(c.x, r);
      c.y = rescale4(c.y, r);
      c.z = rescale4(c.z, r);
      c.w = rescale4(c.w, r);
      *p = c;
    }
  }
  if (threadIdx.x == 0) *scale = sc;   // every thread has read the old one before the barrier
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int it = i * NT + threadIdx.x, t = it >> ush;
    if (t < n) {
      const Unit u = unit_at(it & (units - 1), rot, IL);
      if (pow2) {   // the same quotient, exactly
#pragma unroll
        for (int e = 0; e < 16; e += 2) unpair(mul2(pair(y[i][e], y[i][e + 1]), pair(inv, inv)), y[i][e], y[i][e + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[i][e] = __fdiv_rn(y[i][e], sc);
      }
      uint8_t* o = codes + (size_t)(keep + t) * D;
      *reinterpret_cast<uint2*>(o + u.lo) = encode8(y[i]);
      *reinterpret_cast<uint2*>(o + u.hi) = encode8(y[i] + 8);
    }
  }
}

template <typename T, int NT, int IL>
__device__ __forceinline__ void rotate_queries(const AppendArgs& A, long long blk) {
  const Window& w = A.w;
  const int part = (int)(blk % A.q_blocks_per_seq), b = (int)(blk / A.q_blocks_per_seq);
  const Seq s = sequence(w, b);
  const int D = w.head_dim, ush = D == 128 ? 3 : 2, units = 1 << ush, groups = (w.q_heads + QI - 1) / QI;
  // the thread's token, group of QI heads and unit
  const int it = part * NT + threadIdx.x, e = it >> ush, t = e / groups, h0 = (e - t * groups) * QI;
  if (t >= s.count) return;
  const Unit u = unit_at(it & (units - 1), A.rot, IL);
  const long long pos = s.len + t;
  const T* p = static_cast<const T*>(A.q) + (size_t)(s.first + t) * (size_t)A.q_stride + h0 * D;
  T* o = static_cast<T*>(A.q_out) + ((size_t)(s.first + t) * w.q_heads + h0) * D;
  const int heads = min(QI, w.q_heads - h0);
  const bool blank = s.len < 0, past = A.rot && pos >= A.max_pos;
  float x[QI][16];
#pragma unroll
  for (int i = 0; i < QI; ++i)
    if (i < heads) {
      load8(p + i * D + u.lo, x[i]);
      load8(p + i * D + u.hi, x[i] + 8);
    }
  Angles g;
  const bool turn = u.pair >= 0 && !blank && !past;
  if (turn) g.load(A, u.pair, pos);
#pragma unroll
  for (int i = 0; i < QI; ++i)
    if (i < heads) {
      if (turn) g.rotate(x[i], IL);
      if (blank || past) {
#pragma unroll
        for (int k = 0; k < 16; ++k) x[i][k] = blank ? 0.f : __uint_as_float(0x7FC00000u);
      }
      store8(o + i * D + u.lo, x[i]);
      store8(o + i * D + u.hi, x[i] + 8);
    }
}

template <typename T, int NT, int ITEMS, int IL>
__global__ void __launch_bounds__(NT, BLOCKS * 128 / NT) kv_append_kernel(const AppendArgs A) {
  const long long blk = blockIdx.x;
  if (blk < A.kv_blocks)
    append_page<T, NT, ITEMS, IL>(A, blk);
  else
    rotate_queries<T, NT, IL>(A, blk - A.kv_blocks);
}

template <typename T, int NT, int ITEMS>
static sv_status launch_append(AppendArgs& A, cudaStream_t st) {
  const Window& w = A.w;
  A.pages_per_seq = (w.page_size - 1 + w.max_tokens + w.page_size - 1) / w.page_size;
  A.kv_blocks = 2ll * w.B * A.pages_per_seq * w.kv_heads;
  const long long units = (long long)w.max_tokens * ((w.q_heads + QI - 1) / QI) * (w.head_dim / 16);
  const long long per_seq = A.q ? (units + NT - 1) / NT : 0, blocks = A.kv_blocks + per_seq * w.B;
  if (blocks > 2147483647ll || units > 2147483647ll - NT) return SV_ERR_SHAPE;
  A.q_blocks_per_seq = (int)per_seq;
  if (A.interleaved)
    kv_append_kernel<T, NT, ITEMS, 1><<<(unsigned)blocks, NT, 0, st>>>(A);
  else
    kv_append_kernel<T, NT, ITEMS, 0><<<(unsigned)blocks, NT, 0, st>>>(A);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

// Threads and units of a thread so that a page's new tokens fit the block's registers.
// Full pages of bf16 run faster with fewer threads and some spilled registers (440 MB of
// prompts in pages of 64: 94.6 us against 96.5 with 256 threads of two units; pages of
// 128: 100 against 106), those of fp32 with more (835 MB, pages of 64: 142 against 162).
template <typename T>
static sv_status pick_append(AppendArgs& A, cudaStream_t st) {
  const int most = A.w.max_tokens < A.w.page_size ? A.w.max_tokens : A.w.page_size;
  const int units = most * (A.w.head_dim / 16);
  if (units <= 128) return launch_append<T, 128, 1>(A, st);
  if (units <= 256) return launch_append<T, 128, 2>(A, st);
  if constexpr (sizeof(T) == 2)
    return units <= 512 ? launch_append<T, 128, 4>(A, st) : launch_append<T, 256, 4>(A, st);
  else
    return units <= 512 ? launch_append<T, 256, 2>(A, st) : launch_append<T, 512, 2>(A, st);
}

}  // namespace svkv

sv_status spec_kv_append(const void* k, long long k_stride, const void* v, long long v_stride, const void* q,
                         long long q_stride, void* q_out, sv_dtype dtype, const float* cos, const float* sin,
                         int rot_dim, int max_pos, int interleaved, const int32_t* seq_len,
                         const int32_t* cu_tokens, const int32_t* page_table, int B, int N, int max_tokens,
                         int max_pages, int num_pages, int page_size, int q_heads, int kv_heads, int head_dim,
                         void* k_codes, float* k_scale, void* v_codes, float* v_scale, int32_t* flag,
                         void* stream) {
  using namespace svkv;
  if (!k || !v || !seq_len || !cu_tokens || !page_table || !k_codes || !k_scale || !v_codes || !v_scale)
    return SV_ERR_NULL;
  if ((q == nullptr) != (q_out == nullptr) || (rot_dim != 0 && (!cos || !sin))) return SV_ERR_NULL;
  const Window w{seq_len, cu_tokens, page_table, B,       N,        max_tokens, max_pages,
                 num_pages, page_size, q_heads,  kv_heads, head_dim};
  if (bad_window(w) || rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 || (rot_dim && max_pos < 1))
    return SV_ERR_SHAPE;
  if ((long long)B * max_tokens * kv_heads > 2147483647ll) return SV_ERR_SHAPE;
  const long long kw = (long long)kv_heads * head_dim, qw = (long long)q_heads * head_dim;
  if (k_stride < kw || v_stride < kw || (q && q_stride < qw) || (q && q == q_out && q_stride != qw))
    return SV_ERR_SHAPE;
  if (dtype != SV_BF16 && dtype != SV_F32) return SV_ERR_DTYPE;
  const long long es = dtype == SV_BF16 ? 2 : 4;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(cos, 16) ||
      !aligned(sin, 16) || !aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(seq_len, 4) || !aligned(cu_tokens, 4) || !aligned(page_table, 4) ||
      !aligned(flag, 4) || (k_stride * es) % 16 || (v_stride * es) % 16 || (q && (q_stride * es) % 16))
    return SV_ERR_ALIGN;
  AppendArgs A = {};
  A.w = w;
  A.k = k, A.v = v, A.q = q, A.q_out = q_out;
  A.k_stride = k_stride, A.v_stride = v_stride, A.q_stride = q_stride;
  A.cos = cos, A.sin = sin, A.rot = rot_dim, A.max_pos = max_pos, A.interleaved = interleaved != 0;
  A.k_codes = static_cast<uint8_t*>(k_codes), A.v_codes = static_cast<uint8_t*>(v_codes);
  A.k_scale = k_scale, A.v_scale = v_scale, A.flag = flag;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == SV_BF16 ? pick_append<__nv_bfloat16>(A, st) : pick_append<float>(A, st);
}

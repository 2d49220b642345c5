// Token log-probabilities over logit rows, and their gradient (C ABI and
// definitions in include/spec_logprobs.h).
//
// Forward: one cluster of C CTAs per row, each CTA a contiguous segment of it. One
// pass over the segment: a warp takes groups of 32 consecutive 16-byte vectors
// (256 bf16 or 128 fp32 logits), four groups a wave, the next wave's loads in
// flight while the current one is reduced. Per wave it needs
//   - each group's maximum (a warp reduction), kept in shared memory;
//   - the online softmax sums, in the warp's own frame M = fl(m c) for its maximum m,
//     c = log2(e)/T: s = sum 2^(x c - M) and w = sum 2^(x c - M) (x c - M), two logits
//     an instruction. At the end they are made relative to m (the rounding of M is
//     known exactly): lse = m / T + ln2 log2 s and H = ln2 (log2 s - w / s);
//   - the number of logits that come before the token's in the rank order.
// The top n tokens of a segment lie in the n groups with the largest maxima (ties:
// the lower group, whose ids are lower): were one outside, n groups would each hold
// a logit before it. So the alternatives cost one stored maximum per group, and
// n groups read again from L2 at the end. The n-th largest maximum is found by
// bisection on order keys, stopped as soon as few enough groups remain; what those
// groups hold at or above it is ranked by counting.
//
// Backward: elementwise, p = 2^(x c - lse log2 e) with c and lse log2 e carried as
// two floats each; the few places of t and the top ids that fall in a CTA's chunk
// are listed in shared memory and added before the one rounding. Rows whose |lse| passes
// 64 find their maximum and sum again.
//
// Measured. Forward, one read of the rows: 1,000 rows of 151,936 bf16 with 20
// alternatives 74 us (4,100 GB/s), 2,000 rows of 50,257 fp32 of which a quarter are
// skipped 69 us (4,310 GB/s), both bound by each CTA's start and end, with no load in
// flight, and by issue (11 instructions a logit); 320 rows 36 us, 16 warps an SM; 2 rows 11 us,
// latency. Backward, one read and one write: 512 rows of 151,936 bf16 49 us, 6,040 GB/s,
// bound by HBM.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/spec_logprobs.h"

namespace cg = cooperative_groups;

namespace svlp {

constexpr int NT = 256, NW = NT / 32;
constexpr int SMS = 152;               // of a GB300
constexpr int UNR = 4;                 // groups a warp loads at once
constexpr int MAX_TOP = SV_LOGPROBS_MAX_TOP;
constexpr int MAX_GROUPS = 2048;       // 262,144 fp32 logits in groups of 128
constexpr int SEL_EXTRA = 16;          // the bisection stops at n..n+SEL_EXTRA groups
constexpr int MAX_SEL = MAX_TOP + SEL_EXTRA;
constexpr int MAX_CAND = 512;          // candidates ranked by counting
constexpr int MAX_CLUSTER = 8;
constexpr float LN2 = 0.693147180559945309f;
constexpr float LOG2E = 1.44269504088896341f;
constexpr float LOG2E_LO = (float)(1.4426950408889634074 - (double)LOG2E);
constexpr float U_MIN = -1000.f;       // 2^U_MIN is 0: keeps 0 * -inf out of the sums

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int EPV = 8;
  static __device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<float> {
  static constexpr int EPV = 4;
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ float put(float v) { return v; }
};

// Order key of a logit: descending logits have descending keys, -0 counts as +0.
__device__ __forceinline__ uint32_t okey(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float okey_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;

// The next larger value of the type (x > z is x >= succ(z)).
template <typename T>
__device__ __forceinline__ float succ(float z) {
  constexpr uint32_t step = sizeof(T) == 2 ? 0x10000u : 1u;
  const uint32_t u = __float_as_uint(z + 0.f);
  if (u == 0u) return __uint_as_float(step);
  return __uint_as_float((u & 0x80000000u) ? (u - step == 0x80000000u ? 0u : u - step) : u + step);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float a) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ __nv_bfloat162 as_b2(uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); }

template <typename T>
__device__ __forceinline__ uint4 none_vec() {   // a vector of -inf
  const uint32_t w = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
  return make_uint4(w, w, w, w);
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float* x) {
  if (sizeof(T) == 2) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
}

template <typename T>
__device__ __forceinline__ float vec_max(const uint4& v) {   // NaN if any is NaN
  if (sizeof(T) == 2) {
    const __nv_bfloat162 a = __hmax2_nan(__hmax2_nan(as_b2(v.x), as_b2(v.y)), __hmax2_nan(as_b2(v.z), as_b2(v.w)));
    return max_nan(__low2float(a), __high2float(a));
  }
  float x[4];
  unpack<float>(v, x);
  return max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3]));
}

// Logits of the vectors that are >= thr, as a float.
template <typename T>
__device__ __forceinline__ float count_ge(const uint4 (&v)[UNR], float thr) {
  if (sizeof(T) == 2) {
    const __nv_bfloat162 t = __float2bfloat162_rn(thr);   // exact: thr is a value of the type
    __nv_bfloat162 n = __float2bfloat162_rn(0.f);         // up to 4 UNR each: exact too
#pragma unroll
    for (int u = 0; u < UNR; ++u)
      n = __hadd2(n, __hadd2(__hadd2(__hge2(as_b2(v[u].x), t), __hge2(as_b2(v[u].y), t)),
                             __hadd2(__hge2(as_b2(v[u].z), t), __hge2(as_b2(v[u].w), t))));
    return __low2float(n) + __high2float(n);
  }
  int n = 0;
#pragma unroll
  for (int u = 0; u < UNR; ++u) {
    float x[4];
    unpack<float>(v[u], x);
    n += (x[0] >= thr) + (x[1] >= thr) + (x[2] >= thr) + (x[3] >= thr);
  }
  return (float)n;
}

// Pairs of floats in one 64-bit register: the sums run on packed instructions.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Softmax sums relative to the maximum m: s = sum 2^((x - m) c), w = sum 2^((x - m) c) (x - m) c.
struct Sums {
  float m, s, w;
  __device__ __forceinline__ void add(float x, float c) {
    const float u = fmaxf((x - m) * c, U_MIN);
    const float e = ex2(u);
    s += e;
    w = fmaf(e, u, w);
  }
  // the same sums relative to m2 >= m
  __device__ __forceinline__ void move(float m2, float c) {
    if (m == m2) return;
    const float d = fmaxf((m - m2) * c, U_MIN);
    const float f = s > 0.f ? ex2(d) : 0.f;
    w = f * fmaf(s, d, w);
    s = f * s;
    m = m2;
  }
};

// The same sums, two at a time, in the frame M = fl(m c): an exponent is one fused
// multiply-add, x c - M. Logits are raised to `floor` first, which lies 1000 below the
// frame (weight 0), so that -inf needs no case of its own. Where no such floor exists
// in the type, or M is so large that its rounding would matter (2^-8 at 2^16), `off` is
// set and the sums are taken again by clamped_sums().
struct PairSums {
  float M = -INFINITY, floor = -INFINITY;
  uint64_t s = 0, w = 0, c2 = 0, nm2 = 0;
  bool off = false;
  template <typename T>
  __device__ __forceinline__ void move(float m, float c) {
    float a, b, y, z;
    unpair(s, a, b);
    unpair(w, y, z);
    const float M2 = m * c, d = fmaxf(M - M2, U_MIN), sum = a + b;
    const float f = sum > 0.f ? ex2(d) : 0.f;
    s = pair(f * sum, 0.f);
    w = pair(f * fmaf(sum, d, y + z), 0.f);
    M = M2;
    c2 = pair(c, c);
    nm2 = pair(-M, -M);
    floor = (M - fmaxf(1000.f, fabsf(M) * 0.03125f)) / c;   // below M also after its rounding
    if (sizeof(T) == 2) floor = __bfloat162float(__float2bfloat16_rd(floor));
    off |= !(fabsf(M) < 65536.f && floor > -1e38f);
  }
  __device__ __forceinline__ void add(float x0, float x1) {
    const uint64_t u = fma2(pair(x0, x1), c2, nm2);
    float a, b;
    unpair(u, a, b);
    const uint64_t e = pair(ex2(a), ex2(b));
    s = add2(s, e);
    w = fma2(e, u, w);
  }
  template <typename T>
  __device__ __forceinline__ void add(const uint4& v) {
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
    if (sizeof(T) == 2) {
      const __nv_bfloat162 f = __float2bfloat162_rn(floor);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 m = __hmax2(as_b2(q[i]), f);
        const uint32_t r = *reinterpret_cast<const uint32_t*>(&m);
        add(__uint_as_float(r << 16), __uint_as_float(r & 0xFFFF0000u));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        add(fmaxf(__uint_as_float(q[2 * i]), floor), fmaxf(__uint_as_float(q[2 * i + 1]), floor));
    }
  }
  // Relative to m itself: x c - M = (x - m) c + d with d = m c - M, known exactly.
  __device__ __forceinline__ Sums relative(float m, float c) const {
    float a, b, y, z;
    unpair(s, a, b);
    unpair(w, y, z);
    if (m == -INFINITY) return Sums{m, 0.f, 0.f};
    const float d = fmaf(m, c, -M), f = ex2(-d);
    return Sums{m, (a + b) * f, fmaf(-d, a + b, y + z) * f};
  }
};

struct Partial {   // of one CTA
  float m, s, w;
  int count, bad, ntop;
};

// x / T less lse, from the row's maximum m and log2 of its sum relative to it.
__device__ __forceinline__ float log_prob(float x, float m, float temp, float l2) {
  float d = (x - m) / temp;
  if (d == -INFINITY && x > -INFINITY) d = x / temp - m / temp;   // the difference alone left the range
  return fmaf(-LN2, l2, d);
}

// The lanes' partial results as one, in every lane (a butterfly: the same order always).
__device__ __forceinline__ Partial join(Partial p, float c) {
  float m = p.m;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  Sums b{p.m, p.s, p.w};
  if (p.s > 0.f) b.move(m, c);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    b.s += __shfl_xor_sync(0xffffffffu, b.s, o);
    b.w += __shfl_xor_sync(0xffffffffu, b.w, o);
  }
  return Partial{m, b.s, b.w, (int)__reduce_add_sync(0xffffffffu, (unsigned)p.count),
                 (int)__reduce_or_sync(0xffffffffu, (unsigned)p.bad), (int)__reduce_add_sync(0xffffffffu, (unsigned)p.ntop)};
}

struct Smem {
  float gmax[MAX_GROUPS];
  uint32_t key[MAX_GROUPS];
  unsigned long long cand[MAX_CAND];
  unsigned long long top[MAX_TOP];
  unsigned long long merge[MAX_CLUSTER * MAX_TOP];
  int sel[MAX_SEL];
  Partial warps[NW];
  Partial parts[MAX_CLUSTER];                          // the cluster's, in its first CTA
  uint32_t wmin[NW], wmax[NW];
  int nsel, ncand, cnt[3], bad;
  unsigned long long best[NW];
};

template <typename T>
struct Row {
  const T* x;
  int V, a0, nvec, tail;   // a0 logits before the first 16-byte boundary, tail after the last vector
};

// Element id and value of loose logit i (the a0 + tail ones outside the vectors).
template <typename T>
__device__ __forceinline__ int loose_id(const Row<T>& r, int i) {
  return i < r.a0 ? i : r.V - r.tail + (i - r.a0);
}

__device__ __forceinline__ unsigned long long pack_key(float x, int id) {
  return ((unsigned long long)okey(x) << 32) | (uint32_t)~(uint32_t)id;
}

// The thread's sums of the CTA's vectors [v0, v1) relative to m, every exponent clamped (rare).
template <typename T>
__device__ __noinline__ Sums clamped_sums(const Row<T>& r, int v0, int v1, float m, float c) {
  Sums a{m, 0.f, 0.f};
#pragma unroll 1
  for (int v = v0 + threadIdx.x; v < v1; v += NT) {
    float x[Elem<T>::EPV];
    unpack<T>(*reinterpret_cast<const uint4*>(r.x + r.a0 + (size_t)v * Elem<T>::EPV), x);
#pragma unroll
    for (int i = 0; i < Elem<T>::EPV; ++i) a.add(x[i], c);
  }
  return a;
}

// Logits of the lane's vectors v, v + 32, ... (UNR of them, below v1) that come before
// the token's, id by id: for the waves that hold it, or padding.
template <typename T>
__device__ __noinline__ float count_by_id(const Row<T>& r, int v, int v1, float xt, int tok) {
  float n = 0.f;
#pragma unroll 1
  for (int u = 0; u < UNR; ++u, v += 32) {
    if (v >= v1) break;
    float x[Elem<T>::EPV];
    const int id = r.a0 + v * Elem<T>::EPV;
    unpack<T>(*reinterpret_cast<const uint4*>(r.x + id), x);
#pragma unroll
    for (int i = 0; i < Elem<T>::EPV; ++i) n += x[i] > xt || (x[i] == xt && id + i < tok);
  }
  return n;
}

// The best n (key descending) of the segment's entries [0, G) and, in the first CTA,
// of the loose logits, into S.top (0: none); returns how many there are. An entry is
// the maximum of a group, or (fine) of a vector. All threads take part. The loops are
// kept rolled: this runs once a CTA, and fetching long code costs more than running it.
template <typename T>
__device__ __noinline__ int select_top(Smem& S, const Row<T>& r, int g0, int G, int n, bool loose, bool fine) {
  constexpr int EPV = Elem<T>::EPV;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t kmin = 0xFFFFFFFFu, kmax = 0u;
#pragma unroll 1
  for (int g = tid; g < G; g += NT) {
    const uint32_t k = okey(S.gmax[g]);
    S.key[g] = k;                       // a thread's own entries, also below
    kmin = min(kmin, k);
    kmax = max(kmax, k);
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (tid == 0) S.nsel = S.ncand = S.cnt[0] = S.cnt[1] = S.cnt[2] = 0;
  if (lane == 0) S.wmin[warp] = kmin, S.wmax[warp] = kmax;
  if (tid < MAX_TOP) S.top[tid] = 0ull;
  __syncthreads();
  kmin = __reduce_min_sync(0xffffffffu, S.wmin[lane % NW]);
  kmax = __reduce_max_sync(0xffffffffu, S.wmax[lane % NW]);
  // lo: at least n entries reach it; hi: fewer than n do
  uint32_t lo = kmin, hi = kmax + 1u;
  bool tied = G > n + SEL_EXTRA;
  if (!tied) lo = 0u;
  for (int step = 0; tied && hi - lo > 1u; step = step == 2 ? 0 : step + 1) {
    const uint32_t mid = lo + (hi - lo) / 2u;
    int cnt = 0;
#pragma unroll 1
    for (int g = tid; g < G; g += NT) cnt += S.key[g] >= mid;
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0 && cnt) atomicAdd(&S.cnt[step], cnt);
    __syncthreads();
    cnt = S.cnt[step];
    if (tid == 0) S.cnt[step == 0 ? 2 : step - 1] = 0;   // read by all before this barrier, next used after another
    if (cnt >= n) {
      lo = mid;
      tied = cnt > n + SEL_EXTRA;
    } else {
      hi = mid;
    }
  }
  // a tie: more than n + SEL_EXTRA entries reach lo, and fewer than n exceed it: those,
  // then the lowest entries whose maximum is lo
#pragma unroll 1
  for (int g = tid; g < G; g += NT)
    if (S.key[g] >= lo + (tied ? 1u : 0u)) S.sel[atomicAdd(&S.nsel, 1)] = g;
  __syncthreads();
  if (tied && warp == 0) {
    int have = S.nsel;
    for (int g = lane; g - lane < G && have < n; g += 32) {
      const bool eq = g < G && S.key[g] == lo;
      const unsigned b = __ballot_sync(0xffffffffu, eq);
      const int at = have + __popc(b & ((1u << lane) - 1u));
      if (eq && at < n) S.sel[at] = g;
      have += __popc(b);
    }
    __syncwarp();
    if (lane == 0) S.nsel = min(have, n);
  }
  if (tied) __syncthreads();
  const int nsel = S.nsel;
  const uint32_t least = max(lo, KEY_NEG_INF + 1u);   // -inf is never listed
  // Every logit of the selected entries that is at or above the bound: first listed;
  // if there are too many to be ranked by counting (groups only: rows that rise
  // steadily, long runs of ties), n rounds follow, each for the largest key below the last.
  unsigned long long last = ~0ull;
  int nc = 0;
#pragma unroll 1
  for (int j = -1; j < n; ++j) {
    unsigned long long best = 0ull;
    const int items = fine ? nsel : nsel * 32;
    const auto take = [&](float x, int id) {
      if (okey(x) < least) return;
      const unsigned long long k = pack_key(x, id);
      if (j >= 0) {
        if (k < last && k > best) best = k;
      } else {
        const int at = atomicAdd(&S.ncand, 1);
        if (at < MAX_CAND) S.cand[at] = k;
      }
    };
    constexpr int AHEAD = 4;   // loads on their way at once
#pragma unroll 1
    for (int s0 = tid; s0 < items; s0 += AHEAD * NT) {
      uint4 y[AHEAD];
      int id[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int s = s0 + i * NT;
        id[i] = -1;
        if (s < items) {
          const int v = fine ? g0 * 32 + S.sel[s] : (g0 + S.sel[s >> 5]) * 32 + (s & 31);
          if (v < r.nvec) {
            id[i] = r.a0 + v * EPV;
            y[i] = *reinterpret_cast<const uint4*>(r.x + id[i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (id[i] < 0) continue;
        float top = vec_max<T>(y[i]);
        if (okey(top) < least) continue;
        float x[EPV];
        unpack<T>(y[i], x);
#pragma unroll
        for (int e = 0; e < EPV; ++e) take(x[e], id[i] + e);
      }
    }
    if (loose && tid < r.a0 + r.tail) take(Elem<T>::get(r.x + loose_id(r, tid)), loose_id(r, tid));
    if (j < 0) {
      __syncthreads();
      nc = S.ncand;
      if (nc > MAX_CAND) continue;
      // a warp for each candidate: its place is the number of larger keys
#pragma unroll 1
      for (int c = warp; c < nc; c += NW) {
        const unsigned long long k = S.cand[c];
        int before = 0;
#pragma unroll 1
        for (int i = lane; i < nc; i += 32) before += S.cand[i] > k;
        before = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0 && before < n) S.top[before] = k;
      }
      break;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) S.best[warp] = best;
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < NW; ++w) best = max(best, S.best[w]);
    if (tid == 0) S.top[j] = best;
    last = best;
    __syncthreads();
  }
  __syncthreads();
  return min(nc, n);
}

template <typename T>
__global__ void __launch_bounds__(NT, 1024 / NT)
    logprobs_kernel(const T* __restrict__ logits, int V, long long ld, const int32_t* __restrict__ tokens,
                    const float* __restrict__ temperature, int n, float* __restrict__ logprob,
                    int32_t* __restrict__ rank, float* __restrict__ entropy, float* __restrict__ lse,
                    int32_t* __restrict__ top_ids, float* __restrict__ top_lp) {
  constexpr int EPV = Elem<T>::EPV;
  __shared__ Smem S;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), crank = (int)cl.block_rank();
  const long long row = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tok = tokens[row];
  float temp = temperature ? temperature[row] : 1.f;
  if (temp == 0.f) temp = 1.f;
  const float c = LOG2E / temp;
  if (tok < 0 || tok >= V || !(temp > 0.f) || !(c > 0.f) || isinf(c)) {   // the same for the whole cluster
    if (crank == 0) {
      const float bad = tok < 0 ? 0.f : NAN;
      if (tid == 0) {
        logprob[row] = entropy[row] = lse[row] = bad;
        rank[row] = -1;
      }
      if (tid < n) {
        top_ids[row * n + tid] = -1;
        top_lp[row * n + tid] = bad;
      }
    }
    return;
  }
  if (C > 1) cl.barrier_arrive();   // this CTA runs: its shared memory may be written
  Row<T> r;
  r.x = logits + row * ld;
  r.V = V;
  const uintptr_t addr = reinterpret_cast<uintptr_t>(r.x);
  r.a0 = min((int)(((16 - (addr & 15)) & 15) / sizeof(T)), V);
  r.nvec = (V - r.a0) / EPV;
  r.tail = V - r.a0 - r.nvec * EPV;
  const int groups = (r.nvec + 31) / 32;
  const int per = (groups + C - 1) / C;
  const int g0 = min(crank * per, groups), G = min(per, groups - g0);
  const bool fine = per * 32 <= MAX_GROUPS;   // short segments keep each vector's maximum, long ones each group's

  constexpr int STEP = NW * UNR;
  const int v1 = min((g0 + G) * 32, r.nvec);     // the segment's last vector, past it
  const uint4* const base = reinterpret_cast<const uint4*>(r.x + r.a0);
  uint4 nxt[UNR];
  const auto fetch = [&](int v0) {               // v0: the lane's first vector of the wave
    if (v0 - lane + UNR * 32 <= v1) {
#pragma unroll
      for (int u = 0; u < UNR; ++u) nxt[u] = load_stream(base + v0 + u * 32);
    } else {
#pragma unroll
      for (int u = 0; u < UNR; ++u) nxt[u] = v0 + u * 32 < v1 ? load_stream(base + v0 + u * 32) : none_vec<T>();
    }
  };
  fetch((g0 + warp * UNR) * 32 + lane);          // ahead of the token's own logit
  const float xt = Elem<T>::get(r.x + tok);
  const float thr_after = succ<T>(xt);

  PairSums acc;
  float m = -INFINITY, count = 0.f;
  bool bad = false;
#pragma unroll 1
  for (int g = warp * UNR; g < G; g += STEP) {   // a wave: groups g .. g + UNR - 1
    const int v0 = (g0 + g) * 32 + lane;
    const bool whole = v0 - lane + UNR * 32 <= v1;
    uint4 v[UNR];
#pragma unroll
    for (int u = 0; u < UNR; ++u) v[u] = nxt[u];
    if (g + STEP < G) fetch(v0 + STEP * 32);
    float wm = -INFINITY;
    if (n > 0 && !fine) {
      float mine = -INFINITY;
#pragma unroll
      for (int u = 0; u < UNR; ++u) {
        const float x = warp_max_nan(vec_max<T>(v[u]));
        wm = max_nan(wm, x);
        mine = lane == u ? x : mine;
      }
      if (lane < UNR && g + lane < G) S.gmax[g + lane] = mine;
    } else {
#pragma unroll
      for (int u = 0; u < UNR; ++u) {
        const float x = vec_max<T>(v[u]);
        wm = max_nan(wm, x);
        if (n > 0 && g + u < G) S.gmax[(g + u) * 32 + lane] = x;
      }
      wm = warp_max_nan(wm);
    }
    bad |= !(wm < INFINITY);   // NaN or +inf: the row's numbers do not matter any more
    if (wm > m) {
      m = wm;
      acc.move<T>(m, c);
    }
    if (fmaf(wm, c, -acc.M) > -160.f) {   // else every weight is 0 in fp32 (or nothing but -inf so far)
#pragma unroll
      for (int u = 0; u < UNR; ++u) acc.add<T>(v[u]);
    }
    if (wm < xt) continue;     // nothing here comes before the token
    // padding would count beside a -inf token, so a wave that holds it goes id by id
    const int id0 = r.a0 + (v0 - lane) * EPV;
    if (whole && (unsigned)(tok - id0) >= (unsigned)(UNR * 32 * EPV))
      count += count_ge<T>(v, id0 > tok ? thr_after : xt);
    else
      count += count_by_id<T>(r, v0, v1, xt, tok);
  }
  Sums a = acc.relative(m, c);
  if (__syncthreads_or(acc.off)) {   // logits near the type's lowest value: once more, clamped
    if (lane == 0) S.warps[warp].m = m;
    __syncthreads();
    for (int w = 0; w < NW; ++w) m = fmaxf(m, S.warps[w].m);
    __syncthreads();
    a = m > -INFINITY && m < INFINITY ? clamped_sums(r, g0 * 32, v1, m, c) : Sums{m, 0.f, 0.f};
  }
  if (crank == 0 && warp == 0) {
    const int nl = r.a0 + r.tail;
    float x = -INFINITY;
    if (lane < nl) {
      x = Elem<T>::get(r.x + loose_id(r, lane));
      const int id = loose_id(r, lane);
      count += x > xt || (x == xt && id < tok);
    }
    const float wm = warp_max_nan(x);
    if (!(wm < INFINITY)) bad = true;
    if (!bad && wm > m) {
      m = wm;
      a.move(m, c);
    }
    if (!bad && m > -INFINITY && lane < nl) a.add(x, c);
  }
  // the warp's sums, then the CTA's, in a fixed order
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
  }
  const int wcount = __reduce_add_sync(0xffffffffu, (int)count);
  if (lane == 0)
    S.warps[warp] = Partial{m, a.s, a.w, wcount, bad, 0};
  __syncthreads();
  if (C > 1) cl.barrier_wait();
  if (warp == 0) {
    Partial p = lane < NW ? S.warps[lane] : Partial{-INFINITY, 0.f, 0.f, 0, 0, 0};
    p = join(p, c);
    if (lane == 0) {
      S.bad = p.bad;
      *cl.map_shared_rank(&S.parts[crank], 0) = p;
    }
  }
  if (n > 0) {
    __syncthreads();
    int nt = 0;
    if (!S.bad) nt = select_top<T>(S, r, g0, fine ? min(G * 32, r.nvec - g0 * 32) : G, n, crank == 0, fine);
    if (tid < nt) *cl.map_shared_rank(&S.merge[crank * MAX_TOP + tid], 0) = S.top[tid];
    if (tid == 0) cl.map_shared_rank(&S.parts[crank], 0)->ntop = nt;
  }
  if (C > 1)
    cl.sync();
  else
    __syncthreads();
  if (crank != 0) return;
  // the first CTA puts the cluster together
  const Partial p = join(lane < C ? S.parts[lane] : Partial{-INFINITY, 0.f, 0.f, 0, 0, 0}, c);
  const float l2 = log2f(p.s);
  const bool none = p.bad || !(p.s > 0.f);
  if (tid == 0) {
    logprob[row] = none ? NAN : log_prob(xt, p.m, temp, l2);
    entropy[row] = none ? NAN : fmaxf(LN2 * (l2 - p.w / p.s), 0.f);
    lse[row] = none ? NAN : p.m / temp + LN2 * l2;
    rank[row] = none ? -1 : p.count;
  }
  if (n == 0) return;
  const int total = none ? 0 : p.ntop;
  if (tid < n && tid >= total) {   // places past the last finite logit
    top_ids[row * n + tid] = -1;
    top_lp[row * n + tid] = none ? NAN : -INFINITY;
  }
  // a warp for each list, a lane for each token: its place is its place in its own list and, in each
  // of the others (sorted, all keys different), the number of larger keys
  for (int list = warp; list < C && !none; list += NW) {
    const int i = lane;
    if (i >= S.parts[list].ntop) continue;
    const unsigned long long k = S.merge[list * MAX_TOP + i];
    int at = i;
    for (int j = 0; j < C; ++j) {
      if (j == list) continue;
      int lo = 0, hi = S.parts[j].ntop;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (S.merge[j * MAX_TOP + mid] > k)
          lo = mid + 1;
        else
          hi = mid;
      }
      at += lo;
    }
    if (at < n) {
      top_ids[row * n + at] = (int)~(uint32_t)k;
      top_lp[row * n + at] = log_prob(okey_value((uint32_t)(k >> 32)), p.m, temp, l2);
    }
  }
}

// --- gradient ----------------------------------------------------------------

constexpr int BT = 256;      // threads
constexpr int BU = 8;        // vectors a thread has in flight: 49 us for 512 rows of 151,936 bf16, with four 51, with two 62
constexpr int MAX_FIX = MAX_TOP + 1;

struct Coef {
  float chi, clo, lhi, llo;   // c = log2(e)/T and lse log2(e), as two floats each
  float k0, k1;               // dx = p (k0 + k1 u), u = log2 p
};

// Two logits at a time.
__device__ __forceinline__ void grad_at(float& x0, float& x1, const Coef& f) {
  const uint64_t x = pair(x0, x1);
  float a, b;
  unpair(add2(fma2(x, pair(f.chi, f.chi), pair(-f.lhi, -f.lhi)), fma2(x, pair(f.clo, f.clo), pair(-f.llo, -f.llo))), a, b);
  a = fmaxf(a, U_MIN), b = fmaxf(b, U_MIN);
  const uint64_t k = fma2(pair(f.k1, f.k1), pair(a, b), pair(f.k0, f.k0));
  unpair(mul2(pair(ex2(a), ex2(b)), k), x0, x1);
}

// An lse of 32 bits is known to 2^-25 of its size at best, and so would every probability
// be that is formed from it. Up to here that is 2^-19, about what the forward's sum is good to;
// rows past it (low temperatures, logits far from zero) find their maximum and sum again.
constexpr float FAR_LSE = 64.f;
// CTAs that such rows are spread over, at least one a row and at most as many as it has chunks: more
// read each row more often, fewer leave SMs idle (rows of 151,936 bf16, all past FAR_LSE: 2 rows 19
// us, 130 rows 62, 512 rows 154, against 49 if none is; with 1,216 CTAs 130 rows a quarter longer).
constexpr int FAR_CTAS = 4 * SMS;

// f(logit) for the elements [e0, e1) of a row, four 16-byte loads of a thread on their way.
// Elements of vectors that are not there are -inf.
template <typename T, typename F>
__device__ __forceinline__ void over_row(const T* x, int e0, int e1, F&& f) {
  constexpr int EPV = Elem<T>::EPV, U = 4;
  const int tid = threadIdx.x;
  const int a0 = min((int)(((16 - (reinterpret_cast<uintptr_t>(x + e0) & 15)) & 15) / sizeof(T)), e1 - e0);
  const int nvec = (e1 - e0 - a0) / EPV, loose = e1 - e0 - nvec * EPV;
#pragma unroll 1
  for (int i = tid; i < nvec; i += U * BT) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = i + u * BT < nvec ? *reinterpret_cast<const uint4*>(x + e0 + a0 + (i + u * BT) * EPV) : none_vec<T>();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float z[EPV];
      unpack<T>(v[u], z);
#pragma unroll
      for (int j = 0; j < EPV; ++j) f(z[j]);
    }
  }
  if (tid < loose) f(Elem<T>::get(x + e0 + (tid < a0 ? tid : nvec * EPV + tid)));
}

// A row past FAR_LSE: each of `parts` CTAs reads all of it and writes its part. A gradient that
// takes the logits' place has one part: all is read before anything is written.
template <typename T>
__device__ __noinline__ void far_part(const T* x, T* y, int V, int part, int parts, int tok, float temp, float gl,
                                      float gh, float H, int n, const int32_t* ids, const float* gtop) {
  constexpr int EPV = Elem<T>::EPV;
  __shared__ float warps[BT / 32];
  __shared__ int fix_id[MAX_FIX];
  __shared__ float fix_g[MAX_FIX];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float c = LOG2E / temp;
  if (tid <= n) {
    fix_id[tid] = tid < n ? ids[tid] : tok;
    fix_g[tid] = tid < n ? gtop[tid] : gl;
  }
  float m = -INFINITY, s = 0.f, sum = 0.f;
  over_row<T>(x, 0, V, [&](float z) { m = fmaxf(m, z); });
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) warps[warp] = m;
  __syncthreads();
#pragma unroll 1
  for (int w = 0; w < BT / 32; ++w) m = fmaxf(m, warps[w]);
  over_row<T>(x, 0, V, [&](float z) { s += ex2(fmaxf((z - m) * c, U_MIN)); });
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if (lane == 0) warps[warp] = s;
  // the logits of the token and the alternatives, before they may be written over
  const int id = tid <= n ? fix_id[tid] : -1;
  const float xs = id >= 0 && id < V ? Elem<T>::get(x + id) : 0.f;
  __syncthreads();
  s = 0.f;
#pragma unroll 1
  for (int w = 0; w < BT / 32; ++w) s += warps[w];
  const float l2 = log2f(s);
#pragma unroll 1
  for (int k = 0; k <= n; ++k)
    if (fix_id[k] >= 0 && fix_id[k] < V) sum += fix_g[k];
  const float k0 = sum + gh * H, k1 = gh * LN2;
  const auto at = [&](float z, float up) {
    const float u = fmaxf((z - m) * c, U_MIN) - l2;
    return (up - ex2(u) * fmaf(k1, u, k0)) / temp;
  };
  const int b0 = (int)((long long)V * part / parts) & ~63, b1 = part + 1 == parts ? V : (int)((long long)V * (part + 1) / parts) & ~63;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x + b0), ya = reinterpret_cast<uintptr_t>(y + b0);
  const int a0 = min((int)(((16 - (xa & 15)) & 15) / sizeof(T)), b1 - b0);
  const int nvec = ((xa ^ ya) & 15) == 0 ? (b1 - b0 - a0) / EPV : 0, loose = b1 - b0 - nvec * EPV;
#pragma unroll 1
  for (int i = tid; i < nvec; i += BT) {
    float z[EPV];
    unpack<T>(*reinterpret_cast<const uint4*>(x + b0 + a0 + i * EPV), z);
#pragma unroll
    for (int j = 0; j < EPV; ++j) z[j] = at(z[j], 0.f);
    uint4 o;
    if (sizeof(T) == 2) {
      __nv_bfloat162 b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = __floats2bfloat162_rn(z[2 * j % EPV], z[(2 * j + 1) % EPV]);
      o = *reinterpret_cast<uint4*>(b);
    } else {
      o = make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
    }
    *reinterpret_cast<uint4*>(y + b0 + a0 + i * EPV) = o;
  }
#pragma unroll 1
  for (int i = tid; i < loose; i += BT) {
    const int e = b0 + (i < a0 ? i : nvec * EPV + i);
    y[e] = Elem<T>::put(at(Elem<T>::get(x + e), 0.f));
  }
  __syncthreads();
  if (id >= b0 && id < b1) {   // one thread for each place that has a gradient of its own
    float up = 0.f;
    bool first = true;
#pragma unroll 1
    for (int k = 0; k <= n; ++k)
      if (fix_id[k] == id) {
        up += fix_g[k];
        first &= k >= tid;
      }
    if (first) y[id] = Elem<T>::put(at(xs, up));
  }
}

template <typename T>
__global__ void __launch_bounds__(BT, 1024 / BT)   // the rare path may not cost the other one a block on an SM
    logprobs_grad_kernel(const T* logits, int V, long long ld, const int32_t* __restrict__ tokens,
                         const float* __restrict__ temperature, const float* __restrict__ lse,
                         const float* __restrict__ entropy, const float* __restrict__ grad_lp,
                         const float* __restrict__ grad_h, int n, const int32_t* __restrict__ top_ids,
                         const float* __restrict__ grad_top, T* grad, long long gld, int chunks, int far_parts) {
  constexpr int EPV = Elem<T>::EPV;
  constexpr int CHUNK = BT * BU * EPV;
  __shared__ int fix_id[MAX_FIX];
  __shared__ float fix_g[MAX_FIX];
  __shared__ int nfix;
  __shared__ Coef coef;
  __shared__ float fill;   // what a row without a gradient gets: 0, or NaN for a data error
  __shared__ bool far;     // past FAR_LSE
  const long long row = blockIdx.x / chunks;
  const int e0 = (int)(blockIdx.x % chunks) * CHUNK;   // the chunk's first element
  const int tid = threadIdx.x;
  const T* x = logits + row * ld;
  T* y = grad + row * gld;
  const int e1 = min(V, e0 + CHUNK);
  const int tok = tokens[row];
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x + e0), ya = reinterpret_cast<uintptr_t>(y + e0);
  const bool alike = ((xa ^ ya) & 15) == 0;   // else element by element
  const int a0 = min((int)(((16 - (xa & 15)) & 15) / sizeof(T)), e1 - e0);
  const int nvec = alike ? (e1 - e0 - a0) / EPV : 0;
  uint4 v[BU];
#pragma unroll
  for (int u = 0; u < BU; ++u) {
    const int i = u * BT + tid;
    if (i < nvec && tok >= 0) v[u] = *reinterpret_cast<const uint4*>(x + e0 + a0 + i * EPV);
  }
  if (tid < 32) {   // the row's coefficients, and the places of t and the top ids in this chunk
    float temp = temperature ? temperature[row] : 1.f;
    if (temp == 0.f) temp = 1.f;
    const float L = lse[row], gl = grad_lp ? grad_lp[row] : 0.f, gh = grad_h ? grad_h[row] : 0.f, H = entropy[row];
    const int id = tid < n ? top_ids[row * n + tid] : -1;
    const float g = tid < n && id >= 0 && id < V ? grad_top[row * n + tid] : 0.f;
    float sum = g;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const bool here = id >= e0 && id < e1;
    const unsigned b = __ballot_sync(0xffffffffu, here);
    const int at = __popc(b & ((1u << tid) - 1u));
    if (here) {
      fix_id[at] = id;
      fix_g[at] = g / temp;
    }
    if (tid == 0) {
      const bool ok = tok >= 0 && fabsf(L) < INFINITY;
      int k = __popc(b);
      if (gl != 0.f && tok >= e0 && tok < e1) {
        fix_id[k] = tok;
        fix_g[k++] = gl / temp;
      }
      nfix = ok ? k : 0;
      fill = tok < 0 ? 0.f : NAN;
      Coef f{};
      // Two-float products: |x c| reaches tens, and the rounding of one float there
      // would be an error of 1e-6 in every probability. Without a gradient the
      // coefficients make every element `fill`.
      f.chi = LOG2E / temp;
      f.clo = (fmaf(-f.chi, temp, LOG2E) + LOG2E_LO) / temp;
      f.lhi = L * LOG2E;
      f.llo = fmaf(L, LOG2E, -f.lhi) + L * LOG2E_LO;
      f.k0 = -(gl + sum + gh * H) / temp;
      f.k1 = -gh * LN2 / temp;
      if (!ok) f.chi = NAN;
      far = tok >= 0 && tok < V && fabsf(L) > FAR_LSE;
      coef = f;
    }
  }
  __syncthreads();
  if (far) {
    const int part = (int)(blockIdx.x % chunks);
    if (part < far_parts) {
      float temp = temperature ? temperature[row] : 1.f;
      if (temp == 0.f) temp = 1.f;
      far_part<T>(x, y, V, part, far_parts, tok, temp, grad_lp ? grad_lp[row] : 0.f, grad_h ? grad_h[row] : 0.f,
                  entropy[row], n, top_ids + row * n, grad_top + row * n);
    }
    return;
  }
  const int nf = nfix;
  const Coef f = coef;
  const bool none = f.chi != f.chi;
  const float blank = fill;
  const auto one = [&](int id) {
    float d = blank, unused = 0.f;
    if (!none) {
      d = Elem<T>::get(x + id);
      grad_at(d, unused, f);
      for (int k = 0; k < nf; ++k)
        if (fix_id[k] == id) d += fix_g[k];
    }
    y[id] = Elem<T>::put(d);
  };
  if (!alike) {
#pragma unroll 1
    for (int id = e0 + tid; id < e1; id += BT) one(id);
    return;
  }
  const int loose = e1 - e0 - nvec * EPV;   // a0 before the vectors, the rest after them
  if (tid < loose) one(tid < a0 ? e0 + tid : e0 + nvec * EPV + tid);
#pragma unroll
  for (int u = 0; u < BU; ++u) {
    const int i = u * BT + tid;
    if (i >= nvec) break;
    const int id = e0 + a0 + i * EPV;
    float z[EPV];
    if (none) {
#pragma unroll
      for (int j = 0; j < EPV; ++j) z[j] = blank;
    } else {
      unpack<T>(v[u], z);
#pragma unroll
      for (int j = 0; j < EPV; j += 2) grad_at(z[j], z[j + 1], f);
      for (int k = 0; k < nf; ++k) {
        const int at = fix_id[k] - id;
        if ((unsigned)at < (unsigned)EPV) {
#pragma unroll
          for (int j = 0; j < EPV; ++j)
            if (at == j) z[j] += fix_g[k];
        }
      }
    }
    uint4 o;
    if (sizeof(T) == 2) {
      __nv_bfloat162 b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = __floats2bfloat162_rn(z[2 * j % EPV], z[(2 * j + 1) % EPV]);
      o = *reinterpret_cast<uint4*>(b);
    } else {
      o = make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
    }
    *reinterpret_cast<uint4*>(y + id) = o;
  }
}

static bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// CTAs a row is spread over: as many as give every SM two, while each still has a wave
// of groups to stream. More would cost more than they balance: a CTA spends 4 us on its
// start, its alternatives and its share of the join (rows of 151,936 with 20
// alternatives: 320 rows 36 us with one CTA a row, 40 with two, 50 with four; 100 rows 21
// with two, 19 with four, 30 with eight; 40 rows 16 with four, 17 with eight).
static int cluster_size(int R, int V, int epv) {
  const int groups = (V / epv + 31) / 32;
  int c = 1;
  while (c < MAX_CLUSTER && (long long)R * c < 2 * SMS && groups >= c * NW * UNR) c *= 2;
  return c;
}

template <typename T>
static sv_status forward(const void* logits, int R, int V, long long ld, const int32_t* tokens, const float* temp,
                         int n, float* lp, int32_t* rank, float* ent, float* lse, int32_t* ids, float* tlp,
                         cudaStream_t st) {
  const int C = cluster_size(R, V, Elem<T>::EPV);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)R * (unsigned)C);
  cfg.blockDim = dim3(NT);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, static_cast<const T*>(logits), V, ld, tokens,
                                           temp, n, lp, rank, ent, lse, ids, tlp);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

template <typename T>
static sv_status backward(const void* logits, int R, int V, long long ld, const int32_t* tokens, const float* temp,
                          const float* lse, const float* ent, const float* glp, const float* gh, int n,
                          const int32_t* ids, const float* gtop, void* grad, long long gld, cudaStream_t st) {
  const int chunk = BT * BU * Elem<T>::EPV;
  const int chunks = (V + chunk - 1) / chunk;
  const long long blocks = (long long)R * chunks;
  if (blocks > 2147483647LL) return SV_ERR_SHAPE;
  // Parts of a row past FAR_LSE: more read the row more often, fewer leave SMs idle.
  const int far_parts = logits == grad || R >= FAR_CTAS ? 1 : FAR_CTAS / R < chunks ? FAR_CTAS / R : chunks;
  logprobs_grad_kernel<T><<<(unsigned)blocks, BT, 0, st>>>(static_cast<const T*>(logits), V, ld, tokens, temp, lse,
                                                          ent, glp, gh, n, ids, gtop, static_cast<T*>(grad), gld,
                                                          chunks, far_parts);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

static bool bad_shape(int R, int V, long long ld, int n) {
  return R < 1 || R > (1 << 24) || V < 2 || V > 262144 || (ld < V && ld != 0) || n < 0 || n > MAX_TOP;
}

}  // namespace svlp

sv_status spec_token_logprobs(const void* logits, sv_dtype dtype, int R, int V, long long row_stride,
                              const int32_t* tokens, const float* temperature, int top_n, float* logprob,
                              int32_t* rank, float* entropy, float* lse, int32_t* top_ids, float* top_logprobs,
                              void* stream) {
  using namespace svlp;
  if (!logits || !tokens || !logprob || !rank || !entropy || !lse) return SV_ERR_NULL;
  if (top_n > 0 && (!top_ids || !top_logprobs)) return SV_ERR_NULL;
  if (bad_shape(R, V, row_stride, top_n)) return SV_ERR_SHAPE;
  if (dtype != SV_BF16 && dtype != SV_F32) return SV_ERR_DTYPE;
  if (!aligned(logits, dtype == SV_BF16 ? 2 : 4) || !aligned(tokens, 4) || !aligned(temperature, 4) ||
      !aligned(logprob, 4) || !aligned(rank, 4) || !aligned(entropy, 4) || !aligned(lse, 4) ||
      !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
    return SV_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == SV_BF16
             ? forward<__nv_bfloat16>(logits, R, V, row_stride, tokens, temperature, top_n, logprob, rank, entropy,
                                      lse, top_ids, top_logprobs, st)
             : forward<float>(logits, R, V, row_stride, tokens, temperature, top_n, logprob, rank, entropy, lse,
                              top_ids, top_logprobs, st);
}

sv_status spec_token_logprobs_backward(const void* logits, sv_dtype dtype, int R, int V, long long row_stride,
                                       const int32_t* tokens, const float* temperature, const float* lse,
                                       const float* entropy, const float* grad_logprob, const float* grad_entropy,
                                       int top_n, const int32_t* top_ids, const float* grad_top, void* grad_logits,
                                       long long grad_stride, void* stream) {
  using namespace svlp;
  if (!logits || !tokens || !lse || !entropy || !grad_logits) return SV_ERR_NULL;
  if (top_n > 0 && (!top_ids || !grad_top)) return SV_ERR_NULL;
  if (bad_shape(R, V, row_stride, top_n) || grad_stride < V) return SV_ERR_SHAPE;
  if (logits == grad_logits && row_stride != grad_stride) return SV_ERR_SHAPE;
  if (dtype != SV_BF16 && dtype != SV_F32) return SV_ERR_DTYPE;
  const uintptr_t es = dtype == SV_BF16 ? 2 : 4;
  if (!aligned(logits, es) || !aligned(grad_logits, es) || !aligned(tokens, 4) || !aligned(temperature, 4) ||
      !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(grad_logprob, 4) || !aligned(grad_entropy, 4) ||
      !aligned(top_ids, 4) || !aligned(grad_top, 4))
    return SV_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == SV_BF16
             ? backward<__nv_bfloat16>(logits, R, V, row_stride, tokens, temperature, lse, entropy, grad_logprob,
                                       grad_entropy, top_n, top_ids, grad_top, grad_logits, grad_stride, st)
             : backward<float>(logits, R, V, row_stride, tokens, temperature, lse, entropy, grad_logprob,
                               grad_entropy, top_n, top_ids, grad_top, grad_logits, grad_stride, st);
}

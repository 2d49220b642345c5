// Token log-probabilities over logit rows, and their gradient (C ABI and
// definitions in include/spec_logprobs.h).
//
// Forward: one cluster of C CTAs per row, each CTA a contiguous segment of it. One
// pass over the segment: a warp takes groups of 32 consecutive 16-byte vectors
// (256 bf16 or 128 fp32 logits), four groups a wave, the next wave's loads in
// flight while the current one is reduced. Per wave it needs
//   - each group's maximum (a warp reduction), kept in shared memory;
//   - the online softmax sums, in the warp's own frame M = fl(m c), c = log2(e)/T:
//     s = sum 2^(x c - M) and w = sum 2^(x c - M) (x c - M). Every exponent is one
//     fused multiply-add, so lse = ln2 (M + log2 s) and H = ln2 (log2 s - w / s)
//     hold for the frame as it was rounded;
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
// are listed in shared memory and added before the one rounding.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/spec_logprobs.h"

namespace cg = cooperative_groups;

namespace svlp {

constexpr int NT = 512, NW = NT / 32;
constexpr int UNR = 4;                 // groups a warp loads at once
constexpr int MAX_TOP = SV_LOGPROBS_MAX_TOP;
constexpr int MAX_GROUPS = 2048;       // 262,144 fp32 logits in groups of 128
constexpr int SEL_EXTRA = 16;          // the bisection stops at n..n+SEL_EXTRA groups
constexpr int MAX_SEL = MAX_TOP + SEL_EXTRA;
constexpr int MAX_CAND = NT;           // candidates ranked by counting
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

// Logits of the vector that are >= thr, as a float.
template <typename T>
__device__ __forceinline__ float count_ge(const uint4& v, float thr) {
  if (sizeof(T) == 2) {
    const __nv_bfloat162 t = __float2bfloat162_rn(thr);   // exact: thr is a value of the type
    const __nv_bfloat162 a = __hadd2(__hadd2(__hge2(as_b2(v.x), t), __hge2(as_b2(v.y), t)),
                                     __hadd2(__hge2(as_b2(v.z), t), __hge2(as_b2(v.w), t)));
    return __low2float(a) + __high2float(a);
  }
  float x[4];
  unpack<float>(v, x);
  return (float)((x[0] >= thr) + (x[1] >= thr) + (x[2] >= thr) + (x[3] >= thr));
}

// Softmax sums in the frame M (s and w as above); m is the maximum they have seen.
struct Sums {
  float M, s, w;
  __device__ __forceinline__ void add(float x, float c) {
    const float u = fmaxf(fmaf(x, c, -M), U_MIN);
    const float e = ex2(u);
    s += e;
    w = fmaf(e, u, w);
  }
  // the same sums in the frame M2 >= M
  __device__ __forceinline__ void move(float M2) {
    if (M == M2) return;
    const float d = fmaxf(M - M2, U_MIN);
    const float f = s > 0.f ? ex2(d) : 0.f;
    w = f * fmaf(s, d, w);
    s = f * s;
    M = M2;
  }
};

struct Partial {   // of one CTA
  float M, s, w;
  int count, bad, any;
};

struct Smem {
  float gmax[MAX_GROUPS];
  unsigned long long cand[MAX_CAND];
  unsigned long long top[MAX_TOP];
  unsigned long long merge[MAX_CLUSTER * MAX_TOP];
  int sel[MAX_SEL];
  float wM[NW], ws[NW], ww[NW];
  int wcount[NW], wbad[NW];
  uint32_t wmin[NW], wmax[NW];
  int nsel, ncand;
  Partial part;
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

// The best n (key descending) of the segment's groups [g0, g0 + G) and, in the first
// CTA, of the loose logits, into S.top (0: none). All threads take part.
template <typename T>
__device__ void select_top(Smem& S, const Row<T>& r, int g0, int G, int n, bool loose) {
  constexpr int EPV = Elem<T>::EPV;
  constexpr int SLOTS = MAX_GROUPS / NT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) S.nsel = S.ncand = 0;
  uint32_t key[SLOTS], kmin = 0xFFFFFFFFu, kmax = 0u;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int g = i * NT + tid;
    key[i] = g < G ? okey(S.gmax[g]) : 0u;   // 0 lies below every key
    if (g < G) {
      kmin = min(kmin, key[i]);
      kmax = max(kmax, key[i]);
    }
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (lane == 0) {
    S.wmin[warp] = kmin;
    S.wmax[warp] = kmax;
  }
  __syncthreads();
  for (int w = 0; w < NW; ++w) {
    kmin = min(kmin, S.wmin[w]);
    kmax = max(kmax, S.wmax[w]);
  }
  // lo: at least n groups reach it; hi: fewer than n do
  uint32_t lo = kmin, hi = kmax + 1u;
  bool tied = G > n + SEL_EXTRA;
  if (!tied) lo = 0u;
  while (tied && hi - lo > 1u) {
    const uint32_t mid = lo + (hi - lo) / 2u;
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (i * NT < G) cnt += __syncthreads_count(key[i] >= mid);
    if (cnt >= n) {
      lo = mid;
      tied = cnt > n + SEL_EXTRA;
    } else {
      hi = mid;
    }
  }
  if (tied) {
    // more than n + SEL_EXTRA groups reach lo, and fewer than n exceed it: those,
    // then the lowest groups whose maximum is lo
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (key[i] > lo) S.sel[atomicAdd(&S.nsel, 1)] = i * NT + tid;
    __syncthreads();
    if (warp == 0) {
      int have = S.nsel;
      for (int g = lane; g - lane < G && have < n; g += 32) {
        const bool eq = g < G && okey(S.gmax[g]) == lo;
        const unsigned b = __ballot_sync(0xffffffffu, eq);
        const int at = have + __popc(b & ((1u << lane) - 1u));
        if (eq && at < n) S.sel[at] = g;
        have += __popc(b);
      }
      if (lane == 0) S.nsel = min(have, n);
    }
  } else {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (i * NT + tid < G && key[i] >= lo) S.sel[atomicAdd(&S.nsel, 1)] = i * NT + tid;
  }
  __syncthreads();
  const int nsel = S.nsel;
  const uint32_t least = max(lo, KEY_NEG_INF + 1u);   // -inf is never listed
  const int nloose = loose ? r.a0 + r.tail : 0;
  const auto push = [&](float x, int id) {
    if (okey(x) < least) return;
    const int at = atomicAdd(&S.ncand, 1);
    if (at < MAX_CAND) S.cand[at] = pack_key(x, id);
  };
  for (int s = warp; s < nsel; s += NW) {
    const int v = (g0 + S.sel[s]) * 32 + lane;
    if (v < r.nvec) {
      float x[EPV];
      const int id = r.a0 + v * EPV;
      unpack<T>(*reinterpret_cast<const uint4*>(r.x + id), x);
#pragma unroll
      for (int i = 0; i < EPV; ++i) push(x[i], id + i);
    }
  }
  if (tid < nloose) push(Elem<T>::get(r.x + loose_id(r, tid)), loose_id(r, tid));
  if (tid < MAX_TOP) S.top[tid] = 0ull;
  __syncthreads();
  const int nc = S.ncand;
  if (nc <= MAX_CAND) {
    if (tid < nc) {
      const unsigned long long k = S.cand[tid];
      int before = 0;
      for (int i = 0; i < nc; ++i) before += S.cand[i] > k;
      if (before < n) S.top[before] = k;
    }
    __syncthreads();
    return;
  }
  // more logits at or above the bound than are ranked by counting (rows that rise
  // steadily, long runs of ties): n rounds, each the largest key below the last
  unsigned long long last = ~0ull;
  for (int j = 0; j < n; ++j) {
    unsigned long long best = 0ull;
    const auto take = [&](float x, int id) {
      const unsigned long long k = pack_key(x, id);
      if (okey(x) >= least && k < last && k > best) best = k;
    };
    for (int s = warp; s < nsel; s += NW) {
      const int v = (g0 + S.sel[s]) * 32 + lane;
      if (v < r.nvec) {
        float x[EPV];
        const int id = r.a0 + v * EPV;
        unpack<T>(*reinterpret_cast<const uint4*>(r.x + id), x);
#pragma unroll
        for (int i = 0; i < EPV; ++i) take(x[i], id + i);
      }
    }
    if (tid < nloose) take(Elem<T>::get(r.x + loose_id(r, tid)), loose_id(r, tid));
#pragma unroll
    for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) S.best[warp] = best;
    __syncthreads();
    for (int w = 0; w < NW; ++w) best = max(best, S.best[w]);
    if (tid == 0) S.top[j] = best;
    last = best;
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(NT, 2)
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

  const float xt = Elem<T>::get(r.x + tok);
  const float thr_after = succ<T>(xt);

  Sums a{-INFINITY, 0.f, 0.f};
  float m = -INFINITY, count = 0.f;
  bool bad = false;
  uint4 nxt[UNR];
  const auto fetch = [&](int g) {
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      const int v = (g0 + g + u) * 32 + lane;
      nxt[u] = g + u < G && v < r.nvec ? load_stream(r.x + r.a0 + (size_t)v * EPV) : none_vec<T>();
    }
  };
  int g = warp * UNR;
  if (g < G) fetch(g);
  for (; g < G; g += NW * UNR) {
    uint4 cur[UNR];
#pragma unroll
    for (int u = 0; u < UNR; ++u) cur[u] = nxt[u];
    if (g + NW * UNR < G) fetch(g + NW * UNR);
    float wm = -INFINITY, gm[UNR];
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      gm[u] = warp_max_nan(vec_max<T>(cur[u]));
      wm = max_nan(wm, gm[u]);
    }
#pragma unroll
    for (int u = 0; u < UNR; ++u)
      if (lane == u && g + u < G) S.gmax[g + u] = gm[u];
    if (!(wm < INFINITY)) {   // NaN or +inf
      bad = true;
      break;
    }
    if (wm > m) {
      m = wm;
      a.move(m * c);
    }
    const bool live = m > -INFINITY;   // else nothing but -inf so far
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      float x[EPV];
      unpack<T>(cur[u], x);
#pragma unroll
      for (int i = 0; i < EPV; ++i)
        if (live) a.add(x[i], c);
      const int v = (g0 + g + u) * 32 + lane, id = r.a0 + v * EPV;
      if (g + u >= G || v >= r.nvec) continue;   // padding: would count beside a -inf token
      if (id + EPV <= tok || id > tok) {
        count += count_ge<T>(cur[u], id > tok ? thr_after : xt);
      } else {
#pragma unroll
        for (int i = 0; i < EPV; ++i) count += x[i] > xt || (x[i] == xt && id + i < tok);
      }
    }
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
      a.move(m * c);
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
  if (lane == 0) {
    S.wM[warp] = a.M;
    S.ws[warp] = a.s;
    S.ww[warp] = a.w;
    S.wcount[warp] = wcount;
    S.wbad[warp] = bad || isinf(a.M) != (m == -INFINITY) || a.M == INFINITY;
  }
  __syncthreads();
  if (tid == 0) {
    Partial p{-INFINITY, 0.f, 0.f, 0, 0, 0};
    for (int w = 0; w < NW; ++w) {
      p.M = fmaxf(p.M, S.wM[w]);
      p.count += S.wcount[w];
      p.bad |= S.wbad[w];
    }
    for (int w = 0; w < NW; ++w) {
      Sums b{S.wM[w], S.ws[w], S.ww[w]};
      if (b.s > 0.f) {
        b.move(p.M);
        p.s += b.s;
        p.w += b.w;
      }
    }
    S.part = p;
  }
  __syncthreads();
  if (n > 0 && !S.part.bad) select_top<T>(S, r, g0, G, n, crank == 0);
  if (C > 1) cl.sync();
  if (crank == 0) {
    Partial p = S.part;
    if (C > 1) {
      for (int k = 1; k < C; ++k) {
        const Partial* q = cl.map_shared_rank(&S.part, k);
        p.M = fmaxf(p.M, q->M);
        p.count += q->count;
        p.bad |= q->bad;
      }
      p.s = p.w = 0.f;
      for (int k = 0; k < C; ++k) {
        const Partial* q = cl.map_shared_rank(&S.part, k);
        Sums b{q->M, q->s, q->w};
        if (b.s > 0.f) {
          b.move(p.M);
          p.s += b.s;
          p.w += b.w;
        }
      }
    }
    const bool none = p.bad || !(p.s > 0.f);
    const float l2 = log2f(p.s);
    if (tid == 0) {
      logprob[row] = none ? NAN : LN2 * (fmaf(xt, c, -p.M) - l2);
      entropy[row] = none ? NAN : fmaxf(LN2 * (l2 - p.w / p.s), 0.f);
      lse[row] = none ? NAN : LN2 * (p.M + l2);
      rank[row] = none ? -1 : p.count;
    }
    if (n > 0) {
      unsigned long long k = 0ull;
      int at = tid;
      if (C == 1 || none) {
        if (tid < n && !none) k = S.top[tid];
      } else {
        if (tid < C * n) S.merge[tid] = k = cl.map_shared_rank(&S.top[0], tid / n)[tid % n];
        __syncthreads();
        if (tid < C * n) {
          // equal keys are the empty places only: they keep their order
          at = 0;
          for (int i = 0; i < C * n; ++i) at += S.merge[i] > k || (S.merge[i] == k && i < tid);
        } else {
          at = n;
        }
      }
      if (at < n) {
        const float x = okey_value((uint32_t)(k >> 32));
        top_ids[row * n + at] = k ? (int)~(uint32_t)k : -1;
        top_lp[row * n + at] = none ? NAN : (k ? LN2 * (fmaf(x, c, -p.M) - l2) : -INFINITY);
      }
    }
  }
  if (C > 1) cl.sync();   // the other CTAs' shared memory lives until it has been read
}

// --- gradient ----------------------------------------------------------------

constexpr int BT = 256;      // threads
constexpr int BU = 4;        // vectors a thread has in flight
constexpr int MAX_FIX = MAX_TOP + 1;

struct Coef {
  float chi, clo, lhi, llo;   // c = log2(e)/T and lse log2(e), as two floats each
  float k0, k1;               // dx = p (k0 + k1 u), u = log2 p
};

template <typename T>
__device__ __forceinline__ float grad_at(float x, const Coef& f) {
  const float u = fmaxf(fmaf(x, f.chi, -f.lhi) + fmaf(x, f.clo, -f.llo), U_MIN);
  return ex2(u) * fmaf(f.k1, u, f.k0);
}

template <typename T>
__global__ void __launch_bounds__(BT)
    logprobs_grad_kernel(const T* logits, int V, long long ld, const int32_t* __restrict__ tokens,
                         const float* __restrict__ temperature, const float* __restrict__ lse,
                         const float* __restrict__ entropy, const float* __restrict__ grad_lp,
                         const float* __restrict__ grad_h, int n, const int32_t* __restrict__ top_ids,
                         const float* __restrict__ grad_top, T* grad, long long gld, int chunks) {
  constexpr int EPV = Elem<T>::EPV;
  constexpr int CHUNK = BT * BU * EPV;
  __shared__ int fix_id[MAX_FIX];
  __shared__ float fix_g[MAX_FIX];
  __shared__ int nfix;
  const long long row = blockIdx.x / chunks;
  const int e0 = (int)(blockIdx.x % chunks) * CHUNK;   // the chunk's first element
  const int tid = threadIdx.x;
  const T* x = logits + row * ld;
  T* y = grad + row * gld;
  const int e1 = min(V, e0 + CHUNK);
  const int tok = tokens[row];
  float temp = temperature ? temperature[row] : 1.f;
  if (temp == 0.f) temp = 1.f;
  const float L = lse[row];
  const bool skip = tok < 0, bad = !skip && !(fabsf(L) < INFINITY);
  Coef f{};
  if (!skip && !bad) {
    // Two-float products: |x c| reaches tens, and the rounding of one float there
    // would be an error of 1e-6 in every probability.
    f.chi = LOG2E / temp;
    f.clo = (fmaf(-f.chi, temp, LOG2E) + LOG2E_LO) / temp;
    f.lhi = L * LOG2E;
    f.llo = fmaf(L, LOG2E, -f.lhi) + L * LOG2E_LO;
    const float gl = grad_lp ? grad_lp[row] : 0.f, gh = grad_h ? grad_h[row] : 0.f;
    float gsum = gl;
    for (int i = 0; i < n; ++i) {
      const int id = top_ids[row * n + i];
      if (id >= 0 && id < V) gsum += grad_top[row * n + i];
    }
    f.k0 = -(gsum + gh * entropy[row]) / temp;
    f.k1 = -gh * LN2 / temp;
    if (tid == 0) {
      int k = 0;
      if (gl != 0.f && tok >= e0 && tok < e1) {
        fix_id[k] = tok;
        fix_g[k++] = gl / temp;
      }
      for (int i = 0; i < n; ++i) {
        const int id = top_ids[row * n + i];
        if (id >= e0 && id < e1) {
          fix_id[k] = id;
          fix_g[k++] = grad_top[row * n + i] / temp;
        }
      }
      nfix = k;
    }
  } else if (tid == 0) {
    nfix = 0;
  }
  __syncthreads();
  const int nf = nfix;
  const auto one = [&](int id, float v) {
    float d = skip ? 0.f : bad ? NAN : grad_at<T>(v, f);
    for (int k = 0; k < nf; ++k)
      if (fix_id[k] == id) d += fix_g[k];
    return Elem<T>::put(d);
  };
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x + e0), ya = reinterpret_cast<uintptr_t>(y + e0);
  if (((xa ^ ya) & 15) != 0) {   // rows that sit differently to 16 bytes: element by element
    for (int id = e0 + tid; id < e1; id += BT) y[id] = one(id, skip ? 0.f : Elem<T>::get(x + id));
    return;
  }
  const int a0 = min((int)(((16 - (xa & 15)) & 15) / sizeof(T)), e1 - e0);
  const int nvec = (e1 - e0 - a0) / EPV;
  const int loose = e1 - e0 - nvec * EPV;   // a0 before the vectors, the rest after them
  if (tid < loose) {
    const int id = tid < a0 ? e0 + tid : e0 + nvec * EPV + tid;
    y[id] = one(id, skip ? 0.f : Elem<T>::get(x + id));
  }
  uint4 v[BU];
#pragma unroll
  for (int u = 0; u < BU; ++u) {
    const int i = u * BT + tid;
    if (i < nvec && !skip) v[u] = *reinterpret_cast<const uint4*>(x + e0 + a0 + i * EPV);
  }
#pragma unroll
  for (int u = 0; u < BU; ++u) {
    const int i = u * BT + tid;
    if (i >= nvec) break;
    const int id = e0 + a0 + i * EPV;
    float z[EPV];
    if (skip || bad) {
#pragma unroll
      for (int j = 0; j < EPV; ++j) z[j] = skip ? 0.f : NAN;
    } else {
      unpack<T>(v[u], z);
#pragma unroll
      for (int j = 0; j < EPV; ++j) z[j] = grad_at<T>(z[j], f);
      for (int k = 0; k < nf; ++k) {
        const int at = fix_id[k] - id;
#pragma unroll
        for (int j = 0; j < EPV; ++j)
          if (at == j) z[j] += fix_g[k];
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

// CTAs a row is spread over: as many as keep 304 CTAs (two on each of 152 SMs) busy,
// while each still has two waves of groups to stream.
static int cluster_size(int R, int V, int epv) {
  const int groups = (V / epv + 31) / 32;
  int c = 1;
  while (c < MAX_CLUSTER && (long long)R * c < 304 && groups >= 2 * c * NW * UNR) c *= 2;
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
  logprobs_grad_kernel<T><<<(unsigned)blocks, BT, 0, st>>>(static_cast<const T*>(logits), V, ld, tokens, temp, lse,
                                                          ent, glp, gh, n, ids, gtop, static_cast<T*>(grad), gld,
                                                          chunks);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

static bool bad_shape(int R, int V, long long ld, int n) {
  return R < 1 || R > (1 << 24) || V < 2 || V > 262144 || ld < V || n < 0 || n > MAX_TOP;
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

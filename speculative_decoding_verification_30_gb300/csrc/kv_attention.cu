// Attention of a window of new tokens over the paged 8-bit cache (C ABI and
// definitions in include/spec_kv.h).
//
// A window has few query rows (new tokens x query heads of a kv head) and reads the
// whole cache once, so the bound is HBM: 2 head_dim bytes for each cached token and
// kv head. The work is cut into units of 32 cached tokens of one item = (sequence,
// kv head, tile of up to 8 NT query rows), and every warp takes an equal share of
// all units, whatever the sequences' lengths: it streams its units through a ring of
// shared-memory stages of its own (cp.async; nothing waits on another warp) and
// keeps a softmax of its own. An item that lies within one warp's share is written
// out; the others leave (max, sum, weighted values) in the workspace for
// kv_combine_kernel.
//
// Per unit the products are transposed, S^T = K Q^T and O^T += V^T P^T, so that the
// cached tokens (and head_dim) fill the 16-row side of the matrix instruction and
// the query rows only its 8-column side: 20 rows cost 24 and not 32. e4m3 codes are
// converted to fp16 in registers, which is exact. Both contractions may take their
// index in any order, so each lane loads 16 neighbouring bytes and calls them
// whatever the fragment wants; the value scale of a page enters through the exponent
// (weight 2^(s + log2 scale - m)) and the key scale through the logit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kv_common.cuh"
#include "launch_cache.h"

namespace svkv {

constexpr int TOK = 32;        // cached tokens of a unit
constexpr int WARPS = 8;
constexpr int MAX_NT = 4;      // query rows of an item: 8 NT
constexpr int MIN_UNITS = 2;   // a warp takes at least this many
// Weights are 2^(t - m) with m = LIFT below the running maximum of the exponents t,
// and m moves only when a weight would exceed 2^TOP: they stay within fp16 (65504)
// and the small ones keep as much of its range as there is.
constexpr float LIFT = 7.f, TOP = 15.f;
constexpr float LN2F = 0.693147180559945309f, LOG2EF = 1.44269504088896341f;

struct AttnArgs {
  Window w;
  const __nv_bfloat16* q;
  long long q_stride;
  const uint8_t *k_codes, *v_codes;
  const float *k_scale, *v_scale;
  float scale;        // times log2(e)
  int window;
  __nv_bfloat16* out;
  float* lse;
  long long* prefix;   // workspace: units before each sequence, [B + 1], then the warps in use
  float* part;         // workspace: 2 slots for each warp
  int workers;
};

struct Meta {          // of a stage
  int b, h, rt, tile;  // unit: 32 tokens from 32 tile of (b, h, rt)
  int first, last;     // of the warp's share of the item
  int slot;            // of the workspace, if the share is a part of the item
  int pad;
  float ks[2], vs[2];  // scales of the two halves of 16 tokens
};

template <int D>
struct Stage {
  uint8_t k[TOK * D], v[TOK * D];
  Meta m;
};
static_assert(sizeof(Meta) % 16 == 0, "stages stay 16-byte aligned");
template <int D>
constexpr int stages() { return D == 128 ? 3 : 6; }

// Units of sequence b: kv_heads * row tiles * token tiles (at least one tile, so
// that every row is written).
struct Span {
  int tile0, tiles, rts;
};
template <int NT>
__device__ __forceinline__ Span span(const AttnArgs& A, const Seq& s) {
  Span p{0, 0, 0};
  if (s.count == 0) return p;
  const long long cap = (long long)A.w.max_pages * A.w.page_size;
  const long long end = s.len < 0 ? 0 : min(s.len + s.count, cap);
  long long lo = A.window && s.len >= 0 ? max(s.len - A.window + 1, 0ll) : 0ll;
  lo = min(lo, end);
  p.tile0 = (int)(lo / TOK);
  p.tiles = max((int)((end + TOK - 1) / TOK) - p.tile0, 1);
  p.rts = (int)(((long long)s.count * (A.w.q_heads / A.w.kv_heads) + 8 * NT - 1) / (8 * NT));
  return p;
}
template <int NT>
__device__ __forceinline__ long long units_of(const AttnArgs& A, int b) {
  const Span p = span<NT>(A, sequence(A.w, b));
  return (long long)A.w.kv_heads * p.rts * p.tiles;
}

__device__ __forceinline__ long long share_start(long long w, long long units, long long workers) {
  return w * units / workers;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {   // zeros when off
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float ex2f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Four e4m3 codes as two pairs of fp16 (exact).
__device__ __forceinline__ void widen(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk c of token t in a stage's tile: chunks are permuted by
// the token so that the fragments' loads touch every bank once (head_dim 64: twice).
template <int D>
__device__ __forceinline__ int chunk_at(int t, int c) {
  return D == 128 ? t * 128 + ((c ^ (t & 7)) << 4) : t * 64 + ((c ^ ((t >> 1) & 3)) << 4);
}

// The value product of 16 tokens one token at a time, each added only to the rows
// that see it (rare: only where a masked unit holds NaN values). Works on copies, so
// that the caller's accumulators stay in registers.
template <int D, int NT>
struct ByToken {
  float o[D / 16][NT][4];
  uint32_t v[4][D / 32], pf[NT][2];
  uint32_t seen[NT][2];   // bit k: the thread's row (n, e) sees token k
};
template <int D, int NT>
__device__ __noinline__ void add_by_token(ByToken<D, NT>& x, int q) {
#pragma unroll 1
  for (int k = 0; k < 16; ++k) {
    const bool mine = q == (k & 7) >> 1;
    const int slot = (k & 1) + 2 * (k >> 3);
#pragma unroll 1
    for (int j = 0; j < D / 16; ++j) {
      const uint32_t pick = j & 1 ? 0x7362u : 0x5140u;
      uint32_t a0, a1, a2, a3, y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = mine && i == slot ? x.v[i][j >> 1] : 0u;
      widen(__byte_perm(y[0], y[1], pick), a0, a1);
      widen(__byte_perm(y[2], y[3], pick), a2, a3);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma16816(c, a0, a1, a2, a3, x.pf[n][0], x.pf[n][1]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (x.seen[n][e] >> k & 1u) {
            x.o[j][n][e] += c[e];
            x.o[j][n][2 + e] += c[2 + e];
          }
      }
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(WARPS * 32, 1) kv_attention_kernel(const AttnArgs A) {
  constexpr int NS = stages<D>();
  constexpr int KW = D / 16;       // words (4 codes) of a token in a lane = steps of the key product
  constexpr int DT = D / 16;       // 16-row tiles of head_dim in the value product
  constexpr int VW = D / 32;       // words of a token's values in a lane
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_sum[WARPS], s_start_pre[WARPS];
  __shared__ int s_start_b[WARPS];
  const Window& w = A.w;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int G = w.q_heads / w.kv_heads;

  // --- shares: total units, then the sequence in which each warp's share begins
  long long mine = 0;
  for (int b = tid; b < w.B; b += WARPS * 32) mine += units_of<NT>(A, b);
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s_sum[warp] = mine;
  if (tid < WARPS) s_start_b[tid] = -1;
  __syncthreads();
  long long units = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) units += s_sum[i];
  const long long workers = min((long long)A.workers, max(units / MIN_UNITS, 1ll));
  __syncthreads();
  long long before = 0;
  for (int b0 = 0; b0 < w.B; b0 += WARPS * 32) {
    const int b = b0 + tid;
    const long long u = b < w.B ? units_of<NT>(A, b) : 0;
    long long inc = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    long long pre = before;
    for (int i = 0; i < warp; ++i) pre += s_sum[i];
    for (int i = 0; i < WARPS; ++i) before += s_sum[i];
    pre += inc - u;
    for (int i = 0; i < WARPS; ++i) {
      const long long wk = (long long)blockIdx.x * WARPS + i;
      if (wk < workers) {
        const long long at = share_start(wk, units, workers);
        if (u > 0 && at >= pre && at < pre + u) {
          s_start_b[i] = b;
          s_start_pre[i] = pre;
        }
      }
    }
    if (blockIdx.x == 0 && b < w.B) A.prefix[b] = pre;
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) {
    A.prefix[w.B] = units;
    A.prefix[w.B + 1] = workers;
  }
  const long long wk = (long long)blockIdx.x * WARPS + warp;
  int cb = s_start_b[warp];
  if (wk >= workers || cb < 0) return;
  const long long u0 = share_start(wk, units, workers), u1 = share_start(wk + 1, units, workers);
  Stage<D>* ring = reinterpret_cast<Stage<D>*>(smem) + warp * NS;

  // --- cursor of the copies: unit `cu` is tile `ct` of item (cb, ch, cr)
  long long cu = u0;
  Seq cs = sequence(w, cb);
  Span cp = span<NT>(A, cs);
  int ct, ch, cr;
  {
    const long long x = u0 - s_start_pre[warp];
    const long long item = x / cp.tiles;
    ct = (int)(x % cp.tiles);
    ch = (int)(item / cp.rts);
    cr = (int)(item % cp.rts);
  }
  const auto issue = [&](int stage) {
    if (cu < u1) {
      Stage<D>& S = ring[stage];
      const int tile = cp.tile0 + ct;
      const int left = (int)min((long long)cp.tiles - ct, u1 - cu);   // units to the end of the share of this item
      const long long end = cs.len < 0 ? 0 : cs.len + cs.count;
      constexpr int CH = D / 16;            // chunks of a token
      constexpr int RPI = 32 / CH;          // tokens a warp copies at once
      const int c = lane % CH;
      int page[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) page[i] = page_of(w, cb, ((long long)tile * TOK + 16 * i) / w.page_size);
#pragma unroll
      for (int i = 0; i < TOK / RPI; ++i) {
        const int t = i * RPI + lane / CH;
        const long long pos = (long long)tile * TOK + t;
        const int pg = page[t >> 4];
        const bool on = pg >= 0 && pos < end;
        const size_t off = (((size_t)(on ? pg : 0) * w.kv_heads + ch) * w.page_size + (size_t)(pos % w.page_size)) * D + c * 16;
        copy16(smem_u32(S.k + chunk_at<D>(t, c)), A.k_codes + off, on);
        copy16(smem_u32(S.v + chunk_at<D>(t, c)), A.v_codes + off, on);
      }
      if (lane < 4) {
        const int i = lane & 1;
        const int pg = i ? page[1] : page[0];
        const size_t off = (size_t)max(pg, 0) * w.kv_heads + ch;
        copy4(smem_u32(lane < 2 ? &S.m.ks[i] : &S.m.vs[i]), (lane < 2 ? A.k_scale : A.v_scale) + off, pg >= 0);
      }
      if (lane == 0) {
        S.m.b = cb;
        S.m.h = ch;
        S.m.rt = cr;
        S.m.tile = tile;
        S.m.first = ct == 0 || cu == u0;
        S.m.last = left == 1;
        S.m.slot = cu - u0 < (long long)ct + 1 ? 0 : 1;
      }
      ++cu;
      if (++ct == cp.tiles) {
        ct = 0;
        if (++cr == cp.rts) {
          cr = 0;
          if (++ch == w.kv_heads) {
            ch = 0;
            if (cu < u1) {
              do {
                cs = sequence(w, ++cb);
                cp = span<NT>(A, cs);
              } while (cp.rts == 0 && cb + 1 < w.B);
            }
          }
        }
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) issue(i);

  uint32_t qf[NT][2 * KW];     // query fragments
  float rs[NT][2];             // logit factor of the thread's rows 8 n + 2 q + {0, 1}
  float m[NT][2], l[NT][2], o[DT][NT][4];
  int stage = 0, begin = 0;    // begin: the tile at which the share of the item began
  Seq s{};
  for (long long u = u0; u < u1; ++u) {
    copies_wait<NS - 2>();
    __syncwarp();
    issue(stage == 0 ? NS - 1 : stage - 1);
    const Stage<D>& S = ring[stage];
    const Meta& M = S.m;
    const int row0 = M.rt * ROWS;
    if (M.first) {
      begin = M.tile;
      s = sequence(w, M.b);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // the lane's row is 8 n + g, its D / 4 elements from q D / 4
        const int row = row0 + 8 * n + g, i = row / G, hd = M.h * G + row % G;
        uint32_t x[D / 8];
        if (i < s.count) {
          const uint4* p = reinterpret_cast<const uint4*>(A.q + (size_t)(s.first + i) * (size_t)A.q_stride + (size_t)hd * D + q * (D / 4));
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const uint4 v = p[k];
            x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int k = 0; k < D / 8; ++k) x[k] = 0u;
        }
        // scaled by a power of two so that the row's largest element lies in [2^7, 2^8)
        uint32_t top = 0u;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const uint32_t a = (x[k] << 16) & 0x7FFFFFFFu, b = x[k] & 0x7FFF0000u;
          if (a < 0x7F800000u) top = max(top, a);
          if (b < 0x7F800000u) top = max(top, b);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = top ? min(max((int)(top >> 23) - 127 - 7, -100), 119) : 0;   // 2^e times [2^7, 2^8)
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
          qf[n][k] = pack_h2(__uint_as_float(x[k] << 16) * down, __uint_as_float(x[k] & 0xFFFF0000u) * down);
        const float f = up * A.scale;
        rs[n][0] = __shfl_sync(0xffffffffu, f, 8 * q);
        rs[n][1] = __shfl_sync(0xffffffffu, f, 8 * q + 4);
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[j][n][k] = 0.f;
      }
    }

    // --- logits: sc[t][n] holds tokens 16 t + g (+ 8), rows 8 n + 2 q (+ 1)
    float sc[2][NT][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t ka[KW], kb[KW];
      const int ta = 16 * t + g;
      if (D == 128) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 a = *reinterpret_cast<const uint4*>(S.k + chunk_at<D>(ta, 2 * q + i));
          const uint4 b = *reinterpret_cast<const uint4*>(S.k + chunk_at<D>(ta + 8, 2 * q + i));
          ka[4 * i % KW] = a.x, ka[(4 * i + 1) % KW] = a.y, ka[(4 * i + 2) % KW] = a.z, ka[(4 * i + 3) % KW] = a.w;
          kb[4 * i % KW] = b.x, kb[(4 * i + 1) % KW] = b.y, kb[(4 * i + 2) % KW] = b.z, kb[(4 * i + 3) % KW] = b.w;
        }
      } else {
        const uint4 a = *reinterpret_cast<const uint4*>(S.k + chunk_at<D>(ta, q));
        const uint4 b = *reinterpret_cast<const uint4*>(S.k + chunk_at<D>(ta + 8, q));
        ka[0] = a.x, ka[1] = a.y, ka[2] = a.z, ka[3] = a.w;
        kb[0] = b.x, kb[1] = b.y, kb[2] = b.z, kb[3] = b.w;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[t][n][k] = 0.f;
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        uint32_t a0, a1, a2, a3;
        widen(ka[k], a0, a2);
        widen(kb[k], a1, a3);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(sc[t][n], a0, a1, a2, a3, qf[n][2 * k], qf[n][2 * k + 1]);
      }
    }

    // --- weights. A token's exponent is its logit (base 2) plus log2 of its value scale
    const int tok0 = M.tile * TOK;
    float inv[2];
    bool gap = false;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float ks = M.ks[t], vs = M.vs[t], lv = log2f(vs);
      inv[t] = vs > 0.f ? __frcp_rn(vs) : 0.f;
      gap |= vs == 0.f;     // an unmapped page (its copies were zeros)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[t][n][k] = fmaf(sc[t][n][k], rs[n][k & 1] * ks, lv);
    }
    const long long first_pos = s.len;    // the earliest query's position
    const bool masked = gap || s.len < 0 || tok0 + TOK - 1 > first_pos ||
                        (A.window && tok0 <= s.len + s.count - 1 - A.window);
    // whether the thread's row e of tile n sees position p
    const auto sees = [&](int n, int e, int p) {
      const long long pos = s.len + (row0 + 8 * n + 2 * q + e) / G;
      return s.len >= 0 && p <= pos && !(A.window && p <= pos - A.window) && inv[((p - tok0) >> 4) & 1] != 0.f;
    };
    if (masked) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (!sees(n, e, tok0 + 16 * t + g + 8 * k)) sc[t][n][2 * k + e] = -INFINITY;
    }
    bool over = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float top = fmaxf(fmaxf(sc[0][n][e], sc[0][n][2 + e]), fmaxf(sc[1][n][e], sc[1][n][2 + e]));
        over |= top > m[n][e] + TOP;
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(fmaxf(sc[0][n][e], sc[0][n][2 + e]), fmaxf(sc[1][n][e], sc[1][n][2 + e]));
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          top -= LIFT;
          if (top > m[n][e]) {
            const float f = ex2f(m[n][e] - top);   // 0 the first time
            m[n][e] = top;
            l[n][e] *= f;
#pragma unroll
            for (int j = 0; j < DT; ++j) {
              o[j][n][e] *= f;
              o[j][n][2 + e] *= f;
            }
          }
        }
    }
    uint32_t pf[2][NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float p0 = ex2f(sc[t][n][2 * k] - m0), p1 = ex2f(sc[t][n][2 * k + 1] - m1);
          l[n][0] = fmaf(p0, inv[t], l[n][0]);
          l[n][1] = fmaf(p1, inv[t], l[n][1]);
          pf[t][n][k] = transpose8(pack_h2(p0, p1));
        }
    }

    // --- values: o[j][n] holds head_dim (D / 8) g + 2 j + {0: k < 2, 1: k >= 2}, rows 8 n + 2 q + (k & 1)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t v[4][VW];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tk = 16 * t + 2 * q + (i & 1) + 8 * (i >> 1);
        if (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(S.v + chunk_at<D>(tk, g));
          v[i][0] = x.x, v[i][1 % VW] = x.y, v[i][2 % VW] = x.z, v[i][3 % VW] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(S.v + chunk_at<D>(tk, g >> 1) + 8 * (g & 1));
          v[i][0] = x.x, v[i][1] = x.y;
        }
      }
      if (masked) {
        // NaN values of tokens that only some rows see: 0 * NaN must not reach the others
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < VW; ++x) nan |= (((v[i][x] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u;
        if (__any_sync(0xffffffffu, nan)) {
          ByToken<D, NT> x;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              x.pf[n][e] = pf[t][n][e];
              x.seen[n][e] = 0u;
#pragma unroll 1
              for (int k = 0; k < 16; ++k) x.seen[n][e] |= (uint32_t)sees(n, e, tok0 + 16 * t + k) << k;
            }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int y = 0; y < VW; ++y) x.v[i][y] = v[i][y];
#pragma unroll
          for (int j = 0; j < DT; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int k = 0; k < 4; ++k) x.o[j][n][k] = o[j][n][k];
          add_by_token<D, NT>(x, q);
#pragma unroll
          for (int j = 0; j < DT; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[j][n][k] = x.o[j][n][k];
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < DT; ++j) {
        const uint32_t pick = j & 1 ? 0x7362u : 0x5140u;   // bytes 2, 3 or 0, 1 of two neighbouring tokens, interleaved
        uint32_t a0, a1, a2, a3;
        widen(__byte_perm(v[0][j >> 1], v[1][j >> 1], pick), a0, a1);
        widen(__byte_perm(v[2][j >> 1], v[3][j >> 1], pick), a2, a3);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(o[j][n], a0, a1, a2, a3, pf[t][n][0], pf[t][n][1]);
      }
    }

    if (M.last) {
      const Span p = span<NT>(A, s);
      const bool whole = begin == p.tile0 && M.tile == p.tile0 + p.tiles - 1;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
          const int r = 8 * n + 2 * q + e, row = row0 + r, i = row / G;
          if (i >= s.count) continue;
          const int hd = M.h * G + row % G;
          const size_t at = (size_t)(s.first + i) * w.q_heads + hd;
          if (whole) {
            const float f = l[n][e] == 0.f ? 0.f : 1.f / l[n][e];
            uint32_t y[D / 16];
#pragma unroll
            for (int j = 0; j < DT; ++j) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(o[j][n][e] * f, o[j][n][2 + e] * f);
              y[j] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            uint4* dst = reinterpret_cast<uint4*>(A.out + at * D + g * (D / 8));
#pragma unroll
            for (int j = 0; j < D / 64; ++j) dst[j] = make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
            if (A.lse && g == 0) A.lse[at] = LN2F * (m[n][e] + log2f(l[n][e]));
          } else {
            float* slot = A.part + ((size_t)wk * 2 + M.slot) * ROWS * (D + 2);
            if (g == 0) {
              slot[2 * r] = m[n][e];
              slot[2 * r + 1] = l[n][e];
            }
            float4* dst = reinterpret_cast<float4*>(slot + 2 * ROWS + r * D + g * (D / 8));
#pragma unroll
            for (int j = 0; j < DT / 2; ++j)
              dst[j] = make_float4(o[2 * j][n][e], o[2 * j][n][2 + e], o[2 * j + 1][n][e], o[2 * j + 1][n][2 + e]);
          }
        }
    }
    stage = stage + 1 == NS ? 0 : stage + 1;
  }
}

// Joins the shares of the items that several warps worked on: a block takes the
// query heads of one (token, kv head).
constexpr int CT = 128;
template <int D, int NT>
__global__ void __launch_bounds__(CT) kv_combine_kernel(const AttnArgs A) {
  constexpr int ROWS = 8 * NT, SUB = CT / D;   // rows a block works on at once
  const Window& w = A.w;
  const int G = w.q_heads / w.kv_heads;
  long long blk = blockIdx.x;
  const int h = (int)(blk % w.kv_heads);
  blk /= w.kv_heads;
  const int i = (int)(blk % w.max_tokens), b = (int)(blk / w.max_tokens);
  const Seq s = sequence(w, b);
  if (i >= s.count) return;
  const Span p = span<NT>(A, s);
  const long long units = A.prefix[w.B], workers = A.prefix[w.B + 1], pre = A.prefix[b];
  const int d = threadIdx.x % D;
  for (int gq = threadIdx.x / D; gq < G; gq += SUB) {
    const int row = i * G + gq, rt = row / ROWS, r = row % ROWS;
    const long long i0 = pre + ((long long)h * p.rts + rt) * p.tiles, i1 = i0 + p.tiles;
    const long long w0 = ((i0 + 1) * workers - 1) / units, w1 = (i1 * workers - 1) / units;
    if (w0 == w1) continue;   // written already
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (long long k = w0; k <= w1; ++k) {
      const float* slot = A.part + ((size_t)k * 2 + (share_start(k, units, workers) < i0 ? 1 : 0)) * ROWS * (D + 2);
      const float mk = slot[2 * r], lk = slot[2 * r + 1], ok = slot[2 * ROWS + r * D + d];
      const float top = fmaxf(m, mk);
      if (top > -INFINITY) {
        const float f = ex2f(m - top), fk = ex2f(mk - top);
        l = fmaf(lk, fk, l * f);
        o = fmaf(ok, fk, o * f);
        m = top;
      } else if (lk != lk) {
        l = lk;
      }
    }
    const size_t at = (size_t)(s.first + i) * w.q_heads + h * G + gq;
    A.out[at * D + d] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
    if (A.lse && d == 0) A.lse[at] = LN2F * (m + log2f(l));
  }
}

static sv::LaunchCache g_attn_cache;

// Row tiles of an item: just enough for the window, at most MAX_NT.
static int row_tiles(int max_tokens, int group) {
  const long long rows = (long long)max_tokens * group;
  return rows >= 8 * MAX_NT ? MAX_NT : (int)((rows + 7) / 8);
}

static int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (g_attn_cache.get(dev, reinterpret_cast<const void*>(&sm_count), 0, 0, &n, [&](int* v) {
        return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
      }) != cudaSuccess)
    return 0;
  return n;
}

static size_t prefix_bytes(int B) { return ((size_t)(B + 2) * sizeof(long long) + 127) & ~(size_t)127; }
static size_t part_bytes(int workers, int nt, int D) { return (size_t)workers * 2 * 8 * nt * (D + 2) * sizeof(float); }

template <int D, int NT>
static sv_status launch_attention(AttnArgs& A, cudaStream_t st) {
  constexpr size_t SMEM = sizeof(Stage<D>) * stages<D>() * WARPS;
  int dev = 0, done = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      g_attn_cache.get(dev, reinterpret_cast<const void*>(kv_attention_kernel<D, NT>), SMEM, 0, &done, [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(kv_attention_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
      }) != cudaSuccess)
    return SV_ERR_CUDA;
  kv_attention_kernel<D, NT><<<A.workers / WARPS, WARPS * 32, SMEM, st>>>(A);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  const long long blocks = (long long)A.w.B * A.w.max_tokens * A.w.kv_heads;
  kv_combine_kernel<D, NT><<<(unsigned)blocks, CT, 0, st>>>(A);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

template <int D>
static sv_status pick_attention(int nt, AttnArgs& A, cudaStream_t st) {
  switch (nt) {
    case 1: return launch_attention<D, 1>(A, st);
    case 2: return launch_attention<D, 2>(A, st);
    case 3: return launch_attention<D, 3>(A, st);
    default: return launch_attention<D, 4>(A, st);
  }
}

}  // namespace svkv

size_t spec_kv_attention_workspace_bytes(int B, int max_tokens, int q_heads, int kv_heads, int head_dim) {
  using namespace svkv;
  if (B < 1 || B > 65535 || max_tokens < 1 || max_tokens > (1 << 24) || kv_heads < 1 || kv_heads > 256 ||
      q_heads < kv_heads || q_heads % kv_heads || q_heads / kv_heads > 64 || (head_dim != 64 && head_dim != 128))
    return 0;
  return prefix_bytes(B) + part_bytes(sm_count() * WARPS, row_tiles(max_tokens, q_heads / kv_heads), head_dim);
}

sv_status spec_kv_attention(const void* q, long long q_stride, const void* k_codes, const float* k_scale,
                            const void* v_codes, const float* v_scale, const int32_t* seq_len,
                            const int32_t* cu_tokens, const int32_t* page_table, int B, int N, int max_tokens,
                            int max_pages, int num_pages, int page_size, int q_heads, int kv_heads, int head_dim,
                            float scale, int window, void* out, float* lse, void* workspace, size_t workspace_bytes,
                            void* stream) {
  using namespace svkv;
  if (!q || !k_codes || !k_scale || !v_codes || !v_scale || !seq_len || !cu_tokens || !page_table || !out || !workspace)
    return SV_ERR_NULL;
  const Window w{seq_len, cu_tokens, page_table, B,       N,        max_tokens, max_pages,
                 num_pages, page_size, q_heads,  kv_heads, head_dim};
  if (bad_window(w) || q_stride < (long long)q_heads * head_dim || window < 0 || !isfinite(scale)) return SV_ERR_SHAPE;
  if ((long long)B * max_tokens * kv_heads > 2147483647ll) return SV_ERR_SHAPE;
  if (!aligned(q, 16) || (q_stride * 2) % 16 || !aligned(out, 16) || !aligned(k_codes, 16) || !aligned(v_codes, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(seq_len, 4) || !aligned(cu_tokens, 4) ||
      !aligned(page_table, 4) || !aligned(lse, 4))
    return SV_ERR_ALIGN;
  const int nt = row_tiles(max_tokens, q_heads / kv_heads);
  const int sms = aligned(workspace, 16) ? sm_count() : 1;
  if (sms < 1) return SV_ERR_CUDA;
  if (!aligned(workspace, 16) || workspace_bytes < prefix_bytes(B) + part_bytes(sms * WARPS, nt, head_dim))
    return SV_ERR_WORKSPACE;
  AttnArgs A = {};
  A.w = w;
  A.q = static_cast<const __nv_bfloat16*>(q);
  A.q_stride = q_stride;
  A.k_codes = static_cast<const uint8_t*>(k_codes), A.v_codes = static_cast<const uint8_t*>(v_codes);
  A.k_scale = k_scale, A.v_scale = v_scale;
  A.scale = scale * LOG2EF;
  A.window = window;
  A.out = static_cast<__nv_bfloat16*>(out);
  A.lse = lse;
  A.prefix = static_cast<long long*>(workspace);
  A.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + prefix_bytes(B));
  A.workers = sms * WARPS;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return head_dim == 128 ? pick_attention<128>(nt, A, st) : pick_attention<64>(nt, A, st);
}

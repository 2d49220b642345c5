// LM-head logits with weights in 4 bits and group scales (C ABI and definitions in
// include/spec_lm_head.h).
//
// For a few rows the bound is the head's bytes, d / 2 and 4 d / group for each vocabulary
// entry. Vocabulary rows are the 16-row side of the matrix instruction, hidden states its
// 8-column side. The contraction may take its index in any order, so a lane keeps the 16
// neighbouring codes that one 8-byte load of a row brings (64 elements of a row for the
// four lanes that share it) and the hidden states are laid out to match, once, in shared memory. A
// code becomes bf16, exactly, by a mask and a multiply-add for two of them. The products of a group are summed by themselves, then scaled:
//   logit += scale * sum (code - 8) h + (bias + 8 scale) * sum h.
// Each warp streams its rows with the codes of the next 256 elements on their way in registers. Where
// there are few tiles, warps share one along d.
// Measured: 1 row x 151,936 x 1,024, groups of 64: 23.5 us, 3,750 GB/s; 5 rows x 4,096, groups of 128: 67 us,
// 4,960 GB/s, 0.73 of measured, with issue at 56% and the loads of the next codes next; 40 rows x 50,257 x
// 2,048, groups of 32: 66 us, latency of shared memory, shuffles and the products with 11 warps on an SM.
// Tried: codes widened as 128 + code less 136 (seven instructions for eight codes and not five: 28 and 84
// us); the next but one codes asked into the L2 (22.9 and 71 us); 16 warps with tiles shared by two of them for 40
// rows (70 us); the 5th-generation tensor cores with codes widened into TMEM (47, 156 and 84 us: each 64 elements
// are handed over and back, which takes longer than widening them).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/spec_lm_head.h"
#include "launch_cache.h"

namespace svq4 {

constexpr int WARPS = 16;                // of a block, at most
constexpr int STEP = 64, SUPER = 4;      // elements of a step; steps of what is on its way
constexpr int SMEM_MAX = 220 * 1024;

struct Args {
  const __nv_bfloat16* hidden;
  const uint8_t* codes;
  const unsigned short *scale, *bias;
  float* logits;
  int M, N, d;
  int supers;          // of a row
  int chunk;           // supers of hidden states in shared memory at a time
  int split;           // warps of a tile
};

__device__ __forceinline__ void mma16816_first(float* c, const uint32_t* a, const uint32_t* b, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
      "%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(b[0]), "r"(a[1]), "r"(b[1]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, const uint32_t* b, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(b[0]), "r"(a[1]), "r"(b[1]), "r"(b0), "r"(b1));
}
// Eight codes as (code - 8) / 64 in bf16, in the order 0 4, 1 5, 2 6, 3 7. A code's bits at the foot of a
// bf16 are a subnormal number, code 2^-133; from bit 4 on that or one of the smallest normal ones, code 2^-129.
// Times 2^127 or 2^123, less 2^-3, both are that, exactly.
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&x)[4]) {
  const uint32_t v = w >> 8;
  const uint32_t c[4] = {w & 0x000F000Fu, w & 0x00F000F0u, v & 0x000F000Fu, v & 0x00F000F0u};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(x[k]) : "r"(c[k]), "r"(k & 1 ? 0x7D007D00u : 0x7F007F00u), "r"(0xBE00BE00u));
}
__device__ __forceinline__ float widen1(unsigned short x) { return __uint_as_float((uint32_t)x << 16); }

// First element of the eight of (step, word) that lane q of four has.
template <int G>
__device__ __forceinline__ int element(int step, int word, int q) {
  return STEP * step + (G == 32 ? 32 * word + 8 * q : 16 * q + 8 * word);
}

// Hidden states of supers c0 .. c1 - 1, as the products want them: [column tile][step][word][lane] of
// eight elements; and the sums of each group [group][column].
template <int G, int NT>
__device__ __forceinline__ void lay_out(const Args& A, int m0, int c0, int c1, uint4* sh, float* sx) {
  const int s0 = c0 * SUPER, steps = (c1 - c0) * SUPER;
  constexpr int AT_ONCE = 8;   // loads on their way
  for (int nt = 0; nt < NT; ++nt)
    for (int x0 = threadIdx.x; x0 < steps * 64; x0 += AT_ONCE * blockDim.x) {
      uint4 v[AT_ONCE];
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int x = x0 + i * blockDim.x, m = m0 + 8 * nt + (x >> 2 & 7), k = element<G>(s0 + (x >> 6), x >> 5 & 1, x & 3);
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (x < steps * 64 && m < A.M && k < A.d) v[i] = *reinterpret_cast<const uint4*>(A.hidden + (size_t)m * A.d + k);
      }
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int x = x0 + i * blockDim.x;
        // pairs 01, 23, 45, 67 to 04, 15, 26, 37
        if (x < steps * 64)
          sh[nt * steps * 64 + x] = make_uint4(__byte_perm(v[i].x, v[i].z, 0x5410), __byte_perm(v[i].x, v[i].z, 0x7632),
                                               __byte_perm(v[i].y, v[i].w, 0x5410), __byte_perm(v[i].y, v[i].w, 0x7632));
      }
    }
  // sums: four lanes to a group
  const int g0 = s0 * STEP / G, groups = steps * STEP / G, q = threadIdx.x & 3;
  const unsigned four = 0xFu << (threadIdx.x & 28);
#pragma unroll 2
  for (int x = threadIdx.x >> 2; x < 8 * NT * groups; x += blockDim.x >> 2) {
    const int m = m0 + x % (8 * NT), g = g0 + x / (8 * NT);
    float sum = 0.f;
    if (m < A.M && g * G < A.d) {
      const uint4* p = reinterpret_cast<const uint4*>(A.hidden + (size_t)m * A.d + g * G) + q;
#pragma unroll
      for (int i = 0; i < G / 32; ++i) {
        const uint4 v = p[4 * i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += __uint_as_float(w[e] << 16) + __uint_as_float(w[e] & 0xFFFF0000u);
      }
    }
    sum += __shfl_xor_sync(four, sum, 1);
    sum += __shfl_xor_sync(four, sum, 2);
    if (q == 0) sx[x] = sum;
  }
}

// G: group; NT: column tiles of 8 rows; R: tiles of 16 vocabulary rows of a warp; PARTS: the hidden states
// do not fit shared memory and are laid out part by part, all over again for each turn
template <int G, int NT, int R, bool PARTS>
__global__ void __launch_bounds__(32 * WARPS, 1) q4_kernel(const Args A) {
  constexpr int PER = SUPER * STEP / G;            // groups of a super: 8, 4 or 2
  constexpr int OWN = PER > 4 ? 2 : 1;             // of which a lane looks up so many
  extern __shared__ uint4 smem[];
  uint4* sh = smem;
  float* sx = reinterpret_cast<float*>(sh + (size_t)NT * A.chunk * SUPER * 64);
  float* red = sx + (size_t)8 * NT * A.chunk * PER;   // [warp][R NT 4][lane]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int m0 = blockIdx.y * 8 * NT, half = A.d / 2, per = A.d / G, steps = A.d / STEP;
  const int slots = (blockDim.x >> 5) / A.split, slot = warp % slots, part = warp / slots;
  const int tiles = (A.N + 16 * R - 1) / (16 * R), turns = (tiles + (int)gridDim.x * slots - 1) / ((int)gridDim.x * slots);
  const int chunks = PARTS ? (A.supers + A.chunk - 1) / A.chunk : 1;
  // the supers of chunk c that are this warp's
  const auto from = [&](int c) { return c * A.chunk + (min(A.chunk, A.supers - c * A.chunk) * part) / A.split; };
  const auto to = [&](int c) { return c * A.chunk + (min(A.chunk, A.supers - c * A.chunk) * (part + 1)) / A.split; };
  const auto tile_of = [&](int turn) { return (turn * slots + slot) * (int)gridDim.x + (int)blockIdx.x; };

  // What is on its way: super `ls` of the tile of turn `lt`; `left` steps are there from its start on
  uint2 code[SUPER][2 * R];
  unsigned short sc[2 * R][OWN], bi[2 * R][OWN];
  int lt = 0, lc = 0, ls = from(0), left = 0;
  const uint8_t* at[2 * R];
  size_t sat[2 * R];
  const auto settle = [&]() {   // on the next super that there is
    while (lt < turns && ls >= to(lc)) {
      if (++lc == chunks) lc = 0, ++lt;
      if (lt < turns) ls = from(lc);
    }
    left = lt < turns && tile_of(lt) < tiles ? steps - ls * SUPER : 0;
  };
  const auto place = [&]() {
#pragma unroll
    for (int j = 0; j < 2 * R; ++j) {
      const size_t row = min(tile_of(min(lt, turns - 1)) * 16 * R + 8 * j + g, A.N - 1);
      at[j] = A.codes + row * half + ls * (SUPER * STEP / 2) + (G == 32 ? 4 : 8) * q;
      sat[j] = row * per + ls * PER + q * OWN;
    }
  };
  // Loads where there is something, without branches, so that steps overlap
  const auto load_codes = [&](int i) {
#pragma unroll
    for (int j = 0; j < 2 * R; ++j) {
      const uint8_t* p = at[j] + i * (STEP / 2);
      if (G == 32)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.lt.s32 p, %3, %4;\n\t@p ld.global.nc.u32 %0, [%2];\n\t@p ld.global.nc.u32 %1, [%2 + 16];\n\t}"
            : "+r"(code[i][j].x), "+r"(code[i][j].y)
            : "l"(p), "r"(i), "r"(left));
      else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.lt.s32 p, %3, %4;\n\t@p ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];\n\t}"
            : "+r"(code[i][j].x), "+r"(code[i][j].y)
            : "l"(p), "r"(i), "r"(left));
    }
  };
  // Groups behind a row's end have scale and bias 0, and their hidden states are 0.
  const auto load_scales = [&]() {
    const int there = left * STEP / G - q * OWN;   // groups from the lane's first one on
#pragma unroll
    for (int o = 0; o < OWN; ++o)
#pragma unroll
      for (int j = 0; j < 2 * R; ++j) {
        sc[j][o] = bi[j][o] = 0;
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.lt.s32 p, %4, %5;\n\t@p ld.global.nc.u16 %0, [%2];\n\t@p ld.global.nc.u16 %1, [%3];\n\t}"
            : "+h"(sc[j][o]), "+h"(bi[j][o])
            : "l"(A.scale + sat[j] + o), "l"(A.bias + sat[j] + o), "r"(o), "r"(PER >= 4 || q < PER ? there : 0));
      }
  };
#pragma unroll
  for (int i = 0; i < SUPER; ++i)
#pragma unroll
    for (int j = 0; j < 2 * R; ++j) code[i][j] = make_uint2(0u, 0u);
  settle();
  place();
  if (!PARTS) {
    // the first codes come to the L2 meanwhile
    if (left > 0)
#pragma unroll
      for (int j = 0; j < 2 * R; ++j) asm volatile("prefetch.global.L2 [%0];" ::"l"(at[j]));
    lay_out<G, NT>(A, m0, 0, A.supers, sh, sx);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < SUPER; ++i) load_codes(i);
  load_scales();

  for (int turn = 0; turn < turns; ++turn) {
    const int tile = tile_of(turn);
    float out[R][NT][4];
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) out[t][n][0] = out[t][n][1] = out[t][n][2] = out[t][n][3] = 0.f;
    for (int c = 0; c < chunks; ++c) {
      if (PARTS) {
        __syncthreads();
        lay_out<G, NT>(A, m0, c * A.chunk, min((c + 1) * A.chunk, A.supers), sh, sx);
        __syncthreads();
      }
      if (tile >= tiles) continue;
      const int held = min(A.chunk, A.supers - c * A.chunk) * SUPER;   // steps in shared memory
#pragma unroll 1
      for (int s = from(c); s < to(c); ++s) {
        float fs[2 * R][OWN], ft[2 * R][OWN];
#pragma unroll
        for (int j = 0; j < 2 * R; ++j)
#pragma unroll
          for (int o = 0; o < OWN; ++o) {
            fs[j][o] = widen1(sc[j][o]);
            ft[j][o] = fmaf(8.f, fs[j][o], widen1(bi[j][o])) * 0.015625f;   // sums are kept in 64ths, as the products are
          }
        // the next super begins to come while this one is worked on
        ++ls;
        left -= SUPER;
        if (s + 1 < to(c)) {
#pragma unroll
          for (int j = 0; j < 2 * R; ++j) at[j] += SUPER * STEP / 2, sat[j] += PER;
        } else {
          settle();
          place();
        }
        load_scales();
        float acc[R][NT][4];
#pragma unroll
        for (int i = 0; i < SUPER; ++i) {
          const int st = s * SUPER + i;
          {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint32_t x[2 * R][4];
#pragma unroll
              for (int j = 0; j < 2 * R; ++j) widen(w ? code[i][j].y : code[i][j].x, x[j]);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint4 b = sh[((n * held + st - c * A.chunk * SUPER) * 2 + w) * 32 + lane];
#pragma unroll
                for (int t = 0; t < R; ++t) {
                  if (G == 32 || (w == 0 && i * STEP % G == 0))
                    mma16816_first(acc[t][n], x[2 * t], x[2 * t + 1], b.x, b.y);
                  else
                    mma16816(acc[t][n], x[2 * t], x[2 * t + 1], b.x, b.y);
                  mma16816(acc[t][n], x[2 * t] + 2, x[2 * t + 1] + 2, b.z, b.w);
                }
              }
              if (G == 32 || (w == 1 && (i + 1) * STEP % G == 0)) {
                const int gi = (i * STEP + 32 * w) / G, own = OWN == 2 ? gi >> 1 : gi;   // of the super; its lane
                float s2[2 * R], t2[2 * R];
#pragma unroll
                for (int j = 0; j < 2 * R; ++j) {
                  s2[j] = __shfl_sync(0xffffffffu, fs[j][gi & (OWN - 1)], (lane & ~3) | own);
                  t2[j] = __shfl_sync(0xffffffffu, ft[j][gi & (OWN - 1)], (lane & ~3) | own);
                }
                const float* px = sx + ((s - c * A.chunk) * PER + gi) * 8 * NT + 2 * q;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  const float2 xs = *reinterpret_cast<const float2*>(px + 8 * n);
#pragma unroll
                  for (int t = 0; t < R; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      out[t][n][e] = fmaf(s2[2 * t + (e >> 1)], acc[t][n][e],
                                          fmaf(t2[2 * t + (e >> 1)], e & 1 ? xs.y : xs.x, out[t][n][e]));
                }
              }
            }
          }
          load_codes(i);
        }
      }
    }
    if (A.split > 1) {
      // the parts of a tile, in their order
      const int id = 1 + slot, threads = 32 * A.split;
      asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");   // the last turn's are read
      float* mine = red + (size_t)warp * (R * NT * 4 * 32) + lane;
      if (part)
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) mine[((t * NT + n) * 4 + e) * 32] = out[t][n][e];
      asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
      if (part) continue;
    }
    if (tile >= tiles) continue;
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = (tile * R + t) * 16 + g + 8 * (e >> 1), m = m0 + 8 * n + 2 * q + (e & 1);
          float x = out[t][n][e];
          for (int p = 1; p < A.split; ++p) x += red[(size_t)(warp + p * slots) * (R * NT * 4 * 32) + ((t * NT + n) * 4 + e) * 32 + lane];
          if (v < A.N && m < A.M) A.logits[(size_t)m * A.N + v] = 64.f * x;
        }
  }
}

static sv::LaunchCache g_cache;
static int sm_count() try {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (g_cache.get(dev, reinterpret_cast<const void*>(&sm_count), 0, 0, &n, [&](int* v) {
        return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
      }) != cudaSuccess)
    return 0;
  return n;
} catch (...) {   // no exception passes the C entry points
  return 0;
}
// The kernel's shared-memory limit, raised once per device.
static bool raise_smem(const void* fn) try {
  int dev = 0, done = 0;
  return cudaGetDevice(&dev) == cudaSuccess && g_cache.get(dev, fn, SMEM_MAX, 0, &done, [&](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
  }) == cudaSuccess;
} catch (...) {
  return false;
}

// Bytes of a super's hidden states and sums in shared memory.
template <int G, int NT>
constexpr size_t super_bytes() {
  return (size_t)NT * SUPER * 64 * sizeof(uint4) + (size_t)8 * NT * (SUPER * STEP / G) * sizeof(float);
}

template <int G, int NT, bool PARTS>
static sv_status launch(Args A, cudaStream_t st) {
  constexpr int R = NT <= 2 ? 2 : 1;
  const int sms = sm_count();
  if (sms < 1 || !raise_smem(reinterpret_cast<const void*>(q4_kernel<G, NT, R, PARTS>))) return SV_ERR_CUDA;
  // Few tiles: as many warps to a tile as leave each SM with 16. Else as many warps in a block as make
  // the turns come out: an SM's time goes by turns x warps.
  const long long tiles = (A.N + 16 * R - 1) / (16 * R);
  A.split = 1;
  while (A.split < 8 && tiles * A.split * 2 <= (long long)sms * WARPS) A.split *= 2;
  int warps = WARPS;
  if (A.split == 1)
    for (long long w = WARPS - 1, best = 1ll << 60; w >= WARPS / 2; --w) {
      const auto cost = [&](long long x) { return (tiles + sms * x - 1) / (sms * x) * x; };
      if (best == 1ll << 60) best = cost(WARPS);
      if (cost(w) < best) best = cost(w), warps = (int)w;
    }
  const size_t fixed = A.split > 1 ? (size_t)WARPS * R * NT * 4 * 32 * sizeof(float) : 0, each = super_bytes<G, NT>();
  const size_t fit = (SMEM_MAX - fixed) / each;
  A.chunk = PARTS && (size_t)A.supers > fit ? (int)fit : A.supers;
  const long long blocks = (tiles * A.split + warps - 1) / warps;
  const dim3 grid((unsigned)(blocks < sms ? blocks : sms), (unsigned)((A.M + 8 * NT - 1) / (8 * NT)));
  q4_kernel<G, NT, R, PARTS><<<grid, 32 * warps, A.chunk * each + fixed, st>>>(A);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
// Shared memory that is always left for the sums of warps that share a tile.
template <int G, int NT>
static bool fits(const Args& A) {
  return A.supers * super_bytes<G, NT>() + (size_t)WARPS * (NT <= 2 ? 2 : 1) * NT * 4 * 32 * sizeof(float) <= SMEM_MAX;
}
template <int G, int NT>
static sv_status whole_or(const Args& A, cudaStream_t st) {
  constexpr int UP = NT == 1 ? 1 : NT <= 4 ? 4 : 8;   // of the kernels that lay out parts there are three
  return fits<G, NT>(A) ? launch<G, NT, false>(A, st) : launch<G, UP, true>(A, st);
}
template <int G>
static sv_status pick(Args A, cudaStream_t st) {
  A.supers = (A.d + SUPER * STEP - 1) / (SUPER * STEP);
  switch (A.M >= 64 ? 8 : (A.M + 7) / 8) {
    case 1: return whole_or<G, 1>(A, st);
    case 2: return whole_or<G, 2>(A, st);
    case 3: return whole_or<G, 3>(A, st);
    case 4: return whole_or<G, 4>(A, st);
    case 5: return whole_or<G, 5>(A, st);
    case 6: return whole_or<G, 6>(A, st);
    default: return whole_or<G, 8>(A, st);
  }
}

static bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace svq4

sv_status spec_lm_head_logits_q4(const void* hidden, const uint8_t* codes, const void* scale, const void* bias, int M,
                                 int N, int d, int group, float* logits, void* stream) {
  using namespace svq4;
  if (!hidden || !codes || !scale || !bias || !logits) return SV_ERR_NULL;
  if (M < 1 || M > 65536 || N < 1 || N > 16776960 || d < 64 || d > 65536 || d % 64 ||
      (group != 32 && group != 64 && group != 128) || d % group)
    return SV_ERR_SHAPE;
  if (!aligned(hidden, 16) || !aligned(codes, 16) || !aligned(scale, 4) || !aligned(bias, 4) || !aligned(logits, 4))
    return SV_ERR_ALIGN;
  Args A = {};
  A.hidden = static_cast<const __nv_bfloat16*>(hidden);
  A.codes = codes;
  A.scale = static_cast<const unsigned short*>(scale), A.bias = static_cast<const unsigned short*>(bias);
  A.logits = logits;
  A.M = M, A.N = N, A.d = d;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return group == 32 ? pick<32>(A, st) : group == 64 ? pick<64>(A, st) : pick<128>(A, st);
}

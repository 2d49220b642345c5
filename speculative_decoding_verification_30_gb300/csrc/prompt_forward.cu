// Causal attention over packed prompts (C ABI and definitions in include/spec_prompt.h).
//
// A block works on two tiles of 128 query rows that share their keys and values: two heads of
// a kv head, or, where their number is odd, two runs of 128 tokens of one head. The tiles take
// turns: while one is in its softmax, the tensor cores work for the other. For each 128 keys:
//   S = Q K^T    tcgen05, operands in shared memory, S in TMEM;
//   softmax      a thread to a row: S in registers, weights to TMEM as bf16 over S;
//   O += P V     weights from TMEM, values with their rows contracted.
// O stays in TMEM and is scaled there when a row's frame moves, which it does only when a
// weight would pass 2^8. Rows of a tile are one head's tokens, so that any number of heads to a kv
// head will do.
// Measured: 2 prompts of 8,192 tokens, 32 heads on 8 of 128: 745 us, 1,475 TFLOP/s; 24 of up to 1,500
// tokens 196 us; 8 of up to 4,001 in a window of 1,000, 12 heads of 64: 102 us. Clocks of a unit of
// both tiles in long prompts: 2,850, of which the products take 2,200 (16 of a tile 1,100, issued
// without a pause). A tile's softmax is 1,250 (load 50, maximum and votes 290, exponentials and packing
// 740, store 160) and its products' results 250 behind the last one, so that the tensor cores
// wait some 300 clocks a tile. Head_dim 64 halves the products and not the softmax. Short prompts: an
// item's end takes 4,500 clocks (the results' way out 3,500) beside 2,850 for a unit. The maximum
// taken from registers, 765 us; products issued from a branch of one lane, with descriptors in its
// registers, 85 clocks each and not 64, 936 us; waits and commits one after the other between
// weights and product, 816 us; a lane writing its row's 256 bytes by itself, which keeps the store
// unit, and the barriers behind it, busy, 842 us.
// Warps: 0 walks the work and copies (TMA), 1 issues the products, 2-3
// look for values that are not finite in units that not every row sees, 4-7 and 8-11 are the
// rows. Every wait is bounded; one that runs out stops the block, which then writes NaN to
// all of its rows.
#include "prompt_common.cuh"

namespace svpr {

constexpr int THREADS = 384;
constexpr float TOP = 8.f;               // log2 of the largest weight in a row's frame
constexpr float NO_FRAME = -1e30f;       // frame of a row that has seen nothing (finite: -inf - m stays -inf)
constexpr int NI = 4;                    // items announced at a time

struct FwdArgs {
  Prompts p;
  float scale;        // times log2(e)
  __nv_bfloat16* out;
  float* lse;
  int pair_heads;     // the tiles are two heads, not two runs of tokens
};

// Two tiles of queries and their units of 128 keys j0 .. n[t] - 1.
struct Item {
  int first, len, end;       // of the sequence; end: no item
  int head[2], q0[2], n[2];  // n[t] == j0: the tile has no rows
  int j0;
};
__device__ __forceinline__ int units_end(const Item& I) { return max(I.n[0], I.n[1]); }
// Whether some row of tile t does not see all keys of unit j.
__device__ __forceinline__ bool masked(const Prompts& p, int q0, int j) {
  return BLK * j + BLK - 1 > q0 || (p.window && BLK * j <= q0 + BLK - 1 - p.window);
}

template <int D>
struct Shape {
  static constexpr int TILE = D / 64 * COL;
  static constexpr int NK = D == 128 ? 2 : 3, NV = NK;
};
template <int D>
struct __align__(16) Ctl {
  static constexpr int NK = Shape<D>::NK, NV = Shape<D>::NV;
  uint4 turn[8][32 * 4];       // of each warp of rows: 32 columns on their way out
  uint4 odd[NV][BLK];          // values that are not finite: a bit for each element of a token
  Item item[NI];
  Bar kfull[NK], kempty[NK], vfull[NV], vempty[NV], vseen[NV];
  Bar sfull[2], pfull[2], qfull[2], qempty[2], ofull[2], ready[NI], taken[NI], done;
  int odd_unit[NV][2];         // the unit (+ 1) that last had any in that half of its tokens
  uint32_t taddr;
  int err;
};
template <int D>
constexpr int smem_bytes() {
  return 1024 + (2 + Shape<D>::NK + Shape<D>::NV) * Shape<D>::TILE + (int)sizeof(Ctl<D>);
}
static_assert(smem_bytes<128>() <= 227 * 1024 && smem_bytes<64>() <= 227 * 1024, "one block on an SM");

__device__ __forceinline__ Item item_of(const FwdArgs& A, const Seq& s, int token, int slot) {
  Item I;
  I.first = s.first, I.len = s.len, I.end = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    I.head[t] = A.pair_heads ? 2 * slot + t : slot;
    I.q0[t] = A.pair_heads ? token : token + BLK * t;
  }
  I.j0 = A.p.window ? max(token - A.p.window + 1, 0) / BLK : 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) I.n[t] = I.q0[t] < s.len ? I.q0[t] / BLK + 1 : I.j0;
  return I;
}

// A row's weights for 128 logits in its frame, to TMEM over the logits; returns their sum.
__device__ __forceinline__ float weights(uint32_t* x, uint32_t s, float rs, float m) {
  const uint64_t a = pair(rs, rs), b = pair(-m, -m);
  uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t p[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float y0, y1;
      unpair(fma2(pair(__uint_as_float(x[32 * c + 2 * k]), __uint_as_float(x[32 * c + 2 * k + 1])), a, b), y0, y1);
      y0 = ex2f(y0);
      y1 = ex2f(y1);
      sum[k & 1] = add2(sum[k & 1], pair(y0, y1));
      p[k] = pack_bf2(y0, y1);
    }
    tmem_st16(s + 16 * c, p);
  }
  float s0, s1;
  unpair(add2(sum[0], sum[1]), s0, s1);
  return s0 + s1;
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    prompt_forward_kernel(const FwdArgs A, const __grid_constant__ CUtensorMap map_q,
                          const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  constexpr int TILE = Shape<D>::TILE, NK = Shape<D>::NK, NV = Shape<D>::NV;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char *sq = smem, *sk = sq + 2 * TILE, *sv = sk + NK * TILE;
  Ctl<D>& C = *reinterpret_cast<Ctl<D>*>(sv + NV * TILE);
  volatile int* err = &C.err;
  const Prompts& P = A.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int span = A.pair_heads ? BLK : 2 * BLK, slots = A.pair_heads ? P.q_heads / 2 : P.q_heads;

  if (tid == 0) {
    for (int i = 0; i < NK; ++i) bar_init(&C.kfull[i], 1), bar_init(&C.kempty[i], 1);
    for (int i = 0; i < NV; ++i) {
      bar_init(&C.vfull[i], 1), bar_init(&C.vempty[i], 1), bar_init(&C.vseen[i], 2);
      C.odd_unit[i][0] = C.odd_unit[i][1] = 0;
    }
    for (int t = 0; t < 2; ++t) {
      bar_init(&C.sfull[t], 1), bar_init(&C.pfull[t], 4), bar_init(&C.qfull[t], 1), bar_init(&C.qempty[t], 1);
      bar_init(&C.ofull[t], 1);
    }
    for (int i = 0; i < NI; ++i) bar_init(&C.ready[i], 1), bar_init(&C.taken[i], THREADS / 32 - 1);
    bar_init(&C.done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    C.err = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&C.taddr)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    before_sync();
  }
  __syncthreads();
  after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, C.taddr, 0);   // S (and P) of tile t at columns 128 t, O at 256 + 128 t

  if (warp < 4) {
  // registers: 128 x 72 and 256 x 216 are the 384 x 168 of the launch
  asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 0) {
    // --- the walk, and the copies
    Walk w = walk_start(P, span, slots, 0, lane);
    int u = 0, uses[2] = {0, 0};
    bool ok = true;
    for (int it = 0; ok; ++it) {
      Seq s;
      int token, slot;
      const bool on = walk_to(P, w, piece_of(it), lane, s, token, slot);
      const Item I = on ? item_of(A, s, token, slot) : Item{0, 0, 1, {0, 0}, {0, 0}, {0, 0}, 0};
      if (it >= NI) ok = wait_warp(&C.taken[it % NI], (uint32_t)(it / NI - 1) & 1, err);   // by all other warps
      if (!ok) break;
      if (lane == 0) {
        C.item[it % NI] = I;
        arrive(&C.ready[it % NI]);
      }
      if (!on) break;
      for (int t = 0; t < 2; ++t) {
        if (I.n[t] == I.j0) continue;
        if (uses[t]) ok = wait_warp(&C.qempty[t], (uint32_t)(uses[t] - 1) & 1, err);
        if (!ok) break;
        ++uses[t];
        if (lane == 0) {
          expect(&C.qfull[t], TILE);
          copy_tile<D>(sq + t * TILE, &map_q, I.head[t], I.first + I.q0[t], &C.qfull[t]);
        }
      }
      const int kv = I.head[0] / P.group, n = units_end(I);
      for (int j = I.j0; j < n && ok; ++j, ++u) {
        const int ks = u % NK, vs = u % NV;
        if (u >= NK) ok = wait_warp(&C.kempty[ks], (uint32_t)(u / NK - 1) & 1, err);
        if (!ok) break;
        if (lane == 0) {
          expect(&C.kfull[ks], TILE);
          copy_tile<D>(sk + ks * TILE, &map_k, kv, I.first + BLK * j, &C.kfull[ks]);
        }
        if (u >= NV) ok = wait_warp(&C.vempty[vs], (uint32_t)(u / NV - 1) & 1, err);
        if (!ok) {   // the keys were asked for, the values were not
          if (lane == 0) {
            int never = 0;
            wait(&C.kfull[ks], (uint32_t)(u / NK) & 1, &never, LAND_NS);
          }
          break;
        }
        if (lane == 0) {
          expect(&C.vfull[vs], TILE);
          copy_tile<D>(sv + vs * TILE, &map_v, kv, I.first + BLK * j, &C.vfull[vs]);
        }
      }
    }
    // what was asked for lands before the block ends, also when the others have stopped
    if (lane == 0) {
      int never = 0;
      for (int i = max(0, u - NK); i < u; ++i) wait(&C.kfull[i % NK], (uint32_t)(i / NK) & 1, &never, LAND_NS);
      for (int i = max(0, u - NV); i < u; ++i) wait(&C.vfull[i % NV], (uint32_t)(i / NV) & 1, &never, LAND_NS);
      for (int t = 0; t < 2; ++t)
        if (uses[t]) wait(&C.qfull[t], (uint32_t)(uses[t] - 1) & 1, &never, LAND_NS);
    }
    __syncwarp();
  } else if (warp == 1) {
    // --- products. The warp stays together, so that addresses and descriptors are the same in all of it;
    // one lane issues.
    int u = 0, uses[2] = {0, 0}, pu[2] = {0, 0};   // units; items and units of each tile
    bool ok = true;
    for (int it = 0; ok; ++it) {
      ok = wait_warp(&C.ready[it % NI], (uint32_t)(it / NI) & 1, err);
      if (!ok) break;
      const int end = __shfl_sync(0xffffffffu, C.item[it % NI].end, 0), j0 = __shfl_sync(0xffffffffu, C.item[it % NI].j0, 0);
      const int n0 = __shfl_sync(0xffffffffu, C.item[it % NI].n[0], 0), n1 = __shfl_sync(0xffffffffu, C.item[it % NI].n[1], 0);
      if (end) break;
      if (lane == 0) arrive(&C.taken[it % NI]);
      const int n = max(n0, n1);
      // S of tile t and unit j, by the lane that issues; the last of the tiles gives the keys' stage back
      const auto qk = [&](int t, int j, int at) {
        mma_dims<D>(tmem + 128 * t, sq + t * TILE, sk + (at % NK) * TILE);
        commit(&C.sfull[t]);
        if (j == (t ? n1 : n0) - 1) commit(&C.qempty[t]);
        if (t == (j < n1 ? 1 : 0)) commit(&C.kempty[at % NK]);
      };
      ok = wait_warp(&C.kfull[u % NK], (uint32_t)(u / NK) & 1, err);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!ok || (t ? n1 : n0) == j0) continue;
        ok = wait_warp(&C.qfull[t], (uint32_t)uses[t] & 1, err);
        if (!ok) continue;
        ++uses[t];
        after_sync();
        if (elect()) qk(t, j0, u);
        __syncwarp();
      }
      for (int j = j0; j < n && ok; ++j, ++u) {
        ok = wait_warp(&C.vseen[u % NV], (uint32_t)(u / NV) & 1, err);   // and the next unit's keys
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int nt = t ? n1 : n0;
          if (!ok || j >= nt) continue;
          ok = wait_warp(&C.pfull[t], (uint32_t)pu[t] & 1, err);
          if (!ok) continue;
          ++pu[t];
          after_sync();
          if (elect()) {
            mma_rows<D>(tmem + 256 + 128 * t, tmem + 128 * t, sv + (u % NV) * TILE, j != j0);
            if (j == nt - 1) commit(&C.ofull[t]);
            if (t == (j < n1 ? 1 : 0)) commit(&C.vempty[u % NV]);
            if (j + 1 < nt) qk(t, j + 1, u + 1);
          }
          __syncwarp();
        }
      }
    }
    // nothing is in flight when the block ends
    if (elect()) {
      commit(&C.done);
      int never = 0;
      wait(&C.done, 0, &never, LAND_NS);
    }
    __syncwarp();
  } else {
    // --- values: where not every row sees every token, what is not finite becomes zero and is
    // kept aside, so that 0 times it reaches no row that does not see it. A warp has 64 tokens
    // of each unit.
    int u = 0;
    const int half = warp - 2;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      ok = wait_warp(&C.ready[it % NI], (uint32_t)(it / NI) & 1, err);
      if (!ok) break;
      const Item& I = C.item[it % NI];
      if (I.end) break;
      const int n = units_end(I);
      for (int j = I.j0; j < n; ++j, ++u) {
        const int vs = u % NV;
        ok = wait_warp(&C.vfull[vs], (uint32_t)(u / NV) & 1, err);
        if (!ok) break;
        if (masked(P, I.q0[0], j) || masked(P, I.q0[1], j)) {
          unsigned char* at = sv + vs * TILE + half * 64 * 128;
          uint32_t hit = 0;
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c)
#pragma unroll 8
            for (int i = 0; i < 64 * 128; i += 512) {
              const uint4 x = *reinterpret_cast<const uint4*>(at + c * COL + i + 16 * lane);
              hit |= odd_bf2(x.x) | odd_bf2(x.y) | odd_bf2(x.z) | odd_bf2(x.w);
            }
          if (__any_sync(0xffffffffu, hit)) {
            const int live = I.len - BLK * j - 64 * half;
            for (int c = 0; c < D / 64; ++c)
#pragma unroll 1
              for (int i = 0; i < 64; i += 4) {
                const int r = i + (lane >> 3), k = lane & 7;   // chunk k of 8 elements of token r
                uint4* p = reinterpret_cast<uint4*>(at + c * COL + r * 128 + ((k ^ (r & 7)) << 4));
                const uint4 x = *p;
                uint32_t y[4] = {x.x, x.y, x.z, x.w}, bits = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t o = odd_bf2(y[e]);
                  if (o & 0x8000u) bits |= 1u << (2 * e), y[e] &= 0xFFFF0000u;
                  if (o & 0x80000000u) bits |= 2u << (2 * e), y[e] &= 0xFFFFu;
                }
                if (bits) *p = make_uint4(y[0], y[1], y[2], y[3]);
                reinterpret_cast<unsigned char*>(&C.odd[vs][64 * half + r])[8 * c + k] = r < live ? (unsigned char)bits : 0;
              }
            if (lane == 0) C.odd_unit[vs][half] = u + 1;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
        }
        // a wait less for the warp that issues products: the next unit's keys are there too
        if (j + 1 < n) ok = wait_warp(&C.kfull[(u + 1) % NK], (uint32_t)((u + 1) / NK) & 1, err);
        if (!ok) break;
        __syncwarp();
        if (lane == 0) arrive(&C.vseen[vs]);
      }
      if (lane == 0) arrive(&C.taken[it % NI]);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // --- rows: thread `r` of tile `t`
    const int t = (warp - 4) >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 128 * t, to = tmem + lanes + 256 + 128 * t;
    // rows outside every sequence
    {
      const int before = min(max(P.cu[0], 0), P.N), behind = min(max(P.cu[P.B], 0), P.N);
      const long long all = ((long long)before + P.N - behind) * P.q_heads;
      for (long long x = (long long)blockIdx.x * 256 + tid - 128; x < all; x += (long long)gridDim.x * 256) {
        const long long y = x < (long long)before * P.q_heads ? x : x + (long long)(behind - before) * P.q_heads;
        for (int k = 0; k < D / 8; ++k) reinterpret_cast<uint4*>(A.out + y * D)[k] = make_uint4(0u, 0u, 0u, 0u);
        if (A.lse) A.lse[y] = -INFINITY;
      }
    }
    int u = 0, su = 0, uses = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      // a tile without rows waits for as long as the other one works
      ok = wait_warp(&C.ready[it % NI], (uint32_t)(it / NI) & 1, err, 16 * SPEC_PROMPT_WAIT_NS);
      if (!ok) break;
      const Item& I = C.item[it % NI];
      if (I.end) break;
      const int n = I.n[t], j0 = I.j0, all = units_end(I) - j0, q0 = I.q0[t], other = I.q0[t ^ 1], i = q0 + r;
      float m = NO_FRAME, l = 0.f;
      uint32_t bad[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
      for (int j = j0; j < n; ++j, ++su) {
        ok = wait_warp(&C.sfull[t], (uint32_t)su & 1, err);
        if (!ok) break;
        after_sync();
        uint32_t x[128];
        float best[4];   // the load finds the maxima
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_max32(x + 32 * c, best[c], ts + 32 * c);
        tmem_wait_ld();
        pin<128>(x);
#pragma unroll
        for (int c = 0; c < 4; ++c) asm volatile("" : "+f"(best[c]));
        const int hi = i - BLK * j, lo = P.window ? hi - P.window : -1;
        if (masked(P, q0, j)) {
          // nearly always one of the two
          if (BLK * j + BLK - 1 > q0)
#pragma unroll
            for (int k = 0; k < 128; ++k)
              if (k > hi) x[k] = 0xFF800000u;
          if (P.window && BLK * j <= q0 + BLK - 1 - P.window)
#pragma unroll
            for (int k = 0; k < 128; ++k)
              if (k <= lo) x[k] = 0xFF800000u;
#pragma unroll
          for (int k = 0; k < 4; ++k) best[k] = __uint_as_float(x[k]);
#pragma unroll
          for (int k = 4; k < 128; ++k) best[k & 3] = fmaxf(best[k & 3], __uint_as_float(x[k]));
        }
        const float top = fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3])) * A.scale;
        const bool move = top > m + TOP;
        if (__any_sync(0xffffffffu, move)) {
          // some weight would leave its range: those rows' frames move to their maxima
          const float m2 = move ? top : m, f = move ? ex2f(m - m2) : 1.f;   // f: 0 the first time
          if (j != j0) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t y[32];
              tmem_ld32(y, to + 32 * c);
              tmem_wait_ld();
              pin<32>(y);
#pragma unroll
              for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
              tmem_st32(to + 32 * c, y);
            }
          }
          l *= f;
          m = m2;
        }
        l += weights(x, ts, A.scale, m);
        const int at = u + j - j0;
        if (masked(P, q0, j) || masked(P, other, j)) {
          // the stage holds the unit until both tiles' weights are there
          const int vs = at % NV;
          ok = wait_warp(&C.vseen[vs], (uint32_t)(at / NV) & 1, err);
          if (!ok) break;
          for (int half = 0; half < 2; ++half)
            if (*reinterpret_cast<volatile int*>(&C.odd_unit[vs][half]) == at + 1)
              for (int p = max(lo + 1, 64 * half); p <= min(hi, 64 * half + 63); ++p) {
                const uint4 b = C.odd[vs][p];
                bad[0] |= b.x, bad[1] |= b.y, bad[2] |= b.z, bad[3] |= b.w;
              }
        }
        tmem_wait_st();
        before_sync();
        __syncwarp();
        if (lane == 0) arrive(&C.pfull[t]);
      }
      if (!ok) break;
      u += all;
      if (n == j0) {
        __syncwarp();
        if (lane == 0) arrive(&C.taken[it % NI]);
        continue;
      }
      ok = wait_warp(&C.ofull[t], (uint32_t)uses & 1, err);
      if (!ok) break;
      ++uses;
      after_sync();
      const bool there = i < I.len;
      const size_t at = (size_t)(I.first + i) * P.q_heads + I.head[t];
      const size_t row_at = (size_t)(I.first + i - lane) * P.q_heads + I.head[t];   // of the warp's first row
      uint4* turn = C.turn[warp - 4];
      const float f = l == 0.f ? 0.f : 1.f / l;
      const uint64_t f2 = pair(f, f);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t y[32];
        tmem_ld32(y, to + 32 * c);
        tmem_wait_ld();
        pin<32>(y);
        const uint32_t b = c == 0 ? bad[0] : c == 1 ? bad[1] : c == 2 ? bad[2] : bad[3];
        if (b)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (b >> k & 1) y[k] = 0x7FC00000u;
        uint32_t z[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float y0, y1;
          unpair(mul2(pair(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1])), f2), y0, y1);
          z[k] = pack_bf2(y0, y1);
        }
        // through shared memory, so that four lanes write 64 bytes of a row: a lane to a row takes the
        // store unit four times as long, and the barriers' instructions wait behind it
#pragma unroll
        for (int k = 0; k < 4; ++k)
          turn[lane * 4 + (k ^ (lane >> 1 & 3))] = make_uint4(z[4 * k], z[4 * k + 1], z[4 * k + 2], z[4 * k + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int x = 8 * k + (lane >> 2), e = lane & 3;
          if (i - lane + x < I.len)
            reinterpret_cast<uint4*>(A.out + (row_at + (size_t)x * P.q_heads) * D + 32 * c)[e] = turn[x * 4 + (e ^ (x >> 1 & 3))];
        }
        __syncwarp();
      }
      if (there && A.lse) A.lse[at] = LN2F * (m + log2f(l));
      before_sync();
      __syncwarp();
      if (lane == 0) arrive(&C.taken[it % NI]);
    }
    tmem_wait_st();   // of rows that have stopped
  }
  before_sync();
  __syncthreads();
  if (warp == 1) {
    after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  if (C.err) {
    // given up: all rows of the block's pieces
    Walk w = walk_start(P, span, slots, 0, lane);
    Seq s;
    int token, slot;
    for (int it = 0; walk_to(P, w, piece_of(it), lane, s, token, slot); ++it) {
      const Item I = item_of(A, s, token, slot);
      for (int t = 0; t < 2; ++t)
        for (int x = tid; x < BLK && I.q0[t] + x < I.len; x += THREADS) {
          const size_t at = (size_t)(I.first + I.q0[t] + x) * P.q_heads + I.head[t];
          for (int d = 0; d < D; ++d) A.out[at * D + d] = __float2bfloat16_rn(NAN);
          if (A.lse) A.lse[at] = NAN;
        }
    }
  }
}

template <int D>
static sv_status launch(const FwdArgs& A, const void* q, long long qs, const void* k, long long ks, const void* v, long long vs,
                        cudaStream_t st) {
  const int sms = sm_count();
  CUtensorMap mq, mk, mv;
  if (sms < 1 || !raise_smem(reinterpret_cast<const void*>(prompt_forward_kernel<D>), smem_bytes<D>()) ||
      !row_map(&mq, q, A.p.N, A.p.q_heads, D, qs) || !row_map(&mk, k, A.p.N, A.p.kv_heads, D, ks) ||
      !row_map(&mv, v, A.p.N, A.p.kv_heads, D, vs))
    return SV_ERR_CUDA;
  // no more blocks than there can be pieces
  const int span = A.pair_heads ? BLK : 2 * BLK, slots = A.pair_heads ? A.p.q_heads / 2 : A.p.q_heads;
  const long long most = (long long)slots * (A.p.N / span + (A.p.B < A.p.N ? A.p.B : A.p.N));
  prompt_forward_kernel<D><<<(unsigned)(most < sms ? most : sms), THREADS, smem_bytes<D>(), st>>>(A, mq, mk, mv);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace svpr

sv_status spec_prompt_attention(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                                long long v_stride, const int32_t* cu_tokens, int B, int N, int q_heads, int kv_heads,
                                int head_dim, float scale, int window, void* out, float* lse, void* stream) {
  using namespace svpr;
  if (!q || !k || !v || !cu_tokens || !out) return SV_ERR_NULL;
  if (bad_shape(B, N, q_heads, kv_heads, head_dim, scale, window) || bad_stride(q_stride, q_heads, head_dim) ||
      bad_stride(k_stride, kv_heads, head_dim) || bad_stride(v_stride, kv_heads, head_dim))
    return SV_ERR_SHAPE;
  if (!rows_aligned(q, q_stride) || !rows_aligned(k, k_stride) || !rows_aligned(v, v_stride) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(cu_tokens, 4))
    return SV_ERR_ALIGN;
  FwdArgs A = {};
  A.p = Prompts{cu_tokens, B, N, q_heads, kv_heads, q_heads / kv_heads, window < N ? window : 0};
  A.scale = fmaxf(scale * LOG2EF, 1.4e-45f);   // not 0: -inf of what is not seen stays -inf
  A.out = static_cast<__nv_bfloat16*>(out);
  A.lse = lse;
  A.pair_heads = A.p.group % 2 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return head_dim == 128 ? launch<128>(A, q, q_stride, k, k_stride, v, v_stride, st)
                         : launch<64>(A, q, q_stride, k, k_stride, v, v_stride, st);
}

// The gradient of causal attention over packed prompts (C ABI and definitions in
// include/spec_prompt.h).
//
// Three kernels. prompt_rows_kernel leaves delta and lse of each row, head by head, in the
// workspace. prompt_grad_kv_kernel has a tile of 128 keys and walks over the queries that see
// it, of all heads of the group, so that grad_k and grad_v are summed in one place and in one order:
//   S^T = K Q^T, dP^T = V dO^T;  P^T and dS^T as bf16 into TMEM, over S^T and dP^T;
//   grad_v += P^T dO, grad_k += dS^T Q.
// prompt_grad_q_kernel has a tile of 128 queries and walks over its keys: S and dP once more,
// grad_q += dS K. Seven products in the place of the five that one kernel would need, but no
// atomics; and no fp32 sums in memory, except where there are fewer tiles of keys than SMs: there
// pieces of a group's heads are summed through memory, in their order.
// Measured: 12 documents of up to 2,500 tokens, 32 heads on 8 of 128: 738 us, 821 TFLOP/s of the five
// products; rows 46 us (5,700 GB/s), keys' side 367 us (tensor pipe some 63% active), queries' side 295 us
// (some 58%), which begins where the keys' side ends (752 us one after the other; the keys' side
// beginning beside the rows in the same way, 751 us). The keys' side is near what shared memory gives:
// a product of two tiles there reads 64 KB, all that it can in the product's 512 clocks, and 64 KB of
// tiles come in for each unit. Queries have three stages on the keys' side: with two, S waits for its
// copy (788 us when all took 777); waiting for them before P^T dO is issued, 879 us. A unit of the
// queries' side takes some 2,200 clocks, its products 1,650 and its rows, from S to dS, 1,450. dP asked for only
// when dS of the unit before it is there: its kernel 302 us; one wait for a unit's values and the next
// one's keys, which asks for a key stage that is not free yet, 377 us. A lane writing 64 bytes of its
// own row on the way out: 774 us when all took 746.
// Blocks as in the forward kernel: warp 0 walks the work and copies, 1 issues the products, 2-3 see to
// what lies behind a sequence's end, 4-11 have the rows, each half of them 64 columns. Every wait is
// bounded; a block that gives up writes NaN to all of its rows.
#include "prompt_common.cuh"

namespace svpr {

constexpr int THREADS = 384;
constexpr int NI = 4;                    // items announced at a time

struct BwdArgs {
  Prompts p;
  float scale, scale2;                   // scale2: times log2(e)
  const __nv_bfloat16 *go, *out;
  long long go_stride;
  const float* lse;
  __nv_bfloat16 *gq, *gk, *gv;
  float *nlse, *ndelta;                  // workspace [q_heads][N]: -lse log2(e), -delta
  int split;                             // pieces of a group's heads
  float *part_k, *part_v;                // workspace [split][N][kv_heads][D], where split > 1
};

// --- delta and lse of each row. 16 lanes have a row of a head, 8 elements each.
constexpr int ROWS_BLOCK = 64;
template <int D>
__global__ void __launch_bounds__(256) prompt_rows_kernel(const BwdArgs A) {
  constexpr int L = D / 8;               // lanes of a row
  const int h = blockIdx.y, at = threadIdx.x / L, lane = threadIdx.x % L;
#pragma unroll 4
  for (int i = at; i < ROWS_BLOCK; i += 256 / L) {
    const int r = blockIdx.x * ROWS_BLOCK + i;
    float s = 0.f;
    if (r < A.p.N) {
      const uint4 x = *reinterpret_cast<const uint4*>(A.go + (size_t)r * A.go_stride + (size_t)h * D + 8 * lane);
      const uint4 y = *reinterpret_cast<const uint4*>(A.out + ((size_t)r * A.p.q_heads + h) * D + 8 * lane);
      const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s = fmaf(__uint_as_float(a[k] << 16), __uint_as_float(b[k] << 16), s);
        s = fmaf(__uint_as_float(a[k] & 0xFFFF0000u), __uint_as_float(b[k] & 0xFFFF0000u), s);
      }
    }
#pragma unroll
    for (int o = L / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0 && r < A.p.N) {
      A.ndelta[(size_t)h * A.p.N + r] = -s;
      A.nlse[(size_t)h * A.p.N + r] = -A.lse[(size_t)r * A.p.q_heads + h] * LOG2EF;
    }
  }
}

// Rows of a tile from `live` on become zeros: a warp.
template <int D>
__device__ __forceinline__ void clear_tail(unsigned char* tile, int live, int lane) {
  for (int c = 0; c < D / 64; ++c)
    for (int i = live * 128 + 16 * lane; i < COL; i += 512) *reinterpret_cast<uint4*>(tile + c * COL + i) = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}
// 32 columns of a row of TMEM, times f, as bf16, to the lane's row `to` of rows `stride` elements apart, of
// which `rows` are there from the warp's first one on. Four lanes hand one another their parts of 16
// bytes, so that they write 64 bytes of a row together: a lane to a row takes the store unit four times as long.
__device__ __forceinline__ void store32(__nv_bfloat16* to, size_t stride, uint32_t from, float f, int rows) {
  uint32_t y[32], z[4][4];
  tmem_ld32(y, from);
  tmem_wait_ld();
  pin<32>(y);
  const uint64_t f2 = pair(f, f);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    float y0, y1;
    unpair(mul2(pair(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1])), f2), y0, y1);
    z[k >> 2][k & 3] = pack_bf2(y0, y1);
  }
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int round = 1; round <= 2; ++round) {
    const bool odd = lane & round;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c & round) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? z[c][e] : z[c | round][e], round);
        if (odd) z[c][e] = got;
        else z[c | round][e] = got;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)   // part `lane & 3` of row j of the four
    if ((lane & ~3) + j < rows)
      reinterpret_cast<uint4*>(to + ((long long)j - (lane & 3)) * (long long)stride)[lane & 3] =
          make_uint4(z[j][0], z[j][1], z[j][2], z[j][3]);
}
// The same in fp32.
__device__ __forceinline__ void keep32(float* to, uint32_t from, float f, bool there) {
  uint32_t y[32];
  tmem_ld32(y, from);
  tmem_wait_ld();
  pin<32>(y);
  if (!there) return;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    reinterpret_cast<float4*>(to)[k] = make_float4(__uint_as_float(y[4 * k]) * f, __uint_as_float(y[4 * k + 1]) * f,
                                                   __uint_as_float(y[4 * k + 2]) * f, __uint_as_float(y[4 * k + 3]) * f);
}
__device__ __forceinline__ void fill_rows(__nv_bfloat16* p, size_t row, int elements, int lane, int lanes, float x) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, x);
  for (int i = 2 * lane; i < elements; i += 2 * lanes) *reinterpret_cast<__nv_bfloat162*>(p + row * elements + i) = v;
}
// Zeros in the rows outside every sequence, a block of threads to a row.
__device__ __forceinline__ void clear_outside(const Prompts& p, __nv_bfloat16* g, int elements, int tid, int threads) {
  const int before = min(max(p.cu[0], 0), p.N), behind = min(max(p.cu[p.B], 0), p.N);
  for (int x = blockIdx.x; x < before + p.N - behind; x += gridDim.x)
    fill_rows(g, (size_t)(x < before ? x : x + behind - before), elements, tid, threads, 0.f);
}

// A tile of keys (queries) and the tiles of queries (keys) that it goes over.
struct Item {
  int first, len, end;    // of the sequence; end: no item
  int token, head;        // the tile's first token; kv head (query head)
  int h0, h1, part;       // query heads h0 .. h1 - 1 of the kv head, part `part` of them
  int lo, hi;             // tiles lo .. hi - 1, of each of the group's heads (of the kv head)
};

template <int D>
struct KvShape {
  static constexpr int TILE = D / 64 * COL;
  static constexpr int NQ = 3, NO = 2, NS = 2;
};
template <int D>
struct __align__(16) KvCtl {
  using S = KvShape<D>;
  float nlse[S::NS][BLK], ndelta[S::NS][BLK];
  Item item[NI];
  Bar ready[NI], taken[NI], kvfull, kvempty;
  Bar qfull[S::NQ], qseen[S::NQ], qempty[S::NQ], gfull[S::NO], gseen[S::NO], gempty[S::NO], stfull[S::NS], stempty[S::NS];
  Bar sfull, pfull, dpfull, dsfull, ofull, done;
  uint32_t taddr;
  int err;
};
template <int D>
constexpr int kv_smem() {
  return (2 + KvShape<D>::NQ + KvShape<D>::NO) * KvShape<D>::TILE + (int)sizeof(KvCtl<D>);
}
static_assert(kv_smem<128>() <= 227 * 1024, "one block on an SM");

__device__ __forceinline__ Item kv_item(const Prompts& P, int split, const Seq& s, int token, int slot) {
  const int head = slot / split, part = slot - head * split, h0 = P.group * part / split, h1 = P.group * (part + 1) / split;
  const int tiles = (s.len + BLK - 1) / BLK;
  int hi = tiles;
  if (P.window) hi = (int)min((long long)tiles, ((long long)token + BLK - 1 + P.window - 1) / BLK + 1);
  return Item{s.first, s.len, 0, token, head, head * P.group + h0, head * P.group + h1, part, token / BLK, hi};
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    prompt_grad_kv_kernel(const BwdArgs A, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_g) {
  using S = KvShape<D>;
  constexpr int TILE = S::TILE, NQ = S::NQ, NO = S::NO, NS = S::NS;
  extern __shared__ __align__(1024) unsigned char smem_aligned[];   // no room to round up
  unsigned char* smem = smem_aligned;
  unsigned char *sk = smem, *sv = sk + TILE, *sq = sv + TILE, *sg = sq + NQ * TILE;
  KvCtl<D>& C = *reinterpret_cast<KvCtl<D>*>(sg + NO * TILE);
  volatile int* err = &C.err;
  const Prompts& P = A.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the queries' side needs only what the rows' kernel left
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (tid == 0) {
    for (int i = 0; i < NI; ++i) bar_init(&C.ready[i], 1), bar_init(&C.taken[i], THREADS / 32 - 1);
    for (int i = 0; i < NQ; ++i) bar_init(&C.qfull[i], 1), bar_init(&C.qseen[i], 1), bar_init(&C.qempty[i], 1);
    for (int i = 0; i < NO; ++i) bar_init(&C.gfull[i], 1), bar_init(&C.gseen[i], 1), bar_init(&C.gempty[i], 1);
    for (int i = 0; i < NS; ++i) bar_init(&C.stfull[i], 2), bar_init(&C.stempty[i], 8);
    bar_init(&C.kvfull, 1), bar_init(&C.kvempty, 1), bar_init(&C.sfull, 1), bar_init(&C.dpfull, 1);
    bar_init(&C.pfull, 8), bar_init(&C.dsfull, 8), bar_init(&C.ofull, 1), bar_init(&C.done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    C.err = (smem_u32(smem) & 1023) != 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&C.taddr)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    before_sync();
  }
  __syncthreads();
  after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, C.taddr, 0), ts = tmem, tp = tmem + 128, tv = tmem + 256, tk = tmem + 384;

  if (warp < 4) {
    // registers: 128 x 72 and 256 x 216 are the 384 x 168 of the launch
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // --- the walk, and the copies
      Walk w = walk_start(P, BLK, P.kv_heads * A.split, 1, lane);
      int u = 0, items = 0, asked_g = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        Seq s;
        int token, slot;
        const bool on = walk_to(P, w, piece_of(it), lane, s, token, slot);
        const Item I = on ? kv_item(P, A.split, s, token, slot) : Item{0, 0, 1, 0, 0, 0, 0, 0, 0, 0};
        if (it >= NI) ok = wait_warp(&C.taken[it % NI], (uint32_t)(it / NI - 1) & 1, err);
        if (!ok) break;
        if (lane == 0) {
          C.item[it % NI] = I;
          arrive(&C.ready[it % NI]);
        }
        if (!on) break;
        if (items) ok = wait_warp(&C.kvempty, (uint32_t)(items - 1) & 1, err);
        if (!ok) break;
        if (lane == 0) {
          expect(&C.kvfull, 2 * TILE);
          copy_tile<D>(sk, &map_k, I.head, I.first + I.token, &C.kvfull);
          copy_tile<D>(sv, &map_v, I.head, I.first + I.token, &C.kvfull);
        }
        ++items;
        for (int h = I.h0; h < I.h1 && ok; ++h)
          for (int i = I.lo; i < I.hi; ++i) {
            if (u >= NQ) ok = wait_warp(&C.qempty[u % NQ], (uint32_t)(u / NQ - 1) & 1, err);
            if (!ok) break;
            if (lane == 0) {
              expect(&C.qfull[u % NQ], TILE);
              copy_tile<D>(sq + (u % NQ) * TILE, &map_q, h, I.first + BLK * i, &C.qfull[u % NQ]);
            }
            ++u;
            if (u > NO) ok = wait_warp(&C.gempty[(u - 1) % NO], (uint32_t)((u - 1) / NO - 1) & 1, err);
            if (!ok) break;
            if (lane == 0) {
              expect(&C.gfull[(u - 1) % NO], TILE);
              copy_tile<D>(sg + ((u - 1) % NO) * TILE, &map_g, h, I.first + BLK * i, &C.gfull[(u - 1) % NO]);
            }
            asked_g = u;
          }
      }
      // what was asked for lands before the block ends, also when the others have stopped
      if (lane == 0) {
        int never = 0;
        for (int i = max(0, u - NQ); i < u; ++i) wait(&C.qfull[i % NQ], (uint32_t)(i / NQ) & 1, &never, LAND_NS);
        for (int i = max(0, asked_g - NO); i < asked_g; ++i) wait(&C.gfull[i % NO], (uint32_t)(i / NO) & 1, &never, LAND_NS);
        if (items) wait(&C.kvfull, (uint32_t)(items - 1) & 1, &never, LAND_NS);
      }
      __syncwarp();
    } else if (warp == 1) {
      // --- products. While dS of a unit is formed, the tensor cores add its P^T dO and form the next S;
      // while the next P is formed, they add dS^T Q and form the next dP. The warp stays together, so
      // that addresses and descriptors are the same in all of it; one lane issues.
      int u = 0;
      bool ok = true;
      const auto scores = [&](int x) {
        ok = wait_warp(&C.qseen[x % NQ], (uint32_t)(x / NQ) & 1, err);
        if (!ok) return;
        after_sync();
        if (elect()) {
          mma_dims<D>(ts, sk, sq + (x % NQ) * TILE);
          commit(&C.sfull);
        }
        __syncwarp();
      };
      const auto products = [&](int x, bool last) {
        ok = wait_warp(&C.gseen[x % NO], (uint32_t)(x / NO) & 1, err);
        if (!ok) return;
        after_sync();
        if (elect()) {
          mma_dims<D>(tp, sv, sg + (x % NO) * TILE);
          commit(&C.dpfull);
          if (last) commit(&C.kvempty);
        }
        __syncwarp();
      };
      for (int it = 0; ok; ++it) {
        ok = wait_warp(&C.ready[it % NI], (uint32_t)(it / NI) & 1, err);
        if (!ok) break;
        const Item& I = C.item[it % NI];
        const int end = __shfl_sync(0xffffffffu, I.end, 0), n = __shfl_sync(0xffffffffu, (I.h1 - I.h0) * (I.hi - I.lo), 0);
        if (end) break;
        if (lane == 0) arrive(&C.taken[it % NI]);
        ok = wait_warp(&C.kvfull, (uint32_t)it & 1, err);
        if (ok) scores(u);
        if (ok) products(u, n == 1);
        for (int x = 0; x < n && ok; ++x, ++u) {
          const bool more = x + 1 < n;
          ok = wait_warp(&C.pfull, (uint32_t)u & 1, err);
          if (!ok) break;
          after_sync();
          if (elect()) {
            mma_rows<D>(tv, ts, sg + (u % NO) * TILE, x != 0, 32);
            commit(&C.gempty[u % NO]);
          }
          __syncwarp();
          if (more) scores(u + 1);
          if (ok) ok = wait_warp(&C.dsfull, (uint32_t)u & 1, err);
          if (!ok) break;
          after_sync();
          if (elect()) {
            mma_rows<D>(tk, tp, sq + (u % NQ) * TILE, x != 0, 32);
            commit(&C.qempty[u % NQ]);
            if (!more) commit(&C.ofull);
          }
          __syncwarp();
          if (more) products(u + 1, x + 2 == n);
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
      // --- warp 2: queries and lse, warp 3: grad_out and delta. Rows behind the sequence's end are
      // zeros, with a weight of 0.
      const bool g = warp == 3;
      int u = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        ok = wait_warp(&C.ready[it % NI], (uint32_t)(it / NI) & 1, err);
        if (!ok) break;
        const Item& I = C.item[it % NI];
        if (I.end) break;
        for (int h = I.h0; h < I.h1 && ok; ++h)
          for (int i = I.lo; i < I.hi; ++i, ++u) {
            const int live = I.len - BLK * i, x = g ? u % NO : u % NQ, y = u % NS;
            const float* from = (g ? A.ndelta : A.nlse) + (size_t)h * P.N + I.first + BLK * i;
            float f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = lane + 32 * k < live ? from[lane + 32 * k] : g ? 0.f : -INFINITY;
            ok = wait_warp(g ? &C.gfull[x] : &C.qfull[x], (uint32_t)(g ? u / NO : u / NQ) & 1, err);
            if (!ok) break;
            if (live < BLK) clear_tail<D>((g ? sg : sq) + x * TILE, live, lane);
            if (lane == 0) arrive(g ? &C.gseen[x] : &C.qseen[x]);
            if (u >= NS) ok = wait_warp(&C.stempty[y], (uint32_t)(u / NS - 1) & 1, err);
            if (!ok) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) (g ? C.ndelta : C.nlse)[y][lane + 32 * k] = f[k];
            __syncwarp();
            if (lane == 0) arrive(&C.stfull[y]);
          }
        if (lane == 0) arrive(&C.taken[it % NI]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // --- key r of the tile, queries 64 half .. 64 half + 63 of a unit
    const int half = (warp - 4) >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, mine = lanes + 64 * half;
    clear_outside(P, A.gk, P.kv_heads * D, tid - 128, 256);
    clear_outside(P, A.gv, P.kv_heads * D, tid - 128, 256);
    int u = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      ok = wait_warp(&C.ready[it % NI], (uint32_t)(it / NI) & 1, err);
      if (!ok) break;
      const Item& I = C.item[it % NI];
      if (I.end) break;
      const int n = (I.h1 - I.h0) * (I.hi - I.lo);
      int i = I.lo;
#pragma unroll 1
      for (int x = 0; x < n; ++x, ++u) {
        const int y = u % NS, q0 = BLK * i;
        if (++i == I.hi) i = I.lo;
        ok = wait_warp(&C.stfull[y], (uint32_t)(u / NS) & 1, err) && wait_warp(&C.sfull, (uint32_t)u & 1, err);
        if (!ok) break;
        after_sync();
        uint32_t p[64];
        tmem_ld32(p, ts + mine);
        tmem_ld32(p + 32, ts + mine + 32);
        tmem_wait_ld();
        pin<64>(p);
        if (q0 < I.token + BLK - 1 || (P.window && q0 + BLK - 1 - I.token >= P.window)) {
          // query c of the half sees the key if c >= lo and, in a window, c < lo + window
          const int lo = I.token + r - q0 - 64 * half, hi = P.window ? lo + P.window : 1 << 30;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < lo) p[c] = 0xFF800000u;
          if (P.window)
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c >= hi) p[c] = 0xFF800000u;
        }
        const uint64_t a = pair(A.scale2, A.scale2);
        const float4* nl = reinterpret_cast<const float4*>(C.nlse[y] + 64 * half);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t z[16];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float4 b = nl[8 * c + k / 2];
            const int e = 32 * c + 2 * k;
            float y0, y1, y2, y3;
            unpair(fma2(pair(__uint_as_float(p[e]), __uint_as_float(p[e + 1])), a, pair(b.x, b.y)), y0, y1);
            unpair(fma2(pair(__uint_as_float(p[e + 2]), __uint_as_float(p[e + 3])), a, pair(b.z, b.w)), y2, y3);
            y0 = ex2f(y0), y1 = ex2f(y1), y2 = ex2f(y2), y3 = ex2f(y3);
            z[k] = pack_bf2(y0, y1);
            z[k + 1] = pack_bf2(y2, y3);
            p[e] = __float_as_uint(y0), p[e + 1] = __float_as_uint(y1);
            p[e + 2] = __float_as_uint(y2), p[e + 3] = __float_as_uint(y3);
          }
          tmem_st16(ts + mine + 16 * c, z);
        }
        tmem_wait_st();
        before_sync();
        __syncwarp();
        if (lane == 0) arrive(&C.pfull);
        ok = wait_warp(&C.dpfull, (uint32_t)u & 1, err);
        if (!ok) break;
        after_sync();
        uint32_t d[64];
        tmem_ld32(d, tp + mine);
        tmem_ld32(d + 32, tp + mine + 32);
        tmem_wait_ld();
        pin<64>(d);
        const float4* nd = reinterpret_cast<const float4*>(C.ndelta[y] + 64 * half);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t z[16];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float4 b = nd[8 * c + k / 2];
            const int e = 32 * c + 2 * k;
            float y0, y1, y2, y3;
            unpair(mul2(add2(pair(__uint_as_float(d[e]), __uint_as_float(d[e + 1])), pair(b.x, b.y)),
                        pair(__uint_as_float(p[e]), __uint_as_float(p[e + 1]))), y0, y1);
            unpair(mul2(add2(pair(__uint_as_float(d[e + 2]), __uint_as_float(d[e + 3])), pair(b.z, b.w)),
                        pair(__uint_as_float(p[e + 2]), __uint_as_float(p[e + 3]))), y2, y3);
            z[k] = pack_bf2(y0, y1);
            z[k + 1] = pack_bf2(y2, y3);
          }
          tmem_st16(tp + mine + 16 * c, z);
        }
        tmem_wait_st();
        before_sync();
        __syncwarp();
        if (lane == 0) {
          arrive(&C.dsfull);
          arrive(&C.stempty[y]);
        }
      }
      if (!ok) break;
      ok = wait_warp(&C.ofull, (uint32_t)it & 1, err);
      if (!ok) break;
      after_sync();
      const bool there = I.token + r < I.len;
      const size_t at = ((size_t)(I.first + I.token + r) * P.kv_heads + I.head) * D;
      if (A.split > 1) {
        float* to = (half ? A.part_k : A.part_v) + (size_t)I.part * P.N * P.kv_heads * D + at;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) keep32(to + c, (half ? tk : tv) + lanes + c, half ? A.scale : 1.f, there);
      } else {
#pragma unroll 1
        for (int c = 0; c < D; c += 32)
          store32((half ? A.gk : A.gv) + at + c, (size_t)P.kv_heads * D, (half ? tk : tv) + lanes + c, half ? A.scale : 1.f,
                  I.len - I.token - (r & ~31));
      }
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
    Walk w = walk_start(P, BLK, P.kv_heads * A.split, 1, lane);
    Seq s;
    int token, slot;
    for (int it = 0; walk_to(P, w, piece_of(it), lane, s, token, slot); ++it)
      for (int x = token + warp; x < min(token + BLK, s.len); x += THREADS / 32) {
        const size_t row = (size_t)(s.first + x) * P.kv_heads + slot / A.split;
        if (A.split > 1) {   // the sum of the parts becomes NaN
          const size_t at = ((size_t)(slot % A.split) * P.N * P.kv_heads + row) * D;
          for (int d = lane; d < D; d += 32) A.part_k[at + d] = A.part_v[at + d] = NAN;
        } else {
          fill_rows(A.gk, row, D, lane, 32, NAN);
          fill_rows(A.gv, row, D, lane, 32, NAN);
        }
      }
  }
}

// The parts' sum, in their order; rows outside every sequence have been written.
template <int D>
__global__ void __launch_bounds__(256) prompt_sum_kernel(const BwdArgs A) {
  const long long n = (long long)A.p.N * A.p.kv_heads * D / 4, x = (long long)blockIdx.x * 256 + threadIdx.x;
  if (x >= n) return;
  const int r = (int)(x / (A.p.kv_heads * (D / 4)));
  if (r < min(max(A.p.cu[0], 0), A.p.N) || r >= min(max(A.p.cu[A.p.B], 0), A.p.N)) return;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const float4* from = reinterpret_cast<const float4*>(v ? A.part_v : A.part_k) + x;
    float4 sum = from[0];
    for (int p = 1; p < A.split; ++p) {
      const float4 y = from[p * n];
      sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
    }
    reinterpret_cast<uint2*>(v ? A.gv : A.gk)[x] = make_uint2(pack_bf2(sum.x, sum.y), pack_bf2(sum.z, sum.w));
  }
}

template <int D>
struct QShape {
  static constexpr int TILE = D / 64 * COL;
  static constexpr int NK = 3, NV = 2;
};
template <int D>
struct __align__(16) QCtl {
  using S = QShape<D>;
  Item item[NI];
  Bar ready[NI], taken[NI], qfull, qempty;
  Bar kfull[S::NK], kseen[S::NK], kempty[S::NK], vfull[S::NV], vseen[S::NV], vempty[S::NV];
  Bar sfull[2], sread[2], dpfull[2], dsfull[2], ofull, done;
  uint32_t taddr;
  int err;
};
template <int D>
constexpr int q_smem() {
  return 1024 + (2 + QShape<D>::NK + QShape<D>::NV) * QShape<D>::TILE + (int)sizeof(QCtl<D>);
}
static_assert(q_smem<128>() <= 227 * 1024, "one block on an SM");

__device__ __forceinline__ Item q_item(const Prompts& P, const Seq& s, int token, int slot) {
  return Item{s.first, s.len, 0, token, slot, slot, slot + 1, 0, P.window ? max(token - P.window + 1, 0) / BLK : 0, token / BLK + 1};
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    prompt_grad_q_kernel(const BwdArgs A, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_g) {
  using S = QShape<D>;
  constexpr int TILE = S::TILE, NK = S::NK, NV = S::NV;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char *sq = smem, *sg = sq + TILE, *sk = sg + TILE, *sv = sk + NK * TILE;
  QCtl<D>& C = *reinterpret_cast<QCtl<D>*>(sv + NV * TILE);
  volatile int* err = &C.err;
  const Prompts& P = A.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NI; ++i) bar_init(&C.ready[i], 1), bar_init(&C.taken[i], THREADS / 32 - 1);
    for (int i = 0; i < NK; ++i) bar_init(&C.kfull[i], 1), bar_init(&C.kseen[i], 1), bar_init(&C.kempty[i], 1);
    for (int i = 0; i < NV; ++i) bar_init(&C.vfull[i], 1), bar_init(&C.vseen[i], 1), bar_init(&C.vempty[i], 1);
    for (int i = 0; i < 2; ++i)
      bar_init(&C.sfull[i], 1), bar_init(&C.sread[i], 8), bar_init(&C.dpfull[i], 1), bar_init(&C.dsfull[i], 8);
    bar_init(&C.qfull, 1), bar_init(&C.qempty, 1), bar_init(&C.ofull, 1), bar_init(&C.done, 1);
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
  const uint32_t tmem = __shfl_sync(0xffffffffu, C.taddr, 0), to = tmem + 384;
  // Three places of 128 columns in turn: S of a unit; dP of the next one there as soon as S has been read;
  // dS over that dP; and then S of the unit after it.
  const auto s_at = [&](int u) { return tmem + 128 * (u % 3); };
  const auto dp_at = [&](int u) { return tmem + 128 * ((u + 2) % 3); };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // --- the walk, and the copies
      Walk w = walk_start(P, BLK, P.q_heads, 0, lane);
      int u = 0, asked_v = 0, items = 0;
      bool ok = true;
      // of unit u: the values' place is free before the keys'
      const auto copy_unit = [&](int kv, int row) {
        if (u >= NV) ok = wait_warp(&C.vempty[u % NV], (uint32_t)(u / NV - 1) & 1, err);
        if (!ok) return;
        if (lane == 0) {
          expect(&C.vfull[u % NV], TILE);
          copy_tile<D>(sv + (u % NV) * TILE, &map_v, kv, row, &C.vfull[u % NV]);
        }
        asked_v = u + 1;
        if (u >= NK) ok = wait_warp(&C.kempty[u % NK], (uint32_t)(u / NK - 1) & 1, err);
        if (!ok) return;
        if (lane == 0) {
          expect(&C.kfull[u % NK], TILE);
          copy_tile<D>(sk + (u % NK) * TILE, &map_k, kv, row, &C.kfull[u % NK]);
        }
        ++u;
      };
      for (int it = 0; ok; ++it) {
        Seq s;
        int token, slot;
        const bool on = walk_to(P, w, piece_of(it), lane, s, token, slot);
        const Item I = on ? q_item(P, s, token, slot) : Item{0, 0, 1, 0, 0, 0, 0, 0, 0, 0};
        if (it >= NI) ok = wait_warp(&C.taken[it % NI], (uint32_t)(it / NI - 1) & 1, err);
        if (!ok) break;
        if (lane == 0) {
          C.item[it % NI] = I;
          arrive(&C.ready[it % NI]);
        }
        if (!on) break;
        // the first unit's before the queries, which the item before needs longer
        const int kv = I.head / P.group;
        copy_unit(kv, I.first + BLK * I.lo);
        if (ok && items) ok = wait_warp(&C.qempty, (uint32_t)(items - 1) & 1, err);
        if (!ok) break;
        if (lane == 0) {
          expect(&C.qfull, 2 * TILE);
          copy_tile<D>(sq, &map_q, I.head, I.first + I.token, &C.qfull);
          copy_tile<D>(sg, &map_g, I.head, I.first + I.token, &C.qfull);
        }
        ++items;
        for (int j = I.lo + 1; j < I.hi && ok; ++j) copy_unit(kv, I.first + BLK * j);
      }
      // what was asked for lands before the block ends, also when the others have stopped
      if (lane == 0) {
        int never = 0;
        for (int i = max(0, u - NK); i < u; ++i) wait(&C.kfull[i % NK], (uint32_t)(i / NK) & 1, &never, LAND_NS);
        for (int i = max(0, asked_v - NV); i < asked_v; ++i) wait(&C.vfull[i % NV], (uint32_t)(i / NV) & 1, &never, LAND_NS);
        if (items) wait(&C.qfull, (uint32_t)(items - 1) & 1, &never, LAND_NS);
      }
      __syncwarp();
    } else if (warp == 1) {
      // --- products: S two units ahead, dP one, as soon as S of the unit before it has been read
      int u = 0;
      bool ok = true;
      const auto scores = [&](int x) {
        ok = wait_warp(&C.kseen[x % NK], (uint32_t)(x / NK) & 1, err);
        if (!ok) return;
        after_sync();
        if (elect()) {
          mma_dims<D>(s_at(x), sq, sk + (x % NK) * TILE);
          commit(&C.sfull[x & 1]);
        }
        __syncwarp();
      };
      const auto products = [&](int x) {   // by the lane that issues
        mma_dims<D>(dp_at(x), sg, sv + (x % NV) * TILE);
        commit(&C.dpfull[x & 1]);
        commit(&C.vempty[x % NV]);
      };
      for (int it = 0; ok; ++it) {
        ok = wait_warp(&C.ready[it % NI], (uint32_t)(it / NI) & 1, err);
        if (!ok) break;
        const Item& I = C.item[it % NI];
        const int end = __shfl_sync(0xffffffffu, I.end, 0), n = __shfl_sync(0xffffffffu, I.hi - I.lo, 0);
        if (end) break;
        if (lane == 0) arrive(&C.taken[it % NI]);
        ok = wait_warp(&C.qfull, (uint32_t)it & 1, err);
        if (ok) scores(u);
        if (ok) ok = wait_warp(&C.vseen[u % NV], (uint32_t)(u / NV) & 1, err);
        if (!ok) break;
        after_sync();
        if (elect()) {
          products(u);
          if (n == 1) commit(&C.qempty);
        }
        __syncwarp();
        if (n > 1) scores(u + 1);
        for (int x = 0; x < n && ok; ++x, ++u) {
          if (x + 1 < n) {
            ok = wait_warp(&C.vseen[(u + 1) % NV], (uint32_t)((u + 1) / NV) & 1, err);
            if (ok) ok = wait_warp(&C.sread[u & 1], (uint32_t)(u >> 1) & 1, err);
            if (!ok) break;
            after_sync();
            if (elect()) {
              products(u + 1);
              if (x + 2 == n) commit(&C.qempty);
            }
            __syncwarp();
          }
          ok = wait_warp(&C.dsfull[u & 1], (uint32_t)(u >> 1) & 1, err);
          if (!ok) break;
          after_sync();
          if (elect()) {
            mma_rows<D>(to, dp_at(u), sk + (u % NK) * TILE, x != 0, 32);
            commit(&C.kempty[u % NK]);
            if (x + 1 == n) commit(&C.ofull);
          }
          __syncwarp();
          if (x + 2 < n) scores(u + 2);
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
      // --- warp 2: keys, warp 3: values: rows behind the sequence's end are zeros
      const bool v = warp == 3;
      int u = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        ok = wait_warp(&C.ready[it % NI], (uint32_t)(it / NI) & 1, err);
        if (!ok) break;
        const Item& I = C.item[it % NI];
        if (I.end) break;
        for (int j = I.lo; j < I.hi; ++j, ++u) {
          const int live = I.len - BLK * j, x = v ? u % NV : u % NK;
          ok = wait_warp(v ? &C.vfull[x] : &C.kfull[x], (uint32_t)(v ? u / NV : u / NK) & 1, err);
          if (!ok) break;
          if (live < BLK) clear_tail<D>((v ? sv : sk) + x * TILE, live, lane);
          if (lane == 0) arrive(v ? &C.vseen[x] : &C.kseen[x]);
        }
        if (lane == 0) arrive(&C.taken[it % NI]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // --- query r of the tile, keys 64 half .. 64 half + 63 of a unit
    const int half = (warp - 4) >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, mine = lanes + 64 * half;
    clear_outside(P, A.gq, P.q_heads * D, tid - 128, 256);
    int u = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      ok = wait_warp(&C.ready[it % NI], (uint32_t)(it / NI) & 1, err);
      if (!ok) break;
      const Item& I = C.item[it % NI];
      if (I.end) break;
      const bool there = I.token + r < I.len;
      const int row = I.first + I.token + (there ? r : 0);
      const float nl = A.nlse[(size_t)I.head * P.N + row], nd = A.ndelta[(size_t)I.head * P.N + row];
      const uint64_t a = pair(A.scale2, A.scale2), nl2 = pair(nl, nl), nd2 = pair(nd, nd);
#pragma unroll 1
      for (int j = I.lo; j < I.hi; ++j, ++u) {
        ok = wait_warp(&C.sfull[u & 1], (uint32_t)(u >> 1) & 1, err);
        if (!ok) break;
        after_sync();
        const uint32_t ts = s_at(u) + mine, tp = dp_at(u) + mine;
        uint32_t p[64];
        tmem_ld32(p, ts);
        tmem_ld32(p + 32, ts + 32);
        tmem_wait_ld();
        pin<64>(p);
        before_sync();
        __syncwarp();
        if (lane == 0) arrive(&C.sread[u & 1]);
        const int k0 = BLK * j;
        if (k0 + BLK - 1 > I.token || (P.window && k0 <= I.token + BLK - 1 - P.window)) {
          // the query sees key c of the half if c <= hi and, in a window, c > hi - window
          const int hi = I.token + r - k0 - 64 * half, lo = P.window ? hi - P.window : -1;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c > hi) p[c] = 0xFF800000u;
          if (P.window)
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c <= lo) p[c] = 0xFF800000u;
        }
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          float y0, y1;
          unpair(fma2(pair(__uint_as_float(p[c]), __uint_as_float(p[c + 1])), a, nl2), y0, y1);
          p[c] = __float_as_uint(ex2f(y0)), p[c + 1] = __float_as_uint(ex2f(y1));
        }
        ok = wait_warp(&C.dpfull[u & 1], (uint32_t)(u >> 1) & 1, err);
        if (!ok) break;
        after_sync();
        uint32_t d[64];
        tmem_ld32(d, tp);
        tmem_ld32(d + 32, tp + 32);
        tmem_wait_ld();
        pin<64>(d);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t z[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int e = 32 * c + 2 * k;
            float y0, y1;
            unpair(mul2(add2(pair(__uint_as_float(d[e]), __uint_as_float(d[e + 1])), nd2),
                        pair(__uint_as_float(p[e]), __uint_as_float(p[e + 1]))), y0, y1);
            z[k] = pack_bf2(y0, y1);
          }
          tmem_st16(tp + 16 * c, z);
        }
        tmem_wait_st();
        before_sync();
        __syncwarp();
        if (lane == 0) arrive(&C.dsfull[u & 1]);
      }
      if (!ok) break;
      ok = wait_warp(&C.ofull, (uint32_t)it & 1, err);
      if (!ok) break;
      after_sync();
      const size_t at = ((size_t)(I.first + I.token + r) * P.q_heads + I.head) * D;
#pragma unroll 1
      for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32)
        store32(A.gq + at + c, (size_t)P.q_heads * D, to + lanes + c, A.scale, I.len - I.token - (r & ~31));
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
    Walk w = walk_start(P, BLK, P.q_heads, 0, lane);
    Seq s;
    int token, slot;
    for (int it = 0; walk_to(P, w, piece_of(it), lane, s, token, slot); ++it)
      for (int x = token + warp; x < min(token + BLK, s.len); x += THREADS / 32)
        fill_rows(A.gq, (size_t)(s.first + x) * P.q_heads + slot, D, lane, 32, NAN);
  }
  // this grid ends only after the one before it
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

static long long most_tiles(int B, int N) { return N / BLK + (B < N ? B : N); }
// Pieces of a group's heads in prompt_grad_kv_kernel: where there are fewer tiles than SMs, as many as
// give each SM one or two (5 texts of up to 333 tokens, 14 heads on 2 of 64: 35 us a call in 7 pieces, 53 in
// one).
static int split_of(int B, int N, int q_heads, int kv_heads, int sms) {
  const long long pieces = most_tiles(B, N) * kv_heads, most = sms * 3ll / 2 / pieces;
  return (int)(most < 1 ? 1 : most < q_heads / kv_heads ? most : q_heads / kv_heads);
}
static size_t rows_bytes(int N, int q_heads) { return (2 * (size_t)N * q_heads * sizeof(float) + 127) & ~(size_t)127; }

template <int D>
static sv_status launch(const BwdArgs& A, const void* q, long long qs, const void* k, long long ks, const void* v, long long vs,
                        cudaStream_t st) {
  const Prompts& P = A.p;
  const int sms = sm_count();
  CUtensorMap mq, mk, mv, mg;
  if (sms < 1 || !raise_smem(reinterpret_cast<const void*>(prompt_grad_kv_kernel<D>), kv_smem<D>()) ||
      !raise_smem(reinterpret_cast<const void*>(prompt_grad_q_kernel<D>), q_smem<D>()) ||
      !row_map(&mq, q, P.N, P.q_heads, D, qs) || !row_map(&mk, k, P.N, P.kv_heads, D, ks) ||
      !row_map(&mv, v, P.N, P.kv_heads, D, vs) || !row_map(&mg, A.go, P.N, P.q_heads, D, A.go_stride))
    return SV_ERR_CUDA;
  prompt_rows_kernel<D><<<dim3((P.N + ROWS_BLOCK - 1) / ROWS_BLOCK, P.q_heads), 256, 0, st>>>(A);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  // no more blocks than there can be pieces
  const long long tiles = most_tiles(P.B, P.N), nk = tiles * P.kv_heads * A.split, nq = tiles * P.q_heads;
  prompt_grad_kv_kernel<D><<<(unsigned)(nk < sms ? nk : sms), THREADS, kv_smem<D>(), st>>>(A, mq, mk, mv, mg);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  // beside the keys' side: in SMs that it has left, or never took
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(nq < sms ? nq : sms));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = q_smem<D>();
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, prompt_grad_q_kernel<D>, A, mq, mk, mv, mg) != cudaSuccess) return SV_ERR_CUDA;
  if (A.split > 1) prompt_sum_kernel<D><<<(unsigned)(((long long)P.N * P.kv_heads * D / 4 + 255) / 256), 256, 0, st>>>(A);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace svpr

size_t spec_prompt_attention_backward_workspace_bytes(int B, int N, int q_heads, int kv_heads, int head_dim) {
  using namespace svpr;
  if (bad_shape(B, N, q_heads, kv_heads, head_dim, 1.f, 0)) return 0;
  const int sms = sm_count(), split = sms < 1 ? 1 : split_of(B, N, q_heads, kv_heads, sms);
  const size_t part = split > 1 ? (size_t)split * N * kv_heads * head_dim * sizeof(float) : 0;
  return sms < 1 ? 0 : rows_bytes(N, q_heads) + 2 * part;
}

sv_status spec_prompt_attention_backward(const void* grad_out, long long go_stride, const void* q, long long q_stride,
                                         const void* k, long long k_stride, const void* v, long long v_stride,
                                         const void* out, const float* lse, const int32_t* cu_tokens, int B, int N,
                                         int q_heads, int kv_heads, int head_dim, float scale, int window,
                                         void* grad_q, void* grad_k, void* grad_v, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  using namespace svpr;
  if (!grad_out || !q || !k || !v || !out || !lse || !cu_tokens || !grad_q || !grad_k || !grad_v || !workspace)
    return SV_ERR_NULL;
  if (bad_shape(B, N, q_heads, kv_heads, head_dim, scale, window) || bad_stride(q_stride, q_heads, head_dim) ||
      bad_stride(k_stride, kv_heads, head_dim) || bad_stride(v_stride, kv_heads, head_dim) ||
      bad_stride(go_stride, q_heads, head_dim))
    return SV_ERR_SHAPE;
  if (!rows_aligned(q, q_stride) || !rows_aligned(k, k_stride) || !rows_aligned(v, v_stride) ||
      !rows_aligned(grad_out, go_stride) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(cu_tokens, 4) ||
      !aligned(grad_q, 16) || !aligned(grad_k, 16) || !aligned(grad_v, 16))
    return SV_ERR_ALIGN;
  const int sms = aligned(workspace, 16) ? sm_count() : 1;
  if (sms < 1) return SV_ERR_CUDA;
  if (!aligned(workspace, 16) ||
      workspace_bytes < spec_prompt_attention_backward_workspace_bytes(B, N, q_heads, kv_heads, head_dim))
    return SV_ERR_WORKSPACE;
  BwdArgs A = {};
  A.p = Prompts{cu_tokens, B, N, q_heads, kv_heads, q_heads / kv_heads, window < N ? window : 0};
  A.scale = scale;
  A.scale2 = fmaxf(scale * LOG2EF, 1.4e-45f);   // not 0: -inf of what is not seen stays -inf
  A.go = static_cast<const __nv_bfloat16*>(grad_out), A.out = static_cast<const __nv_bfloat16*>(out);
  A.go_stride = go_stride;
  A.lse = lse;
  A.gq = static_cast<__nv_bfloat16*>(grad_q), A.gk = static_cast<__nv_bfloat16*>(grad_k);
  A.gv = static_cast<__nv_bfloat16*>(grad_v);
  A.nlse = static_cast<float*>(workspace);
  A.ndelta = A.nlse + (size_t)N * q_heads;
  A.split = split_of(B, N, q_heads, kv_heads, sms);
  A.part_k = reinterpret_cast<float*>(static_cast<char*>(workspace) + rows_bytes(N, q_heads));
  A.part_v = A.part_k + (size_t)A.split * N * kv_heads * head_dim;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return head_dim == 128 ? launch<128>(A, q, q_stride, k, k_stride, v, v_stride, st)
                         : launch<64>(A, q, q_stride, k, k_stride, v, v_stride, st);
}

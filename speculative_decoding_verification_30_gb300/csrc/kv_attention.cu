// Attention of a window of new tokens over the paged 8-bit cache (C ABI and
// definitions in include/spec_kv.h).
//
// A window has few query rows (new tokens x query heads of a kv head) and reads the
// whole cache once, so the bound is HBM: 2 head_dim bytes for each cached token and
// kv head. The work is cut into units of 64 or 128 cached tokens of one item = (sequence,
// kv head, tile of up to 8 NT query rows), and every block takes an equal share of
// all units, whatever the sequences' lengths. A fifth warp walks the share and has its
// units copied into a ring of shared-memory stages (TMA, one box for each page and
// array, swizzled so that the fragments' loads meet no bank conflict), handing each
// over at a block barrier once it is there. An item that lies within one block's
// share is written out; the others leave (max, sum, weighted values) in the workspace
// for kv_combine_kernel.
//
// Both products are transposed, S^T = K Q^T and O^T += V^T P^T, so that the cached
// tokens (and head_dim) fill the 16-row side of the matrix instruction and the query
// rows only its 8-column side: 20 rows cost 24 and not 32. The four warps split the
// unit's tokens for the first product and head_dim for the second: every code is
// widened to fp16 once (exact), and a warp accumulates only a quarter of the output,
// which leaves registers for three or four blocks on an SM. Both contractions may
// take their index in any order, so each lane loads neighbouring bytes and calls
// them whatever the fragment wants. The value scale of a page enters through the
// exponent (weight 2^(s + log2 scale - m)) and the key scale through the logit.
// Measured: 64 sequences of up to 16,000 tokens, 5 new ones, 32 heads on 8: 198 us, 5,440
// GB/s, with the matrix pipe at a third and issue at 40%; 4 of 131,000 tokens, 64 heads on
// 8: 154 us, 4,980 GB/s; 1 of 2,500 tokens 13.4 us, latency.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kv_common.cuh"
#include "launch_cache.h"

namespace svkv {

constexpr int NWARP = 4, NTHR = 32 * NWARP;   // computing; one warp more copies
constexpr int MAX_NT = 8;      // query rows of an item: 8 NT
// What an item costs besides its tokens, in units: its queries, its frame, its end. 64
// sequences of 0 to 16,000 tokens: 195 us with 5, 203 with 3, 236 with 1, 198 with 8.
constexpr int OVERHEAD = 5;
// Units of a block at least: smaller shares cost more to join than they save (1 sequence
// of 2,500 tokens: 13.7 us with 4, 17.5 with 1, 15.4 with 8).
constexpr int MIN_SHARE = 4;
// Weights are 2^(t - m) with m = LIFT below the running maximum of the exponents t,
// and m moves only when a weight would exceed 2^TOP: they stay within fp16 (65504)
// and the small ones keep as much of its range as there is.
constexpr float LIFT = 7.f, TOP = 15.f;
constexpr float NO_FRAME = -1e30f;   // m of a row that has seen nothing (finite: -inf - m stays -inf)
constexpr float LN2F = 0.693147180559945309f, LOG2EF = 1.44269504088896341f;

struct Start {
  long long unit0;     // its first unit
  int tiles, h, rt, row0, count, add;
};
// The shared tokens of a group: `len` of them, in the row `lead` of the page table, seen by all
// of the group's rows, new tokens first .. first + count - 1.
struct Group {
  int len, lead, first, count;
};
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
  long long* prefix;   // workspace: units before each sequence [B + 1], the blocks in use
  Start* start;        // workspace: the item in which each block's share begins
  uint8_t* failed;     // workspace: whether a wait of each block ran out; every block writes its own
  float* part;         // workspace: 2 slots for each block
  // Of spec_kv_attention_shared, else null. Its first pass goes over the shared tokens of
  // each group for all of the group's rows: `groups` says which, the results are kept in
  // fp32. The second pass goes over the rest of each sequence and adds those.
  const Group* groups;   // first pass
  const int32_t* skip;   // second pass: tokens of each sequence that the first has gone over
  float *kept, *kept_lse;   // [N][q_heads][head_dim], [N][q_heads]: written by the first pass, read by the second
  int workers;
  int group;           // query heads of a kv head
  int group_mul;       // 2^16 / group, rounded up
};
// x / group for 0 <= x < 2^8: group_mul is too large by less than 1, and x group < 2^16
__device__ __forceinline__ int over_group(const AttnArgs& A, int x) { return x * A.group_mul >> 16; }

constexpr long long FAR = 1ll << 30;   // past every position of a cache
constexpr int FIRST = 1, LAST = 2, WHOLE = 4, MASKED = 8, END = 16, ADD = 32;   // ADD: to what the first pass kept
constexpr int MAX_RUNS = 8;    // runs of 16 tokens in a unit
struct Meta {                  // of a stage: a unit of item (b, h, rt)
  float4 run[MAX_RUNS];               // of each 16 tokens: key scale, log2 and reciprocal of the value scale
  int flags;                   // FIRST, LAST of the block's share of the item; WHOLE: that is all of it;
                               // MASKED: some row does not see all tokens; END: no unit
  int row0, count;             // as in Seq: first, count
  int i0, r0;                  // the item's first query row is number r0 of new token i0
  int hi0, lo0;                // new token i sees the unit's tokens up to hi0 + i and after lo0 + i
  int h, slot, live, pad;      // slot of the workspace, if the share is not whole; tokens that are there
  int pad2;
};
static_assert(sizeof(Meta) % 16 == 0, "stages stay 16-byte aligned");

// A copy or product that takes longer is given up. The limit of the last wait, for what is
// still in flight before a block ends, is never shorter.
constexpr uint64_t LAND_NS = 200ull * 1000 * 1000;
#ifndef SPEC_KV_WAIT_NS   // a test makes it 0, for all blocks or for one
#define SPEC_KV_WAIT_NS LAND_NS
#endif

template <int D, int TOK>
struct Stage {
  uint8_t k[TOK * D], v[TOK * D];
};
// Layout of a block. Up to 24 query rows keep the queries' fragments in registers; more
// read them from shared memory, which units of 128 tokens do half as often (32 rows of
// 4 sequences of 131,000 tokens: 160 us against 173 with 64, before EARLY; 48 and 64 rows
// have no registers for it: prompt chunks in this kernel 699 us against 650). Narrow heads take 128 tokens too, so
// that a unit is worth its barriers. Blocks on an SM: as many as registers allow (64
// sequences of up to 16,000 tokens, 20 rows: 197 us with three, 215 with two; 256 single
// tokens, 6 rows: 60 us with four, 69 with three).
template <int D, int NT>
struct Shape {
  static constexpr int MT = D == 64 || NT == 4 ? 2 : 1;  // runs of 16 tokens of a warp
  static constexpr int TOK = 16 * MT * NWARP;            // cached tokens of a unit
  static constexpr int BLOCKS = NT <= 2 ? 4 : NT <= 3 ? 3 : 2;
  static constexpr bool QREG = NT <= 3;                  // query fragments in registers
  // Weights before it is known that the frames hold: one barrier less a unit, where a unit
  // is 128 tokens and registers are left (32 rows of 4 sequences of 131,000 tokens 153 us
  // against 163, 6 rows of 256 sequences 58.9 against 59.8; with units of 64 tokens 20 rows
  // 199 against 198 and 4 rows 162 against 160; 64 rows 175 against 147).
  static constexpr bool EARLY = MT == 2 && NT <= 4;
  static constexpr int PSTRIDE = 16 * (NT | 1);          // bytes of a token's weights: odd multiples of 16 spread the banks
  // the queries' and the weights' buffers are one where the queries move on to registers
  static constexpr int QBYTES = 8 * NT * D * 2, PBYTES = TOK * PSTRIDE, PAT = QREG ? 0 : QBYTES;
  static constexpr int BUF = QREG ? (QBYTES > PBYTES ? QBYTES : PBYTES) : QBYTES + PBYTES;
  static constexpr int FIXED = 1024 /* stages lie on 1024-byte boundaries */ + BUF + 8 * NT * 4 * (1 + NWARP);
  static constexpr int ROOM = (227 * 1024) / BLOCKS - 1024 - 256 - FIXED;
  static constexpr int FIT = ROOM / (int)(sizeof(Stage<D, TOK>) + sizeof(Meta) + 8);
  static constexpr int NS = FIT > 6 ? 6 : FIT;           // stages
  static constexpr size_t SMEM = (sizeof(Stage<D, TOK>) + sizeof(Meta) + 8) * NS + FIXED;
  static_assert(NS >= 2, "one unit on its way while one is worked on");
};

// Units of sequence b: kv_heads * row tiles * (OVERHEAD + token tiles), at least one
// tile, so that every row is written. The OVERHEAD units of an item come first and
// hold no tokens: they only even out the shares.
struct Span {
  int tile0, tiles, rts;
};
// Sequence b, or group b in the first pass over shared tokens.
__device__ __forceinline__ Seq rows_of(const AttnArgs& A, int b) {
  if (!A.groups) return sequence(A.w, b);
  const Group g = A.groups[b];
  return Seq{g.len, g.first, g.count, g.count};
}
template <int ROWS, int TOK>
__device__ __forceinline__ Span span_of(const AttnArgs& A, int b, const Seq& s) {
  Span p{0, 0, 0};
  if (s.count == 0) return p;
  const long long cap = (long long)A.w.max_pages * A.w.page_size;
  const long long end = s.len < 0 ? 0 : min(s.len + (A.groups ? 0 : s.count), cap);
  long long lo = A.window && s.len >= 0 ? max(s.len - A.window + 1, 0ll) : 0ll;
  if (A.skip) lo = max(A.skip[b], 0);
  lo = min(lo, end);
  p.tile0 = (int)(lo / TOK);
  p.tiles = max((int)((end + TOK - 1) / TOK) - p.tile0, 1);
  p.rts = (s.count * A.group + ROWS - 1) / ROWS;   // below 2^30
  return p;
}
__device__ __forceinline__ int table_row(const AttnArgs& A, int b) { return A.groups ? A.groups[b].lead : b; }
// ADD where the first pass has gone over tokens of sequence b.
__device__ __forceinline__ int added(const AttnArgs& A, int b, const Seq& s) {
  return A.skip && s.len >= 0 && A.skip[b] > 0 ? ADD : 0;
}
template <int ROWS, int TOK>
__device__ __forceinline__ long long units_of(const AttnArgs& A, int b) {
  const Span p = span_of<ROWS, TOK>(A, b, rows_of(A, b));
  return (long long)A.w.kv_heads * p.rts * (p.tiles + OVERHEAD);
}

// Quotient of non-negative numbers; the 64-bit division is slow and rarely needed.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ long long share_start(long long w, long long units, long long workers) {
  return quotient(w * units, workers);
}

// The block's share [u0, u1) of all units, and the sequence in which it begins with the
// units before that (in shared memory); whether it has one. Block 0 leaves the
// sequences' units for the join.
template <int ROWS, int TOK, int THREADS>
__device__ __forceinline__ bool find_share(const AttnArgs& A, long long* s_sum, int* s_b, long long* s_pre, long long& u0,
                                           long long& u1) {
  constexpr int WARPS = THREADS / 32;
  const Window& w = A.w;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long long mine = 0;
  for (int b = tid; b < w.B; b += THREADS) mine += units_of<ROWS, TOK>(A, b);
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s_sum[warp] = mine;
  if (tid == 0) *s_b = -1;
  __syncthreads();
  long long units = 0;
#pragma unroll 1
  for (int i = 0; i < WARPS; ++i) units += s_sum[i];
  const long long workers = min((long long)A.workers, max(units / MIN_SHARE, 1ll));
  const long long wk = blockIdx.x;
  u0 = share_start(wk, units, workers);
  u1 = wk < workers ? share_start(wk + 1, units, workers) : u0;
  long long before = 0;
  for (int b0 = 0; b0 < w.B; b0 += THREADS) {
    const int b = b0 + tid;
    const long long u = b < w.B ? units_of<ROWS, TOK>(A, b) : 0;
    long long inc = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();   // the last values have been read
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    long long pre = before;
#pragma unroll 1
    for (int i = 0; i < warp; ++i) pre += s_sum[i];
#pragma unroll 1
    for (int i = 0; i < WARPS; ++i) before += s_sum[i];
    pre += inc - u;
    if (u > 0 && u0 >= pre && u0 < pre + u) {
      *s_b = b;
      *s_pre = pre;
    }
    if (blockIdx.x == 0 && b < w.B) A.prefix[b] = pre;
  }
  if (blockIdx.x == 0 && tid == 0) {
    A.prefix[w.B] = units;
    A.prefix[w.B + 1] = workers;
  }
  __syncthreads();
  return u0 < u1 && *s_b >= 0;
}

// Whether the block gave up, in its byte; the last block fills up the 16 bytes its own lies in.
__device__ __forceinline__ void set_failed(const AttnArgs& A, int tid, int x) {
  const int b = blockIdx.x, at = b + tid;
  if (tid == 0 || (b + 1 == A.workers && (at ^ b) < 16)) A.failed[at] = tid == 0 ? x : 0;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool arrived(uint32_t b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(b), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the copies of a stage, for at most `limit` ns (0: gives up at once).
__device__ __forceinline__ bool wait_copies(uint32_t b, uint32_t parity, uint64_t limit) {
  if (limit == 0) return false;
  if (arrived(b, parity)) return true;
  const uint64_t t0 = now_ns();
  while (!arrived(b, parity))
    if (now_ns() - t0 > limit) return false;
  return true;
}
// A box of rows of codes from row y; the first coordinate is 0, the second has no alignment rule.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int y, uint32_t b) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(b)
      : "memory");
}

__device__ __forceinline__ float ex2f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The second pass, which may begin before the first has ended, ends after it.
__device__ __forceinline__ void after_first_pass(const AttnArgs& A) {
  if (A.skip) asm volatile("griddepcontrol.wait;" ::: "memory");
}
// A row's sum l in the frame m and what the first pass kept for it, in one frame: factors of
// the row's weighted values and of the kept ones, and their common sum in l, m.
__device__ __forceinline__ void add_kept(float& m, float& l, float kept_lse, float& own, float& kept) {
  const float k = kept_lse * LOG2EF, top = fmaxf(m, fmaxf(k, NO_FRAME));   // k: -inf where nothing was seen
  own = ex2f(m - top);
  kept = ex2f(k - top);
  l = fmaf(l, own, kept);
  m = top;
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
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t* r, uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm2_trans(uint32_t* r, uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool bar_any(int id, int threads, bool x) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((int)x)
      : "memory");
  return r != 0;
}

// Byte offset of 16-byte chunk c of token t in a stage's tile: TMA's 128-byte (64-byte)
// swizzle, under which the fragments' loads touch every bank once.
template <int D>
__device__ __forceinline__ int chunk_at(int t, int c) {
  return D == 128 ? t * 128 + ((c ^ (t & 7)) << 4) : t * 64 + ((c ^ ((t >> 1) & 3)) << 4);
}

// The weights of run t as the value product wants them.
template <int NT>
__device__ __forceinline__ void load_weights(uint32_t (&pf)[NT][2], const unsigned char* sp, int t, int lane) {
  constexpr int PS = 16 * (NT | 1);
#pragma unroll
  for (int n = 0; n + 1 < NT; n += 2)
    ldsm4_trans(&pf[n][0], smem_u32(sp + (16 * t + (lane & 15)) * PS + (n + (lane >> 4)) * 16));
  if (NT & 1) ldsm2_trans(&pf[NT - 1][0], smem_u32(sp + (16 * t + (lane & 15)) * PS + (NT - 1) * 16));
}

// The value product of 16 tokens one token at a time, each added only to the rows
// that see it (rare: only where a masked unit holds NaN values). Works on copies, so
// that the caller's accumulators stay in registers.
template <int DT, int NT>
struct ByToken {
  float o[DT][NT][4];
  uint32_t v[4], pf[NT][2];
  uint32_t seen[NT][2];   // bit k: the thread's row (n, e) sees token k
};
template <int DT, int NT>
__device__ __noinline__ void add_by_token(ByToken<DT, NT>& x, int q) {
#pragma unroll 1
  for (int k = 0; k < 16; ++k) {
    const bool mine = q == (k & 7) >> 1;
    const int slot = (k & 1) + 2 * (k >> 3);
#pragma unroll
    for (int j = 0; j < DT; ++j) {
      const uint32_t pick = j ? 0x7362u : 0x5140u;
      uint32_t a0, a1, a2, a3, y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = mine && i == slot ? x.v[i] : 0u;
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
__global__ void __launch_bounds__(NTHR + 32, (Shape<D, NT>::BLOCKS))
    kv_attention_kernel(const AttnArgs A, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v) {
  using Sh = Shape<D, NT>;
  constexpr int NS = Sh::NS, MT = Sh::MT, TOK = Sh::TOK;
  constexpr int KW = D / 16;       // words (4 codes) of a token in a lane = steps of the key product
  constexpr int DT = D / 64;       // 16-row tiles of head_dim in a warp's value product
  constexpr int ROWS = 8 * NT, PS = Sh::PSTRIDE;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  using Unit = Stage<D, TOK>;
  Unit* ring = reinterpret_cast<Unit*>(smem);
  Meta* meta = reinterpret_cast<Meta*>(smem + sizeof(Unit) * NS);
  unsigned char* sq = smem + (sizeof(Unit) + sizeof(Meta)) * NS;    // queries, fp16, in fragment order
  unsigned char* sp = sq + Sh::PAT;                                     // weights, fp16 [token][row]
  float* srs = reinterpret_cast<float*>(sq + Sh::BUF);                  // logit factor of each row
  float* swm = srs + ROWS;                                              // [warp][row]: maxima, later sums
  unsigned long long* full = reinterpret_cast<unsigned long long*>(swm + NWARP * ROWS);   // a stage's copies have landed
  __shared__ long long s_sum[NWARP + 1], s_pre;
  __shared__ int s_b;
  const Window& w = A.w;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(full + i)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (A.groups) asm volatile("griddepcontrol.wait;" ::: "memory");   // kv_groups_kernel's
  set_failed(A, tid, 0);
  const int G = A.group;
  constexpr int ALL = NTHR + 32;
  const long long wk = blockIdx.x;
  long long u0, u1;
  const bool some = find_share<ROWS, TOK, ALL>(A, s_sum, &s_b, &s_pre, u0, u1);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!some) {
    after_first_pass(A);
    return;
  }

  if (warp == NWARP) {
    // --- the copying warp. Unit `cu` is number `ct` of item (cb, ch, cr)
    int cb = s_b;
    long long cu = u0;
    Seq cs = rows_of(A, cb);
    Span cp = span_of<ROWS, TOK>(A, cb, cs);
    int add = added(A, cb, cs);
    int ct, ch, cr;
    {
      const long long x = u0 - s_pre;
      const int per = cp.tiles + OVERHEAD;
      const long long item = quotient(x, per);
      ct = (int)(x - item * per);
      ch = (int)quotient(item, cp.rts);
      cr = (int)(item - (long long)ch * cp.rts);
      if (lane == 0) A.start[wk] = Start{u0 - ct, cp.tiles, ch, cr, cs.first, cs.count, add};
    }
    // entries window0 .. window0 + 31 of the sequence's row of the page table and those
    // pages' scales, one in each lane
    int entry = -1, window_b = -1, window_h = -1, window0 = 0;
    float eks = 0.f, elv = 0.f, einv = 0.f;
    const int P = w.page_size, shift = __ffs(P) - 1;
    const int box = min(P, TOK);          // tokens of a copy
    const auto issue = [&](int stage) {
      Unit& S = ring[stage];
      Meta& M = meta[stage];
      if (ct < OVERHEAD) {
        cu += OVERHEAD - ct;
        ct = OVERHEAD;
      }
      const bool on = cu < u1;
      if (!on) {
        if (lane == 0) M.flags = END;
      } else {
        const int tok0 = (cp.tile0 + ct - OVERHEAD) * TOK;     // below 2^27
        const int live = cs.len < 0 ? 0 : (int)min(cs.len + cs.count - tok0, (long long)TOK);
        const int j0 = tok0 >> shift, j1 = (tok0 + TOK - 1) >> shift;
        if (cb != window_b || j0 < window0 || j1 >= window0 + 32) {
          window_b = cb;
          window_h = -1;
          window0 = j0;
          entry = page_of(w, table_row(A, cb), (long long)j0 + lane);
        }
        if (ch != window_h) {
          window_h = ch;
          const size_t at = (size_t)max(entry, 0) * w.kv_heads + ch;
          const float vs = entry < 0 ? 1.f : A.v_scale[at];
          eks = entry < 0 ? 1.f : A.k_scale[at];
          elv = log2f(vs);
          einv = __frcp_rn(vs);
        }
        // the first lanes: the runs of 16 tokens. A run that no query sees counts as unmapped:
        // its page may never have been written, and 0 times what its scale holds may be NaN.
        const int run = 16 * lane & (TOK - 1), from = ((tok0 + run) >> shift) - window0;
        const int listed = __shfl_sync(0xffffffffu, entry, from);
        const int page = run < live && (!A.window || tok0 + run + 16 > cs.len - A.window + 1) ? listed : -1;
        const float ks = __shfl_sync(0xffffffffu, eks, from), lv = __shfl_sync(0xffffffffu, elv, from),
                    inv = __shfl_sync(0xffffffffu, einv, from);
        const bool gap = __any_sync(0xffffffffu, page < 0);
        if (lane < TOK / 16) M.run[lane] = page < 0 ? make_float4(1.f, 0.f, 1.f, 1.f) : make_float4(ks, lv, inv, 0.f);
        // the first TOK / box lanes: a copy of the keys and one of the values
        const int at = tok0 + (lane * box & (TOK - 1));
        const int pg = __shfl_sync(0xffffffffu, entry, (at >> shift) - window0);
        const bool mine = lane * box < TOK && pg >= 0 && at - tok0 < live;
        const int copies = __popc(__ballot_sync(0xffffffffu, mine));
        const uint32_t bar_at = smem_u32(full + stage);
        if (lane == 0)
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar_at), "r"(copies * 2 * box * D) : "memory");
        __syncwarp();
        if (mine) {
          const int y = (pg * w.kv_heads + ch) * P + (at & (P - 1)), d = (at - tok0) * D;
          copy_box(smem_u32(S.k) + d, &map_k, y, bar_at);
          copy_box(smem_u32(S.v) + d, &map_v, y, bar_at);
        }
        if (lane == 0) {
          const long long item0 = cu - ct, item1 = item0 + OVERHEAD + cp.tiles;
          const bool masked = gap || cs.len < 0 || tok0 + TOK - 1 > cs.len ||
                              (A.window && tok0 <= cs.len + cs.count - 1 - A.window);
          M.flags = (ct == OVERHEAD || cu == u0 ? FIRST : 0) | (cu + 1 == item1 || cu + 1 == u1 ? LAST : 0) |
                      (u0 <= item0 + OVERHEAD && u1 >= item1 ? WHOLE : 0) | (masked ? MASKED : 0) | add;
          M.row0 = cs.first;
          M.count = cs.count;
          const long long hi = cs.len < 0 ? -FAR : cs.len - tok0;
          M.hi0 = (int)min(hi, FAR);
          M.lo0 = A.window ? (int)max(min(hi - A.window, FAR), -FAR) : (int)-FAR;
          M.h = ch;
          M.i0 = cr * ROWS / G;
          M.r0 = cr * ROWS % G;
          M.slot = u0 < item0 ? 1 : 0;
          M.live = live;
        }
        ++cu;
        if (++ct == cp.tiles + OVERHEAD) {
          ct = 0;
          if (++cr == cp.rts) {
            cr = 0;
            if (++ch == w.kv_heads) {
              ch = 0;
              if (cu < u1) {
                do {
                  cs = rows_of(A, ++cb);
                  cp = span_of<ROWS, TOK>(A, cb, cs);
                  add = added(A, cb, cs);
                } while (cp.rts == 0 && cb + 1 < w.B);
              }
            }
          }
        }
      }
      return on;
    };
    int ahead = 0;               // units copied or on their way, not yet handed over
#pragma unroll 1
    for (int i = 0; i < NS - 1; ++i) ahead += issue(i);
    uint32_t parity = 0;
    for (int stage = 0;;) {
      if (ahead > 0 && !__all_sync(0xffffffffu, wait_copies(smem_u32(full + stage), parity, SPEC_KV_WAIT_NS))) {
        // given up: the others stop, the join makes every output NaN; what was asked for lands
        if (lane == 0) {
          meta[stage].flags = END;
          A.failed[wk] = 1;
        }
        __syncwarp();
        bar(1, ALL);
        for (int i = 0; i < ahead; ++i) {
          wait_copies(smem_u32(full + stage), parity, LAND_NS);
          if (++stage == NS) stage = 0, parity ^= 1;
        }
        after_first_pass(A);
        return;
      }
      bar(1, ALL);               // the unit is there, and the one before it is done with
      if (ahead == 0) {          // that was the END
        after_first_pass(A);
        return;
      }
      ahead += issue(stage == 0 ? NS - 1 : stage - 1) - 1;
      if (++stage == NS) stage = 0, parity ^= 1;
    }
  }

  uint32_t qf[Sh::QREG ? NT : 1][2 * KW];   // query fragments
  float m[NT][2], l[NT][2], o[DT][NT][4];   // of rows 8 n + 2 q + {0, 1}
  for (int stage = 0;; stage = stage + 1 == NS ? 0 : stage + 1) {
    bar(1, ALL);
    const Unit& S = ring[stage];
    const Meta& M = meta[stage];
    const int flags = M.flags;
    if (flags & END) return;
    if (flags & FIRST) {
      // Queries: four threads to a row, each D / 4 elements; scaled by a power of two
      // so that the row's largest element lies in [2^7, 2^8)
#pragma unroll 1
      for (int r = tid >> 2; r < ROWS; r += NTHR / 4) {
        const int i = M.i0 + over_group(A, M.r0 + r), hd = M.h * G + M.r0 + r - (i - M.i0) * G;
        uint32_t x[D / 8];
        if (i < M.count) {
          const uint4* p = reinterpret_cast<const uint4*>(A.q + (size_t)(M.row0 + i) * (size_t)A.q_stride + (size_t)hd * D + q * (D / 4));
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const uint4 v = p[k];
            x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int k = 0; k < D / 8; ++k) x[k] = 0u;
        }
        uint32_t top = 0u;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const uint32_t a = (x[k] << 16) & 0x7FFFFFFFu, b = x[k] & 0x7FFF0000u;
          if (a < 0x7F800000u) top = max(top, a);
          if (b < 0x7F800000u) top = max(top, b);
        }
        const unsigned four = 0xFu << (lane & ~3);
        top = max(top, __shfl_xor_sync(four, top, 1));
        top = max(top, __shfl_xor_sync(four, top, 2));
        const int e = top ? min(max((int)(top >> 23) - 127 - 7, -100), 119) : 0;   // 2^e times [2^7, 2^8)
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
        // word k of lane q (elements q D / 4 + 2 k, + 1) goes to pair q of 16-byte segment k
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
          *reinterpret_cast<uint32_t*>(sq + r * (D * 2) + ((k ^ (r & 7)) << 4) + q * 4) =
              pack_h2(__uint_as_float(x[k] << 16) * down, __uint_as_float(x[k] & 0xFFFF0000u) * down);
        if (q == 0) srs[r] = up * A.scale;
      }
      bar(2, NTHR);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (Sh::QREG) {
#pragma unroll
          for (int k = 0; k < KW / 2; ++k)
            ldsm4(&qf[n][4 * k], smem_u32(sq + (8 * n + (lane & 7)) * (D * 2) + (((4 * k + (lane >> 3)) ^ (lane & 7)) << 4)));
        }
        m[n][0] = m[n][1] = NO_FRAME;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[j][n][k] = 0.f;
      }
      if (Sh::QREG && Sh::EARLY) bar(2, NTHR);   // the weights go where the queries were
    }

    // --- logits of the warp's runs of 16 tokens: sc[t][n] holds tokens g and g + 8, rows 8 n + 2 q (+ 1)
    float sc[MT][NT][4];
    {
      uint32_t ka[MT][KW], kb[MT][KW];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int ta = 16 * (MT * warp + t) + g;
#pragma unroll
        for (int i = 0; i < KW / 4; ++i) {
          const uint4 a = *reinterpret_cast<const uint4*>(S.k + chunk_at<D>(ta, (KW / 4) * q + i));
          const uint4 b = *reinterpret_cast<const uint4*>(S.k + chunk_at<D>(ta + 8, (KW / 4) * q + i));
          ka[t][4 * i] = a.x, ka[t][4 * i + 1] = a.y, ka[t][4 * i + 2] = a.z, ka[t][4 * i + 3] = a.w;
          kb[t][4 * i] = b.x, kb[t][4 * i + 1] = b.y, kb[t][4 * i + 2] = b.z, kb[t][4 * i + 3] = b.w;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[t][n][k] = 0.f;
      }
#pragma unroll
      for (int k2 = 0; k2 < KW / 2; ++k2) {
        uint32_t a[MT][2][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            widen(ka[t][2 * k2 + k], a[t][k][0], a[t][k][2]);
            widen(kb[t][2 * k2 + k], a[t][k][1], a[t][k][3]);
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t f[4];
          if (Sh::QREG) {
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = qf[Sh::QREG ? n : 0][4 * k2 + k];
          } else {
            ldsm4(f, smem_u32(sq + (8 * n + (lane & 7)) * (D * 2) + (((4 * k2 + (lane >> 3)) ^ (lane & 7)) << 4)));
          }
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            mma16816(sc[t][n], a[t][0][0], a[t][0][1], a[t][0][2], a[t][0][3], f[0], f[1]);
            mma16816(sc[t][n], a[t][1][0], a[t][1][1], a[t][1][2], a[t][1][3], f[2], f[3]);
          }
        }
      }
    }

    // --- weights. A token's exponent is its logit (base 2) plus log2 of its value scale
    // whether the thread's row e of tile n sees token p of the unit
    const auto sees = [&](int n, int e, int p) {
      const int i = M.i0 + over_group(A, M.r0 + 8 * n + 2 * q + e);
      return p <= M.hi0 + i && p > M.lo0 + i;
    };
    float inv[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float4 run = M.run[MT * warp + t];
      inv[t] = run.z;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 rs = *reinterpret_cast<const float2*>(srs + 8 * n + 2 * q);
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[t][n][k] = fmaf(sc[t][n][k], (k & 1 ? rs.y : rs.x) * run.x, run.y);
      }
    }
    if (flags & MASKED) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = M.i0 + over_group(A, M.r0 + 8 * n + 2 * q + e), hi = M.hi0 + i, lo = M.lo0 + i;
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int p = 16 * (MT * warp + t) + g + 8 * k;
              if (p > hi || p <= lo || M.run[MT * warp + t].w != 0.f) sc[t][n][2 * k + e] = -INFINITY;   // w: unmapped
            }
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(sc[0][n][e], sc[0][n][2 + e]);
#pragma unroll
        for (int t = 1; t < MT; ++t) x = fmaxf(x, fmaxf(sc[t][n][e], sc[t][n][2 + e]));
        top = fmaxf(top, x - m[n][e]);
      }
    float early[NT][2];          // this unit's sums, until the frames are known to hold
    float (&part)[NT][2] = Sh::EARLY ? early : l;
    const auto weigh = [&]() {
      if (Sh::EARLY)
#pragma unroll
        for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = 0.f;
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float p0 = ex2f(sc[t][n][2 * k] - m[n][0]), p1 = ex2f(sc[t][n][2 * k + 1] - m[n][1]);
            part[n][0] = fmaf(p0, inv[t], part[n][0]);
            part[n][1] = fmaf(p1, inv[t], part[n][1]);
            *reinterpret_cast<uint32_t*>(sp + (16 * (MT * warp + t) + g + 8 * k) * PS + n * 16 + q * 4) = pack_h2(p0, p1);
          }
    };
    if (Sh::EARLY) weigh();      // nearly always in the right frames
    if (bar_any(2, NTHR, top > TOP)) {
      // some weight would leave its range: move every row's frame to its maximum
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(sc[0][n][e], sc[0][n][2 + e]);
#pragma unroll
          for (int t = 1; t < MT; ++t) x = fmaxf(x, fmaxf(sc[t][n][e], sc[t][n][2 + e]));
#pragma unroll
          for (int y = 4; y < 32; y <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
          if (g == 0) swm[warp * ROWS + 8 * n + 2 * q + e] = x;
        }
      bar(2, NTHR);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = swm[8 * n + 2 * q + e];
#pragma unroll
          for (int i = 1; i < NWARP; ++i) t = fmaxf(t, swm[i * ROWS + 8 * n + 2 * q + e]);
          t -= LIFT;
          if (t > m[n][e]) {
            const float f = ex2f(m[n][e] - t);   // 0 the first time
            m[n][e] = t;
            l[n][e] *= f;
#pragma unroll
            for (int j = 0; j < DT; ++j) {
              o[j][n][e] *= f;
              o[j][n][2 + e] *= f;
            }
          }
        }
      if (Sh::EARLY) {
        weigh();
        bar(2, NTHR);
      }
    }
    // the warp's value words: word i of run t is of token 16 t + 2 q + {0, 1, 8, 9}
    uint32_t v[TOK / 16][4];
#pragma unroll
    for (int t = 0; t < TOK / 16; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tk = 16 * t + 2 * q + (i & 1) + 8 * (i >> 1);
        if (D == 128)
          v[t][i] = *reinterpret_cast<const uint32_t*>(S.v + chunk_at<D>(tk, 2 * warp + (g >> 2)) + 4 * (g & 3));
        else
          v[t][i] = *reinterpret_cast<const uint16_t*>(S.v + chunk_at<D>(tk, warp) + 2 * g);
      }
    if (!Sh::EARLY) weigh();
    bool by_token = false;
    if (flags & MASKED) {
      // what is not there reads as zero
#pragma unroll
      for (int t = 0; t < TOK / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (16 * t + 2 * q + (i & 1) + 8 * (i >> 1) >= M.live || M.run[t].w != 0.f) v[t][i] = 0u;
      // NaN values of tokens that only some rows see: 0 * NaN must not reach the others
      bool nan = false;
#pragma unroll
      for (int t = 0; t < TOK / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) nan |= (((v[t][i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u;
      by_token = __any_sync(0xffffffffu, nan);
    }
    if (!Sh::EARLY) bar(2, NTHR);
    if (Sh::EARLY)
#pragma unroll
      for (int n = 0; n < NT; ++n) l[n][0] += part[n][0], l[n][1] += part[n][1];

    // --- values: o[j][n] holds head_dim (D / 4) warp + (D / 32) g + 2 j + {0: k < 2, 1: k >= 2}
    if (__builtin_expect(!by_token, 1)) {
#pragma unroll
      for (int t = 0; t < TOK / 16; ++t) {
        uint32_t pf[NT][2];
        load_weights<NT>(pf, sp, t, lane);
#pragma unroll
        for (int j = 0; j < DT; ++j) {
          const uint32_t pick = j ? 0x7362u : 0x5140u;   // bytes 2, 3 or 0, 1 of two neighbouring tokens, interleaved
          uint32_t a0, a1, a2, a3;
          widen(__byte_perm(v[t][0], v[t][1], pick), a0, a1);
          widen(__byte_perm(v[t][2], v[t][3], pick), a2, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(o[j][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
        }
      }
    } else {
      ByToken<DT, NT> x;
#pragma unroll
      for (int j = 0; j < DT; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) x.o[j][n][k] = o[j][n][k];
#pragma unroll
      for (int t = 0; t < TOK / 16; ++t) {
        load_weights<NT>(x.pf, sp, t, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) x.v[i] = v[t][i];
        for (int n = 0; n < NT; ++n)
          for (int e = 0; e < 2; ++e) {
            x.seen[n][e] = 0u;
#pragma unroll 1
            for (int k = 0; k < 16; ++k) x.seen[n][e] |= (uint32_t)sees(n, e, 16 * t + k) << k;
          }
        add_by_token<DT, NT>(x, q);
      }
#pragma unroll
      for (int j = 0; j < DT; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[j][n][k] = x.o[j][n][k];
    }

    if (flags & LAST) {
      // the warps' sums of the weights (fixed order), then the rows
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
          if (g == 0) swm[warp * ROWS + 8 * n + 2 * q + e] = l[n][e];
        }
      bar(2, NTHR);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * q + e, i = M.i0 + over_group(A, M.r0 + r);
          float sum = swm[r];
#pragma unroll
          for (int k = 1; k < NWARP; ++k) sum += swm[k * ROWS + r];
          if (i >= M.count) continue;
          const int d0 = (D / 4) * warp + (D / 32) * g;
          if (flags & WHOLE) {
            const size_t at = (size_t)(M.row0 + i) * w.q_heads + M.h * G + M.r0 + r - (i - M.i0) * G;
            if (flags & ADD) {
              after_first_pass(A);
              float own, kept;
              add_kept(m[n][e], sum, A.kept_lse[at], own, kept);
#pragma unroll
              for (int j = 0; j < DT; ++j) {
                const float2 y = *reinterpret_cast<const float2*>(A.kept + at * D + d0 + 2 * j);
                o[j][n][e] = fmaf(o[j][n][e], own, y.x * kept);
                o[j][n][2 + e] = fmaf(o[j][n][2 + e], own, y.y * kept);
              }
            }
            const float f = sum == 0.f ? 0.f : 1.f / sum;
            if (A.groups) {
#pragma unroll
              for (int j = 0; j < DT; ++j)
                *reinterpret_cast<float2*>(A.kept + at * D + d0 + 2 * j) = make_float2(o[j][n][e] * f, o[j][n][2 + e] * f);
              if (warp == 0 && g == 0) A.kept_lse[at] = LN2F * (m[n][e] + log2f(sum));
              continue;
            }
            uint32_t y[DT];
#pragma unroll
            for (int j = 0; j < DT; ++j) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(o[j][n][e] * f, o[j][n][2 + e] * f);
              y[j] = *reinterpret_cast<const uint32_t*>(&b2);
            }
#pragma unroll
            for (int j = 0; j < DT; ++j) *reinterpret_cast<uint32_t*>(A.out + at * D + d0 + 2 * j) = y[j];
            if (A.lse && warp == 0 && g == 0) A.lse[at] = LN2F * (m[n][e] + log2f(sum));
          } else {
            float* slot = A.part + ((size_t)wk * 2 + M.slot) * ROWS * (D + 2);
            if (warp == 0 && g == 0) {
              slot[2 * r] = m[n][e];
              slot[2 * r + 1] = sum;
            }
#pragma unroll
            for (int j = 0; j < DT; ++j)
              *reinterpret_cast<float2*>(slot + 2 * ROWS + r * D + d0 + 2 * j) = make_float2(o[j][n][e], o[j][n][2 + e]);
          }
        }
    }
  }
}

}  // namespace svkv
#include "kv_wide.cuh"
namespace svkv {

// Joins the shares of the items that several blocks worked on. At most one item is cut
// at the start of each share: block (k, n) looks whether share k is the second of its
// item, and if so takes rows 8 n .. 8 n + 7 of it. Eight warps share the rows that are
// there; a warp gathers the frames and sums of its part of the shares, a lane each,
// and adds their weighted values, D / 32 elements a lane. Then the warps of a row are
// joined, in their order.
constexpr int JOIN = 8;   // warps

// Whether some block gave up, in every lane of a warp.
__device__ __forceinline__ bool any_failed(const AttnArgs& A, int lane) {
  uint32_t x = 0u;
  for (int at = 16 * lane; at < A.workers; at += 16 * 32) {
    const uint4 v = *reinterpret_cast<const uint4*>(A.failed + at);
    x |= v.x | v.y | v.z | v.w;
  }
  return __any_sync(0xffffffffu, x != 0u);
}

template <int D, int NT>
__global__ void __launch_bounds__(JOIN * 32) kv_combine_kernel(const AttnArgs A) {
  constexpr int ROWS = 8 * NT, E = D / 32;
  // first of all, in every thread: this grid ends only after the one before it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Window& w = A.w;
  __shared__ bool failed;
  __shared__ float sm[JOIN], sl[JOIN], so[JOIN][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = A.group;
  const long long k = blockIdx.x, units = A.prefix[w.B], workers = A.prefix[w.B + 1];
  if (k == 0) {   // no item is cut at the first share's start: these blocks see to copies that never came
    if (!any_failed(A, lane)) return;
    const long long n = (long long)w.N * w.q_heads;
    for (long long x = (long long)blockIdx.y * (JOIN * 32) + threadIdx.x; x < n * D; x += (long long)gridDim.y * (JOIN * 32)) {
      if (A.groups) {
        A.kept[x] = NAN;
        if (x < n) A.kept_lse[x] = NAN;
        continue;
      }
      A.out[x] = __float2bfloat16_rn(NAN);
      if (A.lse && x < n) A.lse[x] = NAN;
    }
    return;
  }
  if (k >= workers) return;
  const Start item = A.start[k];
  const long long i0 = item.unit0;
  // the shares that hold its first and its last unit with tokens
  const long long w0 = quotient((i0 + OVERHEAD + 1) * workers - 1, units);
  if (w0 != k - 1) return;
  const long long w1 = quotient((i0 + OVERHEAD + item.tiles) * workers - 1, units);
  const int first_row = item.rt * ROWS + 8 * blockIdx.y;
  const int rows = min(item.count * G - first_row, 8);
  if (rows <= 0) return;
  const int team = rows > 4 ? 1 : rows > 2 ? 2 : rows > 1 ? 4 : 8;   // warps of a row
  const int mine = warp / team, r = 8 * blockIdx.y + mine;
  float m = NO_FRAME, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  const int per = (int)((w1 - w0 + team) / team);   // shares of a warp
  const long long from = w0 + (long long)(warp % team) * per, last = mine < rows ? min(w1, from + per - 1) : from - 1;
  // share w0 is the second of its block unless it begins with the item
  const int second = share_start(w0, units, workers) < i0;
  for (long long k0 = from; k0 <= last; k0 += 32) {
    const int n = (int)min(last - k0 + 1, 32ll);
    float mk = NO_FRAME, lk = 0.f;
    const float* part = A.part + ((size_t)(k0 + lane) * 2 + (k0 + lane == w0 ? second : 0)) * (ROWS * (D + 2));
    if (lane < n) mk = part[2 * r], lk = part[2 * r + 1];
    float top = fmaxf(m, mk);
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float f = ex2f(m - top), fk = ex2f(mk - top);
    float sum = lk * fk;
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = fmaf(l, f, sum);
    m = top;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
    // eight at a time; those past the end are the last one again, with weight 0
#pragma unroll 1
    for (int x0 = 0; x0 < n; x0 += 8)
#pragma unroll
    for (int x1 = 0; x1 < 8; ++x1) {
      const int x = min(x0 + x1, n - 1);
      const float* src = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(part), x));
      const float fx = __shfl_sync(0xffffffffu, fk, x), fs = x0 + x1 < n ? fx : 0.f;
      src += 2 * ROWS + r * D + lane * E;
      if (E == 4) {
        const float4 y = *reinterpret_cast<const float4*>(src);
        o[0] = fmaf(y.x, fs, o[0]), o[1 % E] = fmaf(y.y, fs, o[1 % E]);
        o[2 % E] = fmaf(y.z, fs, o[2 % E]), o[3 % E] = fmaf(y.w, fs, o[3 % E]);
      } else {
        const float2 y = *reinterpret_cast<const float2*>(src);
        o[0] = fmaf(y.x, fs, o[0]), o[1] = fmaf(y.y, fs, o[1]);
      }
    }
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  if (warp == JOIN - 1) {   // one warp looks, here: earlier, or in all warps, it costs 0.7 to 4 us a call
    const bool x = any_failed(A, lane);
    if (lane == 0) failed = x;
  }
  __syncthreads();
  if (failed) return;
  if (warp % team || mine >= rows) return;
  m = sm[warp];
  for (int x = 1; x < team; ++x) m = fmaxf(m, sm[warp + x]);
  l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int x = 0; x < team; ++x) {
    const float f = ex2f(sm[warp + x] - m);
    l = fmaf(sl[warp + x], f, l);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(so[warp + x][lane * E + e], f, o[e]);
  }
  const int row = first_row + mine, i = row / G;
  const size_t at = (size_t)(item.row0 + i) * w.q_heads + item.h * G + row % G;
  if (item.add) {
    float own, kept;
    add_kept(m, l, A.kept_lse[at], own, kept);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], own, A.kept[at * D + lane * E + e] * kept);
  }
  const float f = l == 0.f ? 0.f : 1.f / l;
  if (A.groups) {
#pragma unroll
    for (int e = 0; e < E; ++e) A.kept[at * D + lane * E + e] = o[e] * f;
    if (lane == 0) A.kept_lse[at] = LN2F * (m + log2f(l));
    return;
  }
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(A.out + at * D + lane * E + e) = __floats2bfloat162_rn(o[e] * f, o[e + 1] * f);
  if (A.lse && lane == 0) A.lse[at] = LN2F * (m + log2f(l));
}

static sv::LaunchCache g_attn_cache;

// Rows of a window from which the wide kernel takes over (head_dim 128): where these would
// be more than one item and read the cache again. 3 sequences of up to 12,000 tokens, 32
// heads on 8, this kernel and the wide one: 64 rows 48 and 51 us, 96 rows 71 and 52, 128
// rows 74 and 54; 48 of up to 2,000: 64 rows 81 and 97, 96 rows 128 and 98.
constexpr int WIDE_ROWS = 8 * MAX_NT + 1;

// Tiles of 8 rows of an item: just enough for the window, at most MAX_NT, or those of
// the wide kernel.
static int row_tiles(int max_tokens, int group, int head_dim) {
  const long long nt = ((long long)max_tokens * group + 7) / 8;
  if (head_dim == wide::D && nt * 8 >= WIDE_ROWS) return wide::NT;
  return nt <= 4 ? (int)nt : nt <= 6 ? 6 : MAX_NT;
}
static int blocks_per_sm(int nt) { return nt <= 2 ? 4 : nt <= 3 ? 3 : nt <= MAX_NT ? 2 : 1; }   // Shape::BLOCKS

static int sm_count() try {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (g_attn_cache.get(dev, reinterpret_cast<const void*>(&sm_count), 0, 0, &n, [&](int* v) {
        return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
      }) != cudaSuccess)
    return 0;
  return n;
} catch (...) {   // no exception passes the C entry points
  return 0;
}

static size_t prefix_bytes(int B) { return ((size_t)(B + 2) * sizeof(long long) + 127) & ~(size_t)127; }
static size_t start_bytes(int workers) { return (size_t)workers * sizeof(Start); }
static size_t failed_bytes(int workers) { return ((size_t)workers + 127) & ~(size_t)127; }
static size_t part_bytes(int workers, int nt, int D) { return (size_t)workers * 2 * 8 * nt * (D + 2) * sizeof(float); }
static size_t workspace_size(int B, int workers, int nt, int D) {
  return prefix_bytes(B) + start_bytes(workers) + failed_bytes(workers) + part_bytes(workers, nt, D);
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (EncodeTiled) nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// The codes as rows of head_dim bytes, one for each (page, kv head, token).
static bool code_map(CUtensorMap* map, const void* codes, const Window& w, int TOK) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)w.head_dim, (cuuint64_t)w.num_pages * w.kv_heads * w.page_size};
  const cuuint64_t strides[1] = {(cuuint64_t)w.head_dim};
  const cuuint32_t box[2] = {(cuuint32_t)w.head_dim, (cuuint32_t)(w.page_size < TOK ? w.page_size : TOK)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, w.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernel's shared-memory limit, raised once per device.
static bool raise_smem(const void* fn, size_t bytes) try {
  int dev = 0, done = 0;
  return cudaGetDevice(&dev) == cudaSuccess && g_attn_cache.get(dev, fn, bytes, 0, &done, [&](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  }) == cudaSuccess;
} catch (...) {
  return false;
}

// The join: launched while the first kernel still runs, waits for its results on the device.
template <int D, int NT>
static sv_status launch_combine(AttnArgs& A, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)A.workers, (unsigned)NT);
  cfg.blockDim = dim3(JOIN * 32);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_combine_kernel<D, NT>, A) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

// The kernels of the passes over shared tokens begin while the kernel before them ends, and wait on
// the device where they read its results.
template <typename Kernel>
static cudaError_t launch_main(Kernel kernel, const AttnArgs& A, int threads, size_t smem, const CUtensorMap& map_k,
                               const CUtensorMap& map_v, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)A.workers);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = A.groups || A.skip ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, A, map_k, map_v);
}

template <int D, int NT>
static sv_status launch_attention(AttnArgs& A, cudaStream_t st) {
  constexpr size_t SMEM = Shape<D, NT>::SMEM;
  CUtensorMap map_k, map_v;
  if (!raise_smem(reinterpret_cast<const void*>(kv_attention_kernel<D, NT>), SMEM) ||
      !code_map(&map_k, A.k_codes, A.w, Shape<D, NT>::TOK) || !code_map(&map_v, A.v_codes, A.w, Shape<D, NT>::TOK))
    return SV_ERR_CUDA;
  if (launch_main(kv_attention_kernel<D, NT>, A, NTHR + 32, SMEM, map_k, map_v, st) != cudaSuccess) return SV_ERR_CUDA;
  return launch_combine<D, NT>(A, st);
}

static sv_status launch_wide(AttnArgs& A, cudaStream_t st) {
  CUtensorMap map_k, map_v;
  if (!raise_smem(reinterpret_cast<const void*>(wide::kv_wide_kernel), wide::SMEM) ||
      !code_map(&map_k, A.k_codes, A.w, wide::TOK) || !code_map(&map_v, A.v_codes, A.w, wide::TOK))
    return SV_ERR_CUDA;
  if (launch_main(wide::kv_wide_kernel, A, wide::THREADS, wide::SMEM, map_k, map_v, st) != cudaSuccess) return SV_ERR_CUDA;
  return launch_combine<wide::D, wide::NT>(A, st);
}

template <int D>
static sv_status pick_attention(int nt, AttnArgs& A, cudaStream_t st) {
  switch (nt) {
    case 1: return launch_attention<D, 1>(A, st);
    case 2: return launch_attention<D, 2>(A, st);
    case 3: return launch_attention<D, 3>(A, st);
    case 4: return launch_attention<D, 4>(A, st);
    case 6: return launch_attention<D, 6>(A, st);
    default: return launch_attention<D, 8>(A, st);
  }
}

static AttnArgs arguments(const Window& w, const void* q, long long q_stride, const void* k_codes, const float* k_scale,
                          const void* v_codes, const float* v_scale, float scale, int window, void* out, float* lse) {
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
  A.group = w.q_heads / w.kv_heads;
  A.group_mul = ((1 << 16) + A.group - 1) / A.group;
  return A;
}

// Shapes and alignments of an attention call.
static sv_status check_attention(const Window& w, const void* q, long long q_stride, const void* k_codes, const float* k_scale,
                                 const void* v_codes, const float* v_scale, float scale, int window, const void* out,
                                 const float* lse) {
  if (bad_window(w) || q_stride < (long long)w.q_heads * w.head_dim || window < 0 || !isfinite(scale)) return SV_ERR_SHAPE;
  if ((long long)w.B * w.max_tokens * w.kv_heads > 2147483647ll) return SV_ERR_SHAPE;
  if (!aligned(q, 16) || (q_stride * 2) % 16 || !aligned(out, 16) || !aligned(k_codes, 16) || !aligned(v_codes, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(w.seq_len, 4) || !aligned(w.cu_tokens, 4) ||
      !aligned(w.page_table, 4) || !aligned(lse, 4))
    return SV_ERR_ALIGN;
  return SV_OK;
}

// The kernel for nt tiles of rows and its join, in workspace_size(A.w.B, ...) bytes.
static sv_status launch_pass(AttnArgs& A, int nt, int workers, char* workspace, cudaStream_t st) {
  A.prefix = reinterpret_cast<long long*>(workspace);
  A.start = reinterpret_cast<Start*>(workspace + prefix_bytes(A.w.B));
  A.failed = reinterpret_cast<uint8_t*>(workspace) + prefix_bytes(A.w.B) + start_bytes(workers);
  A.part = reinterpret_cast<float*>(A.failed + failed_bytes(workers));
  A.workers = workers;
  if (nt == wide::NT) return launch_wide(A, st);
  return A.w.head_dim == 128 ? pick_attention<128>(nt, A, st) : pick_attention<64>(nt, A, st);
}

// --- shared tokens. 64 windows of 5 tokens, 32 heads on 8 of 128, on 8,000 shared tokens and up to 600 of
// their own: 110 us; of which the first pass 59 us (1,280 rows for a kv head, the wide kernel at 720 TFLOP/s)
// and its join, which the second pass covers, 17; the second 35 (an item's start and end, as in windows of
// few tokens) and its join 9. What the first pass goes over, a warp to a group. Whole units of 128 tokens
// that every sequence with new tokens holds: no row of the group is masked there, and the second
// pass begins at the start of a unit.
constexpr int SHARED_UNIT = 128;
constexpr long long SHARED_BYTES = 320ll << 20;
static_assert(SHARED_UNIT % wide::TOK == 0, "units of the first pass");

__global__ void __launch_bounds__(256) kv_groups_kernel(const Window w, const int32_t* cu_groups, const int32_t* shared_len,
                                                        int groups, Group* out, int32_t* skip) {
  const int g = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (g >= groups) return;
  const int b0 = min(max(cu_groups[g], 0), w.B), b1 = min(max(cu_groups[g + 1], b0), w.B);
  // sequences of no group
  if (g == 0)
    for (int b = lane; b < b0; b += 32) skip[b] = 0;
  if (g == groups - 1)
    for (int b = b1 + lane; b < w.B; b += 32) skip[b] = 0;
  long long len = min((long long)shared_len[g], (long long)w.max_pages * w.page_size);
  int lead = w.B;
  for (int b = b0 + lane; b < b1; b += 32) {
    const Seq s = sequence(w, b);
    if (s.count > 0 && s.len >= 0) {
      len = min(len, s.len);
      lead = min(lead, b);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    len = min(len, __shfl_xor_sync(0xffffffffu, len, o));
    lead = min(lead, __shfl_xor_sync(0xffffffffu, lead, o));
  }
  const int n = lead == w.B || len < 0 ? 0 : (int)len / SHARED_UNIT * SHARED_UNIT;
  for (int b = b0 + lane; b < b1; b += 32) skip[b] = n;
  if (lane == 0) {
    const int first = min(max(w.cu_tokens[b0], 0), w.N), end = min(w.cu_tokens[b1], w.N);
    out[g] = n ? Group{n, lead, first, max(end - first, 0)} : Group{0, 0, 0, 0};
  }
}

// Tiles of 8 rows of an item of the first pass: the wide kernel's as in row_tiles, else those with the
// fewest rows to spare.
static int shared_tiles(long long rows, int D) {
  const long long nt = (rows + 7) / 8;
  if (D == wide::D && nt * 8 >= WIDE_ROWS) return wide::NT;
  if (nt <= 4) return (int)nt;
  const auto spent = [&](int t) { return (nt + t - 1) / t * t; };
  return spent(6) <= spent(MAX_NT) ? 6 : MAX_NT;
}

// How spec_kv_attention_shared lies in its workspace.
struct SharedPlan {
  int nt1, nt2, workers1, workers2;
  size_t groups, skip, kept, lse, pass1, pass2, total;   // offsets
};
static SharedPlan shared_plan(int B, int groups, int N, int max_tokens, int group, int heads, int D, int sms) {
  SharedPlan p;
  p.nt1 = shared_tiles((long long)((N + groups - 1) / groups) * group, D);
  p.nt2 = row_tiles(max_tokens, group, D);
  p.workers1 = sms * blocks_per_sm(p.nt1), p.workers2 = sms * blocks_per_sm(p.nt2);
  const auto up = [](size_t x) { return (x + 127) & ~(size_t)127; };
  p.groups = 0;
  p.skip = up((size_t)groups * sizeof(Group));
  p.kept = p.skip + up((size_t)B * sizeof(int32_t));
  p.lse = p.kept + up((size_t)N * heads * D * sizeof(float));
  p.pass1 = p.lse + up((size_t)N * heads * sizeof(float));
  p.pass2 = p.pass1 + up(workspace_size(groups, p.workers1, p.nt1, D));   // the passes overlap: each has its own
  p.total = p.pass2 + workspace_size(B, p.workers2, p.nt2, D);
  return p;
}

}  // namespace svkv

size_t spec_kv_attention_workspace_bytes(int B, int max_tokens, int q_heads, int kv_heads, int head_dim) {
  using namespace svkv;
  if (B < 1 || B > 65535 || max_tokens < 1 || max_tokens > (1 << 24) || kv_heads < 1 || kv_heads > 256 ||
      q_heads < kv_heads || q_heads % kv_heads || q_heads / kv_heads > 64 || (head_dim != 64 && head_dim != 128))
    return 0;
  const int nt = row_tiles(max_tokens, q_heads / kv_heads, head_dim);
  const int workers = sm_count() * blocks_per_sm(nt);
  return workers < 1 ? 0 : workspace_size(B, workers, nt, head_dim);
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
  if (const sv_status bad = check_attention(w, q, q_stride, k_codes, k_scale, v_codes, v_scale, scale, window, out, lse)) return bad;
  const int nt = row_tiles(max_tokens, q_heads / kv_heads, head_dim);
  const int sms = aligned(workspace, 16) ? sm_count() : 1;
  if (sms < 1) return SV_ERR_CUDA;
  const int workers = sms * blocks_per_sm(nt);
  if (!aligned(workspace, 16) || workspace_bytes < workspace_size(B, workers, nt, head_dim))
    return SV_ERR_WORKSPACE;
  AttnArgs A = arguments(w, q, q_stride, k_codes, k_scale, v_codes, v_scale, scale, window, out, lse);
  return launch_pass(A, nt, workers, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream));
}

size_t spec_kv_attention_shared_workspace_bytes(int B, int groups, int N, int max_tokens, int q_heads, int kv_heads,
                                                int head_dim) {
  using namespace svkv;
  if (groups < 1 || groups > B || N < 1 || N > (1 << 24) || max_tokens > N ||
      spec_kv_attention_workspace_bytes(B, max_tokens, q_heads, kv_heads, head_dim) == 0)
    return 0;
  return shared_plan(B, groups, N, max_tokens, q_heads / kv_heads, q_heads, head_dim, sm_count()).total;
}

sv_status spec_kv_attention_shared(const void* q, long long q_stride, const void* k_codes, const float* k_scale,
                                   const void* v_codes, const float* v_scale, const int32_t* seq_len,
                                   const int32_t* cu_tokens, const int32_t* page_table, const int32_t* cu_groups,
                                   const int32_t* shared_len, int B, int groups, int N, int max_tokens, int max_pages,
                                   int num_pages, int page_size, int q_heads, int kv_heads, int head_dim, float scale,
                                   void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace svkv;
  if (!q || !k_codes || !k_scale || !v_codes || !v_scale || !seq_len || !cu_tokens || !page_table || !cu_groups ||
      !shared_len || !out || !workspace)
    return SV_ERR_NULL;
  const Window w{seq_len, cu_tokens, page_table, B,       N,        max_tokens, max_pages,
                 num_pages, page_size, q_heads,  kv_heads, head_dim};
  if (const sv_status bad = check_attention(w, q, q_stride, k_codes, k_scale, v_codes, v_scale, scale, 0, out, lse)) return bad;
  if (groups < 1 || groups > B) return SV_ERR_SHAPE;
  if (!aligned(cu_groups, 4) || !aligned(shared_len, 4)) return SV_ERR_ALIGN;
  const int sms = aligned(workspace, 16) ? sm_count() : 1;
  if (sms < 1) return SV_ERR_CUDA;
  const SharedPlan p = shared_plan(B, groups, N, max_tokens, q_heads / kv_heads, q_heads, head_dim, sms);
  if (!aligned(workspace, 16) || workspace_bytes < p.total) return SV_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AttnArgs A = arguments(w, q, q_stride, k_codes, k_scale, v_codes, v_scale, scale, 0, out, lse);
  A.kept = reinterpret_cast<float*>(ws + p.kept);
  A.kept_lse = reinterpret_cast<float*>(ws + p.lse);
  Group* g = reinterpret_cast<Group*>(ws + p.groups);
  int32_t* skip = reinterpret_cast<int32_t*>(ws + p.skip);
  // What is read again at most where every sequence reads its own row of the table; below this much two passes
  // take longer: 4 samples on 3,000 tokens, 20 MB: 27 us in one pass and 41 in two; 96 samples of 6 prompts of 5,000
  // tokens, narrow heads, 300 MB: 51 and 58; 64 windows on 8,000 tokens, 1.1 GB: 199 and 110.
  if ((long long)(B - groups) * max_pages * page_size * kv_heads * 2 * head_dim < SHARED_BYTES)
    return launch_pass(A, p.nt2, p.workers2, ws + p.pass2, st);
  kv_groups_kernel<<<(groups + 7) / 8, 256, 0, st>>>(w, cu_groups, shared_len, groups, g, skip);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  A.groups = g;
  A.w.B = groups;
  if (const sv_status bad = launch_pass(A, p.nt1, p.workers1, ws + p.pass1, st)) return bad;
  A.groups = nullptr;
  A.w.B = B;
  A.skip = skip;
  return launch_pass(A, p.nt2, p.workers2, ws + p.pass2, st);
}

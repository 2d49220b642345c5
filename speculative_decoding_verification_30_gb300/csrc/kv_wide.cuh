// kv_wide.cuh -- attention of many query rows over the paged 8-bit cache (prompt
// chunks): included by kv_attention.cu, whose schedule and join it shares.
//
// With some hundred query rows the products outweigh the cache's bytes, so they run on
// the 5th-generation tensor cores: 4 head_dim flops for each (row, key). An item has up
// to 256 rows, two tiles of 128 that take turns: while one is in its softmax the tensor
// cores work for the other. Per unit of 128 tokens:
//   S = Q K^T  in fp16: keys widened (exactly) into shared memory, queries
//              scaled by a power of two so that the row's largest element is in [2^7, 2^8).
//              Elements keep their 8 bits down to 2^-24 of that, as in the kernel for few
//              rows: a query's precision does not depend on what else is in the batch;
//   softmax    a thread to a row: S from TMEM, weights to TMEM as fp16 over S;
//   O += P V   weights from TMEM, values widened likewise, head_dim along the rows.
// O stays in TMEM and is scaled there when a row's frame moves.
// Measured: 3 sequences of up to 700 new tokens on up to 12,000 cached, 32 heads on 8: 240
// us, 824 TFLOP/s. Bound by the chain of a tile, next logits, softmax, second product, of
// which the softmax is the longest part: 2,100 clocks a unit (of 4,400, taken before keys were
// widened), 1,500 of them the weights. Their exponentials need a third of that (32 a clock on an SM, measured); the rest is
// the latency of loading, waiting for and computing a row's quarters in turn. Tried, when the
// products ran on the codes themselves with a query as the sum of two e4m3 numbers (228 us, but
// elements below 2^-9 of a row's largest lost bits: logits 1e-2 off beside a channel 300 times
// the others): units in halves of 64 tokens, so that one half's products run beside the other's
// softmax, 291 us (twice the products, each with N = 64 and little faster than N = 128); weights
// handed over in two halves, 239; one pass that guesses the frame and repeats, 280 against 257
// for two passes.
// Warps: 0 copies (TMA), 1 issues the products, 2-3 widen values, 12-13 keys, 4-7 and 8-11
// are the two tiles' rows. Every wait is bounded; one that runs out stops the block, and the
// join makes every output NaN.
#pragma once

namespace svkv {
namespace wide {

constexpr int D = 128, TOK = 128, ROWS = 256, NT = ROWS / 8;
constexpr int THREADS = 448, NM = 8;   // stages of a unit's facts
// Stages of codes of keys and of values, and of these widened. A unit's widened values are
// read by the second product of both tiles, and the next ones are not wanted before the
// first tile's next softmax is through: one stage does. Keys are wanted as soon as that
// product is issued, so they are widened a unit ahead.
constexpr int NK = 2, NV = 1, NWK = 2, NWV = 1;
constexpr int TILE8 = TOK * D, TILE16 = 2 * TILE8;
// instruction descriptors: fp16 x fp16, fp32 accumulator, M = 128, N = 128; the second
// operand's rows along K, and along N
constexpr uint32_t ID_QK = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t ID_PV = ID_QK | (1u << 16);

struct Item {                 // what the rows need of an item
  int row0, count, i0, r0, h, slot, flags, pad;
};
struct __align__(16) Ctl {
  Meta meta[NM];
  Item item[NM];
  unsigned long long kfull[NK], kempty[NK], vfull[NV], vempty[NV];           // codes
  unsigned long long wkfull[NWK], wkempty[NWK], wvfull[NWV], wvempty[NWV];   // widened
  unsigned long long sfull[2], pfull[2], qfull[2], ofull[2], ready[NM], done;
  // NaN values of units that only some rows see: a bit for each element of a token, and
  // the unit (+ 1) that last had any
  uint4 nan[NWV][TOK];
  int nan_unit[NWV];
  uint32_t taddr;
  int err;
  long long sum[THREADS / 32], pre;
  int start_b;
};
constexpr int SMEM = 1024 + 2 * TILE16 + (NK + NV) * TILE8 + (NWK + NWV) * TILE16 + (int)sizeof(Ctl);
static_assert(SMEM <= 227 * 1024, "one block on an SM");

__device__ __forceinline__ void arrive(unsigned long long* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void expect(unsigned long long* b, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
// Waits for a phase, for at most `limit` ns, unless another wait of the block has run out.
__device__ __forceinline__ bool wait(unsigned long long* b, uint32_t parity, volatile int* err,
                                     uint64_t limit = SPEC_KV_WAIT_NS) {
  const uint32_t at = smem_u32(b);
  if (limit == 0) {   // a test's
    *err = 1;
    return false;
  }
  if (arrived(at, parity)) return true;
  const uint64_t t0 = now_ns();
  while (!arrived(at, parity)) {
    if (*err) return false;
    if (now_ns() - t0 > limit) {
      *err = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_warp(unsigned long long* b, uint32_t parity, volatile int* err) {
  return __all_sync(0xffffffffu, wait(b, parity, err));
}
__device__ __forceinline__ void after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void commit(unsigned long long* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b)) : "memory");
}
// Shared-memory descriptor, 128-byte swizzle: groups of eight 128-byte rows 1024 bytes
// apart; `lead` between the blocks of 64 fp16 along N (rows along N only).
__device__ __forceinline__ uint64_t desc(uint32_t at, uint32_t lead) {
  return (uint64_t)((at >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_qk(uint32_t d, uint64_t a, uint64_t b, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(ID_QK), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(ID_PV), "r"(add)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// 16 columns and, in `top`, the largest of them (no NaN); not waited for.
__device__ __forceinline__ void tmem_max16(uint32_t (&r)[16], float& top, uint32_t at) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, %16, [%17];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=f"(top)
      : "r"(at));
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Two floats in one 64-bit register, for the packed instructions.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}

// Largest exponent of a row's logits in a unit. `s`: the row's 128 columns of TMEM; rs >= 0,
// so within a run of 16 tokens, whose scales are the same, the largest product has it: the
// load finds that itself.
__device__ __forceinline__ float largest(const Meta& M, uint32_t s, float rs) {
  float best = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 8; c += 4) {
    uint32_t x[4][16];
    float top[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) tmem_max16(x[k], top[k], s + 16 * (c + k));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      asm volatile("" : "+f"(top[k]));   // not before the wait
      const float4 run = M.run[c + k];
      best = fmaxf(best, fmaf(top[k], rs * run.x, run.y));
    }
  }
  return best;
}
// The same where not every row sees every token.
__device__ __forceinline__ float largest_seen(const Meta& M, uint32_t s, float rs, int hi, int lo) {
  float best = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t x[32];
    tmem_ld32(x, s + 32 * c);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float4 run = M.run[2 * c + half];
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int at = 32 * c + 16 * half + k;
        if (at <= hi && at > lo && run.w == 0.f) top = fmaxf(top, __uint_as_float(x[16 * half + k]));
      }
      if (top > -INFINITY) best = fmaxf(best, fmaf(top, rs * run.x, run.y));
    }
  }
  return best;
}

// A row's weights in the frame m, written over its logits as fp16 (a quarter's weights
// cover only columns that have been read); their sum without the value scales.
template <bool MASK>
__device__ __forceinline__ float weights(const Meta& M, uint32_t s, float rs, float m, int hi, int lo) {
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t x[32], p[16];
    tmem_ld32(x, s + 32 * c);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float4 run = M.run[2 * c + half];
      const float a = rs * run.x, b = run.y - m;
      const uint64_t a2 = pair(a, a), b2 = pair(b, b);
      uint64_t part = 0;
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        uint64_t y2;
        float y[2];
        asm("fma.rn.f32x2 %0, %1, %2, %3;"
            : "=l"(y2)
            : "l"(pair(__uint_as_float(x[16 * half + k]), __uint_as_float(x[16 * half + k + 1]))), "l"(a2), "l"(b2));
        unpair(y2, y[0], y[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = 32 * c + 16 * half + k + e;
          if (MASK && (at > hi || at <= lo || run.w != 0.f)) y[e] = -INFINITY;
          y[e] = ex2f(y[e]);
        }
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(part) : "l"(part), "l"(pair(y[0], y[1])));
        p[8 * half + k / 2] = pack_h2(y[0], y[1]);
      }
      float p0, p1;
      unpair(part, p0, p1);
      sum = fmaf(p0 + p1, run.z, sum);
    }
    tmem_st16(s + 16 * c, p);
  }
  return sum;
}

__global__ void __launch_bounds__(THREADS, 1)
    kv_wide_kernel(const AttnArgs A, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char* sq = smem;                       // [tile][d / 64][row][64] fp16
  unsigned char* sk = sq + 2 * TILE16;            // [stage][token][d] codes
  unsigned char* sv = sk + NK * TILE8;
  unsigned char* swk = sv + NV * TILE8;           // [stage][d / 64][token][64] fp16
  unsigned char* swv = swk + NWK * TILE16;
  Ctl& C = *reinterpret_cast<Ctl*>(swv + NWV * TILE16);
  volatile int* err = &C.err;
  const Window& w = A.w;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = A.group;

  if (tid == 0) {
    const auto init = [](unsigned long long* b, int n) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
    };
    for (int i = 0; i < NK; ++i) init(&C.kfull[i], 1), init(&C.kempty[i], 2);
    for (int i = 0; i < NV; ++i) init(&C.vfull[i], 1), init(&C.vempty[i], 2);
    for (int i = 0; i < NWK; ++i) init(&C.wkfull[i], 2), init(&C.wkempty[i], 1);
    for (int i = 0; i < NWV; ++i) init(&C.wvfull[i], 2), init(&C.wvempty[i], 1);
    for (int t = 0; t < 2; ++t) init(&C.sfull[t], 1), init(&C.pfull[t], 4), init(&C.qfull[t], 4), init(&C.ofull[t], 1);
    for (int i = 0; i < NM; ++i) init(&C.ready[i], 1);
    init(&C.done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    C.err = 0;
    for (int i = 0; i < NWV; ++i) C.nan_unit[i] = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&C.taddr)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    before_sync();
  }
  if (A.groups) asm volatile("griddepcontrol.wait;" ::: "memory");   // kv_groups_kernel's
  long long u0, u1;
  const bool some = find_share<ROWS, TOK, THREADS>(A, C.sum, &C.start_b, &C.pre, u0, u1);
  after_sync();
  const uint32_t tmem = C.taddr;   // S (and P) of tile t at columns 128 t, O at 256 + 128 t
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (!some) {
  } else if (warp == 0) {
    // --- copies
    int cb = C.start_b;
    long long cu = u0;
    Seq cs = rows_of(A, cb);
    Span cp = span_of<ROWS, TOK>(A, cb, cs);
    int add = added(A, cb, cs);
    int ct, ch, cr;
    {
      const long long x = u0 - C.pre;
      const int per = cp.tiles + OVERHEAD;
      const long long item = quotient(x, per);
      ct = (int)(x - item * per);
      ch = (int)quotient(item, cp.rts);
      cr = (int)(item - (long long)ch * cp.rts);
      if (lane == 0) A.start[blockIdx.x] = Start{u0 - ct, cp.tiles, ch, cr, cs.first, cs.count, add};
    }
    int entry = -1, window_b = -1, window_h = -1, window0 = 0;
    float eks = 1.f, elv = 0.f, einv = 1.f;
    const int P = w.page_size, shift = __ffs(P) - 1, box = min(P, TOK);
    int j = 0, ni = 0;   // units, items
    int nk = 0, nv = 0;  // units whose keys and values were asked for
    bool ok = true, kend = false, vend = false;
    for (;; ++j) {
      if (ct < OVERHEAD) {
        cu += OVERHEAD - ct;
        ct = OVERHEAD;
      }
      const bool on = cu < u1;
      const int ks_ = j % NK, vs_ = j % NV;
      Meta& M = C.meta[j % NM];
      if (j >= NK) ok = wait_warp(&C.kempty[ks_], (uint32_t)(j / NK - 1) & 1, err);
      if (!ok) break;
      if (!on) {
        if (lane == 0) {
          M.flags = END;
          C.item[ni % NM].flags = END;
          arrive(&C.kfull[ks_]);
          arrive(&C.ready[ni % NM]);
        }
        kend = true;
        if (j >= NV) ok = wait_warp(&C.vempty[vs_], (uint32_t)(j / NV - 1) & 1, err);
        if (!ok) break;
        if (lane == 0) arrive(&C.vfull[vs_]);
        vend = true;
        break;
      }
      const int tok0 = (cp.tile0 + ct - OVERHEAD) * TOK;
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
      // a run of 16 tokens that no query sees counts as unmapped: its page may never have been
      // written, and 0 times what its scale holds may be NaN
      const int run = 16 * lane & (TOK - 1), from = ((tok0 + run) >> shift) - window0;
      const int listed = __shfl_sync(0xffffffffu, entry, from);
      const int page = run < live && (!A.window || tok0 + run + 16 > cs.len - A.window + 1) ? listed : -1;
      const float ks = __shfl_sync(0xffffffffu, eks, from), lv = __shfl_sync(0xffffffffu, elv, from),
                  inv = __shfl_sync(0xffffffffu, einv, from);
      const bool gap = __any_sync(0xffffffffu, page < 0);
      if (lane < TOK / 16) M.run[lane] = page < 0 ? make_float4(1.f, 0.f, 1.f, 1.f) : make_float4(ks, lv, inv, 0.f);
      const int at = tok0 + (lane * box & (TOK - 1));
      const int pg = __shfl_sync(0xffffffffu, entry, (at >> shift) - window0);
      const bool mine = lane * box < TOK && pg >= 0 && at - tok0 < live;
      const int bytes = __popc(__ballot_sync(0xffffffffu, mine)) * box * D;
      __syncwarp();   // every lane's run is there before the stage is announced: without copies that completes it
      if (lane == 0) {
        const long long item0 = cu - ct, item1 = item0 + OVERHEAD + cp.tiles;
        const bool first = ct == OVERHEAD || cu == u0;
        const bool masked = gap || cs.len < 0 || tok0 + TOK - 1 > cs.len || (A.window && tok0 <= cs.len + cs.count - 1 - A.window);
        M.flags = (first ? FIRST : 0) | (cu + 1 == item1 || cu + 1 == u1 ? LAST : 0) | (masked ? MASKED : 0);
        const long long hi = cs.len < 0 ? -FAR : cs.len - tok0;
        M.hi0 = (int)min(hi, FAR);
        M.lo0 = A.window ? (int)max(min(hi - A.window, FAR), -FAR) : (int)-FAR;
        M.live = live;
        if (first) {
          Item& I = C.item[ni % NM];
          I.row0 = cs.first;
          I.count = cs.count;
          I.i0 = cr * ROWS / G;
          I.r0 = cr * ROWS % G;
          I.h = ch;
          I.slot = u0 < item0 ? 1 : 0;
          I.flags = (u0 <= item0 + OVERHEAD && u1 >= item1 ? WHOLE : 0) | add;
          arrive(&C.ready[ni % NM]);
        }
        expect(&C.kfull[ks_], bytes);
      }
      ni += ct == OVERHEAD || cu == u0;
      __syncwarp();
      const int y = (pg * w.kv_heads + ch) * P + (at & (P - 1)), d = (at - tok0) * D;
      if (mine) copy_box(smem_u32(sk + ks_ * TILE8) + d, &map_k, y, smem_u32(&C.kfull[ks_]));
      ++nk;
      if (j >= NV) ok = wait_warp(&C.vempty[vs_], (uint32_t)(j / NV - 1) & 1, err);
      if (!ok) break;
      if (lane == 0) expect(&C.vfull[vs_], bytes);
      __syncwarp();
      if (mine) copy_box(smem_u32(sv + vs_ * TILE8) + d, &map_v, y, smem_u32(&C.vfull[vs_]));
      ++nv;
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
    // What was asked for lands before the block ends, also when the others have stopped. (The
    // END went to stages that were empty.)
    if (lane == 0) {
      int never = 0;
      for (int i = max(0, nk - NK); i < nk; ++i)
        if (!(kend && i % NK == j % NK)) wait(&C.kfull[i % NK], (uint32_t)(i / NK) & 1, &never, LAND_NS);
      for (int i = max(0, nv - NV); i < nv; ++i)
        if (!(vend && i % NV == j % NV)) wait(&C.vfull[i % NV], (uint32_t)(i / NV) & 1, &never, LAND_NS);
    }
    __syncwarp();
  } else if (warp == 1) {
    // --- products, issued by one thread
    if (lane == 0) {
      int items = 0;
      const auto qk = [&](int t, int j) {
        const uint64_t q0 = desc(smem_u32(sq + t * TILE16), 0), k0 = desc(smem_u32(swk + (j % NWK) * TILE16), 0);
#pragma unroll
        for (int half = 0; half < 2; ++half)   // of head_dim
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at = (half * TILE8 + 32 * k) / 16;
            mma_qk(tmem + 128 * t, q0 + at, k0 + at, half | k);
          }
        commit(&C.sfull[t]);
      };
      // unit j's first product for tile t needs the keys, and new queries if an item begins
      const auto begin = [&](int j) {
        if (!wait(&C.wkfull[j % NWK], (uint32_t)(j / NWK) & 1, err)) return -1;
        return C.meta[j % NM].flags;
      };
      int flags = begin(0);
      if (flags >= 0 && !(flags & END)) {
        bool ok = true;
        for (int t = 0; t < 2 && ok; ++t) {
          ok = wait(&C.qfull[t], 0, err);
          after_sync();
          if (ok) qk(t, 0);
        }
        if (ok) commit(&C.wkempty[0]);
        ++items;
        for (int j = 0; ok; ++j) {
          const int now = flags;
          flags = begin(j + 1);
          if (flags < 0) break;
          const bool more = !(flags & END), fresh = flags & FIRST;
          ok = wait(&C.wvfull[j % NWV], (uint32_t)(j / NWV) & 1, err);
          if (!ok) break;
          const uint64_t v0 = desc(smem_u32(swv + (j % NWV) * TILE16), TOK * 128);
          for (int t = 0; t < 2 && ok; ++t) {
            ok = wait(&C.pfull[t], (uint32_t)j & 1, err);
            if (!ok) break;
            after_sync();
#pragma unroll
            for (int k = 0; k < TOK / 16; ++k)
              mma_pv(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k, v0 + 16 * 128 * k / 16,
                     (uint32_t)(k != 0 || !(now & FIRST)));
            if (t == 1) commit(&C.wvempty[j % NWV]);
            if (now & LAST) commit(&C.ofull[t]);
            if (more && !fresh) qk(t, j + 1);
          }
          if (!ok || !more) break;
          if (fresh) {
            for (int t = 0; t < 2 && ok; ++t) {
              ok = wait(&C.qfull[t], (uint32_t)items & 1, err);
              after_sync();
              if (ok) qk(t, j + 1);
            }
            ++items;
          }
          if (ok) commit(&C.wkempty[(j + 1) % NWK]);
        }
      }
      // wake the rows for the END
      commit(&C.done);
      int never = 0;
      wait(&C.done, 0, &never, LAND_NS);
    }
    __syncwarp();
  } else if (warp < 4 || warp >= 12) {
    // --- keys (warps 12 and 13) and values (2 and 3) to fp16. A thread has the chunk of 16
    // codes c of tokens t0, t0 + 8, ...: the swizzle is the same in all of them, so each lies
    // 1024 bytes after the last. (With two warps for both the chunks take 276 us, not 240.)
    const int me = tid & 63, t0 = me >> 3, c = me & 7;
    const int from = t0 * 128 + ((c ^ t0) << 4), to = (c >> 2) * TILE8 + t0 * 128 + (((2 * (c & 3)) ^ t0) << 4);
    const auto chunk = [&](unsigned char* at, const uint4& v) {
      uint32_t o[8];
      widen(v.x, o[0], o[1]);
      widen(v.y, o[2], o[3]);
      widen(v.z, o[4], o[5]);
      widen(v.w, o[6], o[7]);
      *reinterpret_cast<uint4*>(at + to) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(at + (to ^ 16)) = make_uint4(o[4], o[5], o[6], o[7]);
    };
    const auto all = [&](unsigned char* dst, const unsigned char* src) {
#pragma unroll 1
      for (int i = 0; i < TOK * 128; i += 4096) {
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const uint4*>(src + from + i + 1024 * k);
#pragma unroll
        for (int k = 0; k < 4; ++k) chunk(dst + i + 1024 * k, v[k]);
      }
    };
    // the warp's part of the stage is read, and written where the products read it
    const auto hand_over = [&](unsigned long long* empty, unsigned long long* full) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        arrive(empty);
        arrive(full);
      }
    };
    if (warp >= 12) {
      for (int j = 0;; ++j) {
        if (!wait_warp(&C.kfull[j % NK], (uint32_t)(j / NK) & 1, err)) break;
        if (j >= NWK && !wait_warp(&C.wkempty[j % NWK], (uint32_t)(j / NWK - 1) & 1, err)) break;
        const bool end = C.meta[j % NM].flags & END;
        if (!end) all(swk + (j % NWK) * TILE16, sk + (j % NK) * TILE8);
        hand_over(&C.kempty[j % NK], &C.wkfull[j % NWK]);
        if (end) break;
      }
    } else {
      for (int j = 0;; ++j) {
        if (!wait_warp(&C.vfull[j % NV], (uint32_t)(j / NV) & 1, err)) break;
        const Meta& M = C.meta[j % NM];
        if (M.flags & END) break;
        if (j >= NWV && !wait_warp(&C.wvempty[j % NWV], (uint32_t)(j / NWV - 1) & 1, err)) break;
        const unsigned char* src = sv + (j % NV) * TILE8;
        unsigned char* dst = swv + (j % NWV) * TILE16;
        if (!(M.flags & MASKED)) {
          all(dst, src);
        } else {
#pragma unroll 1
          for (int t = t0; t < TOK; t += 8) {
            uint4 v = *reinterpret_cast<const uint4*>(src + from + 128 * (t - t0));
            if (t >= M.live || M.run[t >> 4].w != 0.f) v = make_uint4(0u, 0u, 0u, 0u);   // what is not there reads as zero
            uint32_t q[4] = {v.x, v.y, v.z, v.w}, nan = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t hit = ((q[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
              while (hit) {
                const int b = (__ffs(hit) - 1) >> 3;
                hit &= hit - 1;
                nan |= 1u << (4 * k + b);
                q[k] &= ~(0xFFu << (8 * b));
              }
            }
            // kept aside: only rows that see the token get it
            reinterpret_cast<unsigned short*>(&C.nan[j % NWV][t])[c] = (unsigned short)nan;
            if (nan) *reinterpret_cast<volatile int*>(&C.nan_unit[j % NWV]) = j + 1;
            chunk(dst + 128 * (t - t0), make_uint4(q[0], q[1], q[2], q[3]));
          }
        }
        hand_over(&C.vempty[j % NV], &C.wvfull[j % NWV]);
      }
    }
  } else {
    // --- rows: thread `r` of tile `t`
    const int t = (warp - 4) >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 128 * t, to = tmem + lanes + 256 + 128 * t;
    int j = 0;
    for (int it = 0;; ++it) {
      if (!wait_warp(&C.ready[it % NM], (uint32_t)(it / NM) & 1, err)) break;
      const Item& I = C.item[it % NM];
      if (I.flags & END) break;
      const int x = I.r0 + 128 * t + r, i = I.i0 + x / G, hd = I.h * G + x % G;
      const bool there = i < I.count;
      float rs;
      {
        uint32_t q[64];
        if (there) {
          const uint4* p = reinterpret_cast<const uint4*>(A.q + (size_t)(I.row0 + i) * (size_t)A.q_stride + (size_t)hd * D);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint4 v = p[k];
            q[4 * k] = v.x, q[4 * k + 1] = v.y, q[4 * k + 2] = v.z, q[4 * k + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int k = 0; k < 64; ++k) q[k] = 0u;
        }
        uint32_t top = 0u;
#pragma unroll
        for (int k = 0; k < 64; ++k) {
          const uint32_t a = (q[k] << 16) & 0x7FFFFFFFu, b = q[k] & 0x7FFF0000u;
          if (a < 0x7F800000u) top = max(top, a);
          if (b < 0x7F800000u) top = max(top, b);
        }
        const int e = top ? min(max((int)(top >> 23) - 127 - 7, -100), 119) : 0;
        const float down = copysignf(__uint_as_float((uint32_t)(127 - e) << 23), A.scale);
        rs = __uint_as_float((uint32_t)(127 + e) << 23) * fabsf(A.scale);
        unsigned char* row = sq + t * TILE16 + r * 128;
#pragma unroll
        for (int c = 0; c < 16; ++c) {   // chunks of 8 elements
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t u = q[4 * c + k];
            h[k] = pack_h2(__uint_as_float(u << 16) * down, __uint_as_float(u & 0xFFFF0000u) * down);
          }
          *reinterpret_cast<uint4*>(row + (c >> 3) * TILE8 + (((c & 7) ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(&C.qfull[t]);

      float m = NO_FRAME, l = 0.f;
      uint32_t bad[4] = {0u, 0u, 0u, 0u};   // elements of O that a NaN value reaches
      int flags = 0;
      bool ok = true;
      for (;; ++j) {
        ok = wait_warp(&C.sfull[t], (uint32_t)j & 1, err);
        if (!ok) break;
        after_sync();
        const Meta& M = C.meta[j % NM];
        flags = M.flags;
        const int hi = M.hi0 + i, lo = M.lo0 + i;
        // the unit's largest exponent; loops over its quarters stay rolled (code that is
        // long is fetched again by every warp)
        const float best = flags & MASKED ? largest_seen(M, ts, rs, hi, lo) : largest(M, ts, rs);
        if (__any_sync(0xffffffffu, best > m + TOP)) {
          // some weight would leave its range: move the frames to the rows' maxima
          const float m2 = fmaxf(m, best - LIFT), f = ex2f(m - m2);   // f: 0 the first time
          if (!(flags & FIRST)) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t y[32];
              tmem_ld32(y, to + 32 * c);
#pragma unroll
              for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
              tmem_st32(to + 32 * c, y);
            }
          }
          l *= f;
          m = m2;
        }
        l += flags & MASKED ? weights<true>(M, ts, rs, m, hi, lo) : weights<false>(M, ts, rs, m, hi, lo);
        if (flags & MASKED) {
          // the stage holds unit j until both tiles' weights are there
          ok = wait_warp(&C.wvfull[j % NWV], (uint32_t)(j / NWV) & 1, err);
          if (!ok) break;
          if (*reinterpret_cast<volatile int*>(&C.nan_unit[j % NWV]) == j + 1)
            for (int p = max(lo + 1, 0); p <= min(hi, TOK - 1); ++p) {
              const uint4 b = C.nan[j % NWV][p];
              bad[0] |= b.x, bad[1] |= b.y, bad[2] |= b.z, bad[3] |= b.w;
            }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        before_sync();
        __syncwarp();
        if (lane == 0) arrive(&C.pfull[t]);
        if (flags & LAST) {
          ++j;
          break;
        }
      }
      if (!ok) break;
      if (!wait_warp(&C.ofull[t], (uint32_t)it & 1, err)) break;
      after_sync();
      const size_t at = (size_t)(I.row0 + i) * w.q_heads + hd;
      const bool whole = I.flags & WHOLE, add = whole && there && (I.flags & ADD);
      float own = 1.f, kept = 0.f;
      if (I.flags & ADD) after_first_pass(A);
      if (add) add_kept(m, l, A.kept_lse[at], own, kept);
      const float f = whole ? (l == 0.f ? 0.f : own / l) : 1.f;
      kept = l == 0.f ? 0.f : kept / l;
      float* slot = A.part + ((size_t)blockIdx.x * 2 + I.slot) * ROWS * (D + 2);
      const int row = 128 * t + r;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t y[32];
        tmem_ld32(y, to + 32 * c);
        if (!there) continue;
#pragma unroll
        for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
        if (add)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 z = *reinterpret_cast<const float4*>(A.kept + at * D + 32 * c + 4 * k);
            y[4 * k] = __float_as_uint(fmaf(z.x, kept, __uint_as_float(y[4 * k])));
            y[4 * k + 1] = __float_as_uint(fmaf(z.y, kept, __uint_as_float(y[4 * k + 1])));
            y[4 * k + 2] = __float_as_uint(fmaf(z.z, kept, __uint_as_float(y[4 * k + 2])));
            y[4 * k + 3] = __float_as_uint(fmaf(z.w, kept, __uint_as_float(y[4 * k + 3])));
          }
        const uint32_t b = c == 0 ? bad[0] : c == 1 ? bad[1] : c == 2 ? bad[2] : bad[3];
        if (b)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (b >> k & 1) y[k] = 0x7FC00000u;
        if (whole && !A.groups) {
          uint4* o = reinterpret_cast<uint4*>(A.out + at * D + 32 * c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t z[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(y[8 * k + 2 * b]), __uint_as_float(y[8 * k + 2 * b + 1]));
              z[b] = *reinterpret_cast<const uint32_t*>(&v);
            }
            o[k] = make_uint4(z[0], z[1], z[2], z[3]);
          }
        } else {
          float4* o = reinterpret_cast<float4*>((whole ? A.kept + at * D : slot + 2 * ROWS + row * D) + 32 * c);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            o[k] = make_float4(__uint_as_float(y[4 * k]), __uint_as_float(y[4 * k + 1]), __uint_as_float(y[4 * k + 2]),
                               __uint_as_float(y[4 * k + 3]));
        }
      }
      if (there) {
        if (whole) {
          float* to = A.groups ? A.kept_lse : A.lse;
          if (to) to[at] = LN2F * (m + log2f(l));
        } else {
          slot[2 * row] = m;
          slot[2 * row + 1] = l;
        }
      }
      before_sync();
      __syncwarp();
    }
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");   // of rows that have stopped
  before_sync();
  __syncthreads();
  after_first_pass(A);
  set_failed(A, tid, C.err);
  if (warp == 1) {
    after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace wide
}  // namespace svkv

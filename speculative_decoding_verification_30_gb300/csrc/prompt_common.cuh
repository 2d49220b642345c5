// prompt_common.cuh -- what the kernels of prompt attention and of its gradient share: the
// arguments, the walk over blocks of rows, and the sm_103a instructions they are made of
// (definitions in include/spec_prompt.h).
//
// Tiles are 128 rows of 64 or 128 bf16: in shared memory [64 elements' column][row][128
// bytes], each column 16 KB, with the 128-byte swizzle of the copy that brings it. Such a
// tile is an operand of the tensor cores in both directions: its rows along M or N with
// head_dim contracted, or its rows contracted with head_dim along N.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/spec_prompt.h"
#include "launch_cache.h"

namespace svpr {

constexpr int BLK = 128;                 // rows of a tile
constexpr int COL = BLK * 128;           // bytes of a tile's column of 64 elements
constexpr float LN2F = 0.693147180559945309f, LOG2EF = 1.44269504088896341f;

// A copy or product that takes longer is given up; the limit of the last wait, for what is
// still in flight before a block ends, is never shorter.
constexpr uint64_t LAND_NS = 200ull * 1000 * 1000;
#ifndef SPEC_PROMPT_WAIT_NS   // a test makes it 0, for all blocks or for one
#define SPEC_PROMPT_WAIT_NS LAND_NS
#endif

struct Prompts {
  const int32_t* cu;
  int B, N, q_heads, kv_heads, group, window;   // window 0: no limit
};

// Rows first .. first + len - 1 of sequence b.
struct Seq {
  int first, len;
};
__device__ __forceinline__ Seq sequence(const Prompts& p, int b) {
  Seq s;
  s.first = min(max(p.cu[b], 0), p.N);
  s.len = max(min(p.cu[b + 1], p.N) - s.first, 0);
  return s;
}

// The walk over pieces of work: `span` rows of a sequence for one of `slots` head slots. A piece
// at level x is the one with x spans before it (`up`: behind it), whose keys (queries) it
// goes over. Blocks take the pieces from the highest level to the lowest, in turn and in
// alternating order: the longest come first and the sums of their lengths are nearly even,
// without a queue. A warp walks together.
struct Walk {
  int level, b0, span, slots, up;
  long long before;   // pieces before sequence b0 of this level
};
__device__ __forceinline__ Walk walk_start(const Prompts& p, int span, int slots, int up, int lane) {
  int most = 0;
  for (int b = lane; b < p.B; b += 32) most = max(most, sequence(p, b).len);
#pragma unroll
  for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  return Walk{(most + span - 1) / span - 1, 0, span, slots, up, 0};
}
// Piece n (not below the last one asked for): sequence, its first row's token and the head slot.
__device__ __forceinline__ bool walk_to(const Prompts& p, Walk& w, long long n, int lane, Seq& s, int& token, int& slot) {
  while (w.level >= 0) {
    const int at = w.level * w.span;
    const int b = w.b0 + lane;
    const Seq mine = b < p.B ? sequence(p, b) : Seq{0, 0};
    const unsigned has = __ballot_sync(0xffffffffu, mine.len > at);
    const long long c = (long long)__popc(has) * w.slots;
    if (n < w.before + c) {
      const int x = (int)(n - w.before), r = x / w.slots, from = __fns(has, 0, r + 1);
      s.first = __shfl_sync(0xffffffffu, mine.first, from);
      s.len = __shfl_sync(0xffffffffu, mine.len, from);
      token = w.up ? (s.len - 1) / w.span * w.span - at : at;
      slot = x - r * w.slots;
      return true;
    }
    w.before += c;
    w.b0 += 32;
    if (w.b0 >= p.B) {
      w.b0 = 0;
      --w.level;
    }
  }
  return false;
}
// The piece that a block takes in its turn k.
__device__ __forceinline__ long long piece_of(int k) {
  return (long long)k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
typedef unsigned long long Bar;
__device__ __forceinline__ void bar_init(Bar* b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void arrive(Bar* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void expect(Bar* b, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
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
// Waits for a phase, for at most `limit` ns, unless another wait of the block has run out.
__device__ __forceinline__ bool wait(Bar* b, uint32_t parity, volatile int* err, uint64_t limit = SPEC_PROMPT_WAIT_NS) {
  const uint32_t at = smem_u32(b);
  if (limit == 0) {   // a test's
    *err = 1;
    return false;
  }
  if (arrived(at, parity)) return true;
  // the clock is looked at now and then: reading it takes longer than asking again
  uint64_t t0 = 0;
  for (uint32_t asked = 1; !arrived(at, parity); ++asked) {
    if (asked % 32) continue;
    if (*err) return false;
    const uint64_t t = now_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > limit) {
      *err = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_warp(Bar* b, uint32_t parity, volatile int* err, uint64_t limit = SPEC_PROMPT_WAIT_NS) {
  return __all_sync(0xffffffffu, wait(b, parity, err, limit));
}
// One lane of a warp that has come together, always the same: it issues products and commits them.
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void commit(Bar* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b)) : "memory");
}
// A tile's column: 64 elements from x (a multiple of 64), 128 rows from y.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int y, Bar* b) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(b))
      : "memory");
}
template <int D>
__device__ __forceinline__ void copy_tile(unsigned char* dst, const CUtensorMap* map, int head, int row, Bar* b) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) copy_box(smem_u32(dst) + c * COL, map, head * D + 64 * c, row, b);
}

// Shared-memory descriptor of a tile: 128-byte swizzle, groups of eight rows 1024 bytes apart;
// `lead` between the columns of 64 elements where these lie along N.
__device__ __forceinline__ uint64_t desc(uint32_t at, uint32_t lead) {
  return (uint64_t)((at >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptors: bf16 x bf16, fp32 accumulator, M = 128, N = n; the second operand's rows
// along N, or (FLIP) contracted.
constexpr uint32_t idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
constexpr uint32_t FLIP = 1u << 16;
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(add)
      : "memory");
}
// d [128][128] = a b^T over head_dim, both tiles of shared memory.
template <int D>
__device__ __forceinline__ void mma_dims(uint32_t d, const unsigned char* a, const unsigned char* b) {
  const uint64_t a0 = desc(smem_u32(a), 0), b0 = desc(smem_u32(b), 0);
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = (c * COL + 32 * k) / 16;
      mma_ss(d, a0 + at, b0 + at, idesc(BLK), c | k);
    }
}
// d [128][D] (+)= a b over the rows of the tile b; a: bf16 in TMEM, its second half `gap` columns
// further than behind the first.
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, const unsigned char* b, bool add, int gap = 0) {
  const uint64_t b0 = desc(smem_u32(b), COL);
#pragma unroll
  for (int k = 0; k < BLK / 16; ++k)
    mma_ts(d, a + 8 * k + (k < 4 ? 0 : gap), b0 + 16 * 128 * k / 16, idesc(D) | FLIP, (uint32_t)(k != 0 || add));
}

// 32 columns of TMEM, a row to a lane; not waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t* r, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
// The same and, in `top`, the largest of them as floats (no NaN).
__device__ __forceinline__ void tmem_max32(uint32_t* r, float& top, uint32_t at) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(top)
      : "r"(at));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Holds values that a load brings back until here: the compiler may not move their use before the wait.
template <int N>
__device__ __forceinline__ void pin(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
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
__device__ __forceinline__ float ex2f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Whether one of two bf16 is NaN or infinite.
__device__ __forceinline__ uint32_t odd_bf2(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// --- host

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled encoder() {
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
// Rows of `heads` heads, `stride` elements apart, in boxes of 128 rows and 64 elements; rows
// past N read as zeros.
inline bool row_map(CUtensorMap* map, const void* p, int N, int heads, int D, long long stride) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)heads * D, (cuuint64_t)N};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, BLK}, estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline sv::LaunchCache& cache() {
  static sv::LaunchCache c;
  return c;
}
inline int sm_count() try {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cache().get(dev, reinterpret_cast<const void*>(&sm_count), 0, 0, &n, [&](int* v) {
        return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
      }) != cudaSuccess)
    return 0;
  return n;
} catch (...) {   // no exception passes the C entry points
  return 0;
}
// The kernel's shared-memory limit, raised once per device.
inline bool raise_smem(const void* fn, size_t bytes) try {
  int dev = 0, done = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cache().get(dev, fn, bytes, 0, &done, [&](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  }) == cudaSuccess;
} catch (...) {
  return false;
}
inline bool bad_shape(int B, int N, int qh, int kh, int D, float scale, int window) {
  return B < 1 || B > 65535 || N < 1 || N > (1 << 24) || kh < 1 || kh > 256 || qh < kh || qh % kh || qh / kh > 64 ||
         (D != 64 && D != 128) || !isfinite(scale) || scale < 0.f || window < 0;
}
inline bool bad_stride(long long s, int heads, int D) { return s < (long long)heads * D || s >= (1ll << 30); }
inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool rows_aligned(const void* p, long long s) { return aligned(p, 16) && (s * 2) % 16 == 0; }

}  // namespace svpr

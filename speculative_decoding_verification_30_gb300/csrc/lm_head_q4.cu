// LM-head logits with weights in 4 bits and group scales (C ABI and definitions in
// include/spec_lm_head.h). First form: a warp to each vocabulary entry and row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spec_lm_head.h"

namespace svq4 {

__global__ void q4_kernel(const __nv_bfloat16* hidden, const uint8_t* codes, const __nv_bfloat16* scale,
                          const __nv_bfloat16* bias, int M, int N, int d, int group, float* logits) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (w >= (long long)M * N) return;
  const int m = (int)(w / N), v = (int)(w % N), per = d / group;
  float sum = 0.f;
  for (int g = 0; g < per; ++g) {
    float a = 0.f, x = 0.f;
    for (int j = 2 * lane; j < group; j += 64) {
      const uint8_t c = codes[(size_t)v * (d / 2) + (g * group + j) / 2];
      const __nv_bfloat16* h = hidden + (size_t)m * d + g * group + j;
      const float h0 = __bfloat162float(h[0]), h1 = __bfloat162float(h[1]);
      a = fmaf((float)((c & 15) - 8), h0, fmaf((float)((c >> 4) - 8), h1, a));
      x += h0 + h1;
    }
    const float s = __bfloat162float(scale[(size_t)v * per + g]), b = __bfloat162float(bias[(size_t)v * per + g]);
    sum = fmaf(s, a, fmaf(fmaf(8.f, s, b), x, sum));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) logits[w] = sum;
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
  const long long blocks = ((long long)M * N + 3) / 4;
  if (blocks > 2147483647ll) return SV_ERR_SHAPE;
  q4_kernel<<<(unsigned)blocks, 128, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const __nv_bfloat16*>(hidden), codes, static_cast<const __nv_bfloat16*>(scale),
      static_cast<const __nv_bfloat16*>(bias), M, N, d, group, logits);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

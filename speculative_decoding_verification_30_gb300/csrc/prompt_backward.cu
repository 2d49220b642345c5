// The gradient of causal attention over packed prompts (C ABI and definitions in
// include/spec_prompt.h). First form: a warp to each row, its head's elements spread over
// the lanes.
#include "prompt_common.cuh"

namespace svpr {

struct Args {
  const __nv_bfloat16 *q, *k, *v, *go;
  long long qs, ks, vs, gs;
  const int32_t* cu;
  int B, N, qh, kh, group, window;
  float scale;
  __nv_bfloat16* out;
  float* lse;
  __nv_bfloat16 *gq, *gk, *gv;
  float* delta;
};

// Sequence of row r: [first, end), or an empty one.
__device__ __forceinline__ void rows_of(const Args& A, int r, int& first, int& end) {
  int lo = 0, hi = A.B;   // the last b with cu[b] <= r
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (A.cu[mid] <= r) lo = mid;
    else hi = mid;
  }
  first = max(A.cu[lo], 0);
  end = min(A.cu[lo + 1], A.N);
  if (r < first || r >= end) first = end = r;
}
__device__ __forceinline__ float all_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <int E>
__device__ __forceinline__ void load(float (&x)[E], const __nv_bfloat16* p, int lane) {
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = __bfloat162float(p[lane * E + e]);
}
template <int E>
__device__ __forceinline__ float dot(const float (&x)[E], const float (&y)[E]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) s = fmaf(x[e], y[e], s);
  return all_sum(s);
}

template <int D>
__global__ void grad_q_kernel(const Args A) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (w >= (long long)A.N * A.qh) return;
  const int r = (int)(w / A.qh), h = (int)(w % A.qh), kv = h / A.group;
  int first, end;
  rows_of(A, r, first, end);
  const int lo = A.window ? max(first, r - A.window + 1) : first;
  float q[E], go[E], o[E], g[E];
  load(q, A.q + (size_t)r * A.qs + (size_t)h * D, lane);
  load(go, A.go + (size_t)r * A.gs + (size_t)h * D, lane);
  load(o, A.out + (size_t)w * D, lane);
  const float delta = dot(go, o), lse = A.lse[w];
  if (lane == 0) A.delta[w] = delta;
#pragma unroll
  for (int e = 0; e < E; ++e) g[e] = 0.f;
  if (first < end)
    for (int j = lo; j <= r; ++j) {
      float k[E], v[E];
      load(k, A.k + (size_t)j * A.ks + (size_t)kv * D, lane);
      load(v, A.v + (size_t)j * A.vs + (size_t)kv * D, lane);
      const float ds = expf(dot(q, k) * A.scale - lse) * (dot(go, v) - delta) * A.scale;
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = fmaf(ds, k[e], g[e]);
    }
#pragma unroll
  for (int e = 0; e < E; ++e) A.gq[(size_t)w * D + lane * E + e] = __float2bfloat16_rn(g[e]);
}

template <int D>
__global__ void grad_kv_kernel(const Args A) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (w >= (long long)A.N * A.kh) return;
  const int r = (int)(w / A.kh), kv = (int)(w % A.kh);
  int first, end;
  rows_of(A, r, first, end);
  if (A.window) end = min(end, r + A.window);
  float k[E], v[E], gk[E], gv[E];
  load(k, A.k + (size_t)r * A.ks + (size_t)kv * D, lane);
  load(v, A.v + (size_t)r * A.vs + (size_t)kv * D, lane);
#pragma unroll
  for (int e = 0; e < E; ++e) gk[e] = gv[e] = 0.f;
  for (int h = kv * A.group; h < (kv + 1) * A.group; ++h)
    for (int i = r; i < end; ++i) {
      float q[E], go[E];
      load(q, A.q + (size_t)i * A.qs + (size_t)h * D, lane);
      load(go, A.go + (size_t)i * A.gs + (size_t)h * D, lane);
      const size_t at = (size_t)i * A.qh + h;
      const float p = expf(dot(q, k) * A.scale - A.lse[at]), ds = p * (dot(go, v) - A.delta[at]) * A.scale;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        gk[e] = fmaf(ds, q[e], gk[e]);
        gv[e] = fmaf(p, go[e], gv[e]);
      }
    }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    A.gk[(size_t)w * D + lane * E + e] = __float2bfloat16_rn(gk[e]);
    A.gv[(size_t)w * D + lane * E + e] = __float2bfloat16_rn(gv[e]);
  }
}

template <int D>
static sv_status backward(const Args& A, cudaStream_t st) {
  const unsigned nq = (unsigned)(((long long)A.N * A.qh + 3) / 4), nk = (unsigned)(((long long)A.N * A.kh + 3) / 4);
  grad_q_kernel<D><<<nq, 128, 0, st>>>(A);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  grad_kv_kernel<D><<<nk, 128, 0, st>>>(A);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace svpr

size_t spec_prompt_attention_backward_workspace_bytes(int N, int q_heads) {
  if (N < 1 || N > (1 << 24) || q_heads < 1 || q_heads > 64 * 256) return 0;
  return (((size_t)N * q_heads * sizeof(float)) + 15) & ~(size_t)15;
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
  if (!aligned(workspace, 16) || workspace_bytes < spec_prompt_attention_backward_workspace_bytes(N, q_heads))
    return SV_ERR_WORKSPACE;
  Args A = {};
  A.q = static_cast<const __nv_bfloat16*>(q), A.k = static_cast<const __nv_bfloat16*>(k);
  A.v = static_cast<const __nv_bfloat16*>(v), A.go = static_cast<const __nv_bfloat16*>(grad_out);
  A.qs = q_stride, A.ks = k_stride, A.vs = v_stride, A.gs = go_stride;
  A.cu = cu_tokens;
  A.B = B, A.N = N, A.qh = q_heads, A.kh = kv_heads, A.group = q_heads / kv_heads, A.window = window;
  A.scale = scale;
  A.out = static_cast<__nv_bfloat16*>(const_cast<void*>(out));
  A.lse = const_cast<float*>(lse);
  A.gq = static_cast<__nv_bfloat16*>(grad_q), A.gk = static_cast<__nv_bfloat16*>(grad_k);
  A.gv = static_cast<__nv_bfloat16*>(grad_v);
  A.delta = static_cast<float*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return head_dim == 128 ? backward<128>(A, st) : backward<64>(A, st);
}

/* spec_prompt.h -- causal attention over whole prompts, packed one after the other, and
 * its gradient: what fills a target or draft layer before the first window of new tokens,
 * and what trains a draft head's attention.
 *
 * The prompts. Sequence b has rows cu_tokens[b] .. cu_tokens[b+1] - 1 of N (cu_tokens
 * [B+1] int32, ascending; a sequence that claims rows outside 0..N is cut to what there
 * is, an empty one has no rows). Token i of a sequence sees its tokens j <= i and, with
 * window > 0, j > i - window: every token sees itself. With a_ij = scale * q_i . k_j:
 *   lse_i = ln sum_j exp(a_ij),  out_i = sum_j exp(a_ij - lse_i) v_j
 * Rows of N before the first and behind the last sequence get out = 0, lse = -inf and
 * gradients 0: a buffer may be larger than what it holds.
 *
 * Layouts: q [N][q_heads][head_dim], k, v [N][kv_heads][head_dim], bf16, token r at
 * q + r * q_stride elements (heads adjacent, rows 16-byte aligned): parts of one
 * projection's output can be passed as they lie. Query head h reads kv head
 * h / (q_heads / kv_heads).
 *
 * Limits: 1 <= B <= 65535, 1 <= N <= 2^24, head_dim 64 or 128, kv_heads 1..256, q_heads a
 * multiple of kv_heads and at most 64 times it, strides below 2^30 elements, scale finite
 * and >= 0, window >= 0 (0: no limit). Pointers are device pointers, owned by the caller;
 * nothing is allocated, the calls are asynchronous on `stream` (a cudaStream_t) and read
 * cu_tokens on the device, so they can be captured in a graph and replayed.
 *
 * Products are those of bf16 numbers, exact, summed in fp32; weights are rounded to bf16
 * for the products that take them (the gradient's P and dS too). Repeated calls give the
 * same bits. Every wait for a copy or product is bounded (0.2 s); a block of threads that gives
 * one up writes NaN to all of its rows. Outputs must not overlap inputs.
 */
#ifndef SPEC_PROMPT_H
#define SPEC_PROMPT_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* out [N][q_heads][head_dim] bf16, contiguous, 16-byte aligned (written); lse
 * [N][q_heads] float (written) or NULL. A NaN or infinite value makes the elements of out
 * that it enters NaN or infinite, in the rows that see its token and in no others.
 * Returns SV_ERR_NULL, SV_ERR_SHAPE or SV_ERR_ALIGN before launching, SV_ERR_CUDA when the
 * tensor-map encoder or the launch fails. */
sv_status spec_prompt_attention(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                                long long v_stride, const int32_t* cu_tokens, int B, int N, int q_heads, int kv_heads,
                                int head_dim, float scale, int window, void* out, float* lse, void* stream);

/* Bytes of device workspace of spec_prompt_attention_backward on the current device; 0 for
 * arguments outside the limits or without a device. It need not be cleared and holds nothing between calls; calls that may run at the
 * same time must not share one. */
size_t spec_prompt_attention_backward_workspace_bytes(int B, int N, int q_heads, int kv_heads, int head_dim);

/* The gradient with respect to q, k and v of a loss whose gradient with respect to out is
 * grad_out (token stride go_stride elements, as q). out and lse are what the forward call
 * wrote for the same q, k, v, cu_tokens, scale and window. With P_ij = exp(a_ij - lse_i),
 * delta_i = grad_out_i . out_i and dS_ij = P_ij (grad_out_i . v_j - delta_i):
 *   grad_q_i = scale sum_j dS_ij k_j,  grad_k_j = scale sum_i dS_ij q_i,
 *   grad_v_j = sum_i P_ij grad_out_i   (the last two over all query heads of the kv head)
 * grad_q [N][q_heads][head_dim], grad_k, grad_v [N][kv_heads][head_dim]: bf16, contiguous,
 * 16-byte aligned (written). A NaN or infinite value makes gradients of its own sequence
 * undefined; it reaches no other sequence. workspace: 16-byte aligned.
 * Returns as spec_prompt_attention, and SV_ERR_WORKSPACE. */
sv_status spec_prompt_attention_backward(const void* grad_out, long long go_stride, const void* q, long long q_stride,
                                         const void* k, long long k_stride, const void* v, long long v_stride,
                                         const void* out, const float* lse, const int32_t* cu_tokens, int B, int N,
                                         int q_heads, int kv_heads, int head_dim, float scale, int window,
                                         void* grad_q, void* grad_k, void* grad_v, void* workspace,
                                         size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_PROMPT_H */

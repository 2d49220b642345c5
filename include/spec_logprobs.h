/* spec_logprobs.h -- log-probabilities of given tokens over logit rows, with the
 * distribution's entropy and its best alternatives, and the gradient with respect
 * to the logits. A server reports them for the tokens a verify step emitted; the
 * trainer of a draft head scores its tokens with them and needs the gradient.
 *
 * For one row x[0..V) with token t and temperature T (0 is taken as 1, so that the
 * rows of a greedy sequence are scored as they are), z = x / T and p = softmax(z):
 *   logprob = z_t - lse,  lse = ln sum_j exp(z_j)
 *   rank    = #{j : x_j > x_t} + #{j < t : x_j = x_t}   (0: t is the argmax)
 *   entropy = -sum_j p_j ln p_j   (0 ln 0 = 0)
 *   top     = the top_n tokens in the order (logit descending, id ascending), with
 *             their log-probabilities; -inf logits are never listed: places past
 *             the last finite logit hold id -1 and log-probability -inf.
 * -inf logits are legal and mean probability 0.
 *
 * A row whose token is negative (the places of out_tokens past the last emitted
 * token) is skipped: it is not read, its outputs are 0 (rank and ids -1) and its
 * gradient is 0. A data error in a row (a NaN or +inf logit, a row that is -inf
 * everywhere, a token >= V, a temperature that is negative, NaN or +inf, or so
 * small that 1 / T leaves fp32) is reported in band: NaN outputs with rank and ids -1.
 * The lowest finite value of the type is a logit like any other: a row that holds
 * nothing else is uniform (an output past fp32, then, is infinite).
 *
 * Pointers are device pointers, owned by the caller; the calls allocate nothing,
 * keep no state and are asynchronous on `stream` (a cudaStream_t).
 */
#ifndef SPEC_LOGPROBS_H
#define SPEC_LOGPROBS_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SV_LOGPROBS_MAX_TOP 32

/* Forward.
 *   logits      R rows of V elements of `dtype`, row r at logits + r * row_stride
 *               elements (row_stride >= V, or 0: one row for all tokens); any
 *               alignment of the element type
 *   tokens      [R] int32
 *   temperature [R] float, or NULL for 1
 *   top_n       0..SV_LOGPROBS_MAX_TOP
 *   logprob, entropy, lse [R] float; rank [R] int32; top_ids [R, top_n] int32;
 *   top_logprobs [R, top_n] float: written. The two top arrays may be NULL when
 *               top_n is 0.
 * Sums are held in fp32 per thread and merged in a fixed order: repeated calls give
 * the same bits. Limits: 1 <= R <= 2^24, 2 <= V <= 262144. Returns SV_ERR_SHAPE,
 * SV_ERR_DTYPE, SV_ERR_NULL or SV_ERR_ALIGN before launching anything, SV_ERR_CUDA
 * when the launch fails. */
sv_status spec_token_logprobs(const void* logits, sv_dtype dtype, int R, int V, long long row_stride,
                              const int32_t* tokens, const float* temperature, int top_n, float* logprob,
                              int32_t* rank, float* entropy, float* lse, int32_t* top_ids,
                              float* top_logprobs, void* stream);

/* Gradient of the loss with respect to the logits, from the gradients with respect
 * to logprob, entropy and top_logprobs (the choice of top_ids is held fixed):
 *   dx_j = 1/T ( g_l [j = t] + sum_i g_i [j = id_i] - p_j (g_l + sum_i g_i)
 *                - g_H p_j (ln p_j + H) )
 *   logits, dtype, R, V, row_stride, tokens, temperature: as in the forward call
 *   lse, entropy   [R] float: the forward call's outputs. Probabilities are
 *               exp(x / T - lse) up to |lse| = 64, where the rounding of lse is 2^-19 at
 *               most; past that they are formed from the row's own maximum and sum.
 *   grad_logprob, grad_entropy [R] float: either may be NULL (zero)
 *   top_ids [R, top_n] int32 (ids outside [0, V) count for nothing) and
 *   grad_top [R, top_n] float: NULL when top_n is 0
 *   grad_logits    R rows of V elements of `dtype` at grad_stride: written, rounded
 *               once from fp32. It may be the logits themselves (same stride).
 * A row whose lse is NaN (a data error) gets NaN. Limits and errors as above. */
sv_status spec_token_logprobs_backward(const void* logits, sv_dtype dtype, int R, int V, long long row_stride,
                                       const int32_t* tokens, const float* temperature, const float* lse,
                                       const float* entropy, const float* grad_logprob,
                                       const float* grad_entropy, int top_n, const int32_t* top_ids,
                                       const float* grad_top, void* grad_logits, long long grad_stride,
                                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_LOGPROBS_H */

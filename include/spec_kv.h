/* spec_kv.h -- the target model's paged 8-bit key/value cache around the verify
 * step: a window of new tokens is appended (keys and queries rotated by their
 * position on the way), then its queries attend over the cache.
 *
 * The cache. Keys and values are e4m3 codes (4 exponent and 3 fraction bits, no
 * infinity, largest value 448) in pages of `page_size` tokens:
 *   codes [num_pages][kv_heads][page_size][head_dim] uint8, one array for keys, one
 *         for values; 16-byte aligned
 *   scale [num_pages][kv_heads] float: a cached value is its code times the scale of
 *         its page and head. spec_kv_append writes powers of two; spec_kv_attention
 *         takes any positive scales of keys under which the logits stay in fp32's range, and
 *         scales of values of 2^-100 to 2^100 that lie within a factor of 2^96 of one another
 *         among the keys that a query sees (a page of zeros, to which spec_kv_append
 *         gives 2^-60, beside values up to 2^44). Past that factor, keys on the pages of the
 *         smaller scales may be lost from lse and out.
 *   page_table [B][max_pages] int32: page_table[b][j] holds positions j page_size to
 *         (j + 1) page_size - 1 of sequence b. An entry outside [0, num_pages) is
 *         an unmapped page. Pages that a call appends to belong to one sequence;
 *         pages that are only read may be shared.
 *
 * The window. The new tokens of all sequences are packed: sequence b has rows
 * cu_tokens[b] .. cu_tokens[b+1] - 1 of N (cu_tokens [B+1] int32, ascending from 0
 * to N), at positions seq_len[b] + 0, 1, ...: seq_len [B] int32 is the number of
 * tokens the cache held before the window, as spec_verify_step advances it (a
 * rejected token's place is simply written again by the next window). A negative
 * seq_len marks an empty place of the batch: nothing of it is read or written
 * but its rows of the outputs, which become 0 (lse -inf). max_tokens is a host
 * bound on the new tokens of any one sequence; a close one chooses the better kernel.
 *
 * Layouts of heads: query head h reads kv head h / (q_heads / kv_heads).
 *
 * Limits: 1 <= B <= 65535, 1 <= N <= 2^24, 1 <= max_tokens <= N, page_size 16, 32,
 * 64 or 128, head_dim 64 or 128, kv_heads 1..256, q_heads a multiple of kv_heads
 * and at most 64 times it, B * max_tokens * kv_heads < 2^31, 1 <= max_pages <= 2^20,
 * num_pages * kv_heads < 2^31 / page_size. spec_kv_append also refuses windows that
 * would take 2^31 blocks (about B * max_tokens * (q_heads + kv_heads) * head_dim /
 * 2^12). Pointers are device pointers, owned by the caller; nothing is allocated, the
 * calls are asynchronous on `stream` (a cudaStream_t) and read the lengths on the
 * device, so they can be captured in a graph and replayed.
 */
#ifndef SPEC_KV_H
#define SPEC_KV_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Appends a window.
 *   k, v   [N][kv_heads][head_dim] of `dtype`, token r at k + r * k_stride elements
 *          (heads adjacent; rows 16-byte aligned): parts of one projection's output
 *          can be passed as they lie
 *   q      [N][q_heads][head_dim] of `dtype`, stride q_stride, or NULL
 *   q_out  [N][q_heads][head_dim] of `dtype`, contiguous (written): the rotated
 *          queries; may be q itself when that is contiguous. NULL without q.
 *   cos, sin [max_pos][rot_dim / 2] float: row p holds the angles of position p;
 *          NULL with rot_dim 0 (no rotation). Keys and queries are rotated in fp32,
 *          (a, b) -> (a c - b s, b c + a s) with each product and sum rounded once;
 *          pairs are (i, i + rot_dim / 2), or (2 i, 2 i + 1) when `interleaved`.
 *          rot_dim is a multiple of 16 up to head_dim; the rest passes unchanged.
 * The scale of a page and head becomes the smallest power of two s in 2^-60..2^119
 * with max |x| <= 448 s over the finite new values in it, or stays the larger one
 * it had if the page holds earlier tokens of the sequence; when it grows, the codes
 * of those earlier tokens are rounded again to the new scale (exact but where they
 * become subnormal, as both are powers of two). Codes are x / s rounded to nearest
 * even; larger values and infinities become +-448, NaN stays NaN.
 *   flag   [1] int32 or NULL: set to 1 when a token could not be stored because its
 *          page is unmapped or lies past max_pages, its position is past max_pos, or a
 *          sequence has more than max_tokens; never cleared. The other tokens are
 *          stored; a query past max_pos becomes NaN. Of a sequence with more than
 *          max_tokens, the first max_tokens are stored and their queries written; the
 *          rest of its rows of q_out keep what they held.
 * Returns SV_ERR_NULL, SV_ERR_SHAPE, SV_ERR_DTYPE or SV_ERR_ALIGN before launching,
 * SV_ERR_CUDA when the launch fails. */
sv_status spec_kv_append(const void* k, long long k_stride, const void* v, long long v_stride, const void* q,
                         long long q_stride, void* q_out, sv_dtype dtype, const float* cos, const float* sin,
                         int rot_dim, int max_pos, int interleaved, const int32_t* seq_len,
                         const int32_t* cu_tokens, const int32_t* page_table, int B, int N, int max_tokens,
                         int max_pages, int num_pages, int page_size, int q_heads, int kv_heads, int head_dim,
                         void* k_codes, float* k_scale, void* v_codes, float* v_scale, int32_t* flag, void* stream);

/* Bytes of device workspace that spec_kv_attention needs for these arguments on the
 * current device; 0 for arguments outside the limits or without a device. The workspace need not be
 * cleared and holds nothing between calls; calls that may run at the same time must
 * not share one. */
size_t spec_kv_attention_workspace_bytes(int B, int max_tokens, int q_heads, int kv_heads, int head_dim);

/* Attention of the window's queries over the cache. With a = scale * q . k, query
 * i of sequence b (position seq_len[b] + i) sees the keys at positions p with
 * p <= seq_len[b] + i and, when window > 0, p > seq_len[b] + i - window, that lie on
 * mapped pages:
 *   lse = ln sum_p exp(a_p),  out = sum_p exp(a_p - lse) v_p
 * A query that sees nothing gets out = 0 and lse = -inf; rows of a sequence past its
 * first max_tokens are not written. What the cache holds past a sequence's last new
 * token is never looked at.
 *   q      [N][q_heads][head_dim] bf16, token stride q_stride elements (heads
 *          adjacent; rows 16-byte aligned)
 *   out    [N][q_heads][head_dim] bf16, contiguous, 16-byte aligned (written)
 *   lse    [N][q_heads] float (written) or NULL
 *   scale  a finite factor, usually head_dim^-1/2; window >= 0 (0: no limit)
 *   workspace: 16-byte aligned, spec_kv_attention_workspace_bytes() bytes
 * Products are formed from the codes as they are, from weights rounded to fp16 (11
 * bits) and from queries in fp16, scaled by a power of two for each row so that they keep
 * their 8 significant bits down to 2^-24 of the row's largest element; all sums in fp32.
 * Repeated calls give the same bits.
 * Every wait for a copy is bounded (0.2 s); if one runs out, all outputs are NaN.
 * Returns SV_ERR_NULL, SV_ERR_SHAPE, SV_ERR_ALIGN or SV_ERR_WORKSPACE before
 * launching, SV_ERR_CUDA when the tensor-map encoder or a launch fails. */
sv_status spec_kv_attention(const void* q, long long q_stride, const void* k_codes, const float* k_scale,
                            const void* v_codes, const float* v_scale, const int32_t* seq_len,
                            const int32_t* cu_tokens, const int32_t* page_table, int B, int N, int max_tokens,
                            int max_pages, int num_pages, int page_size, int q_heads, int kv_heads, int head_dim,
                            float scale, int window, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Bytes of device workspace that spec_kv_attention_shared needs for these arguments on the
 * current device (as spec_kv_attention_workspace_bytes). */
size_t spec_kv_attention_shared_workspace_bytes(int B, int groups, int N, int max_tokens, int q_heads, int kv_heads,
                                                int head_dim);

/* spec_kv_attention (without a sliding window) for a batch whose sequences have leading pages in
 * common: samples of one prompt, requests behind one system prompt. The shared pages are read
 * once for all rows of a group instead of once for each sequence; outputs are as spec_kv_attention's
 * but for the rounding of sums.
 *   cu_groups  [groups+1] int32, ascending from 0 to B: group g is the sequences cu_groups[g] ..
 *              cu_groups[g+1] - 1
 *   shared_len [groups] int32: the page table's rows of the group's sequences name pages of the
 *              same contents for the positions below shared_len[g] (the same pages, as a rule);
 *              0: none. seq_len counts these tokens, and every sequence's row of page_table has
 *              its entries for them.
 * Whole units of 128 positions below shared_len[g] and below seq_len of every sequence of the
 * group that has new tokens are read through the first such sequence's row of the table, the rest
 * through each sequence's own. Where the page table has no room for 320 MB of keys and values that
 * would be read again, every sequence reads its own row: that is faster. A negative seq_len marks an empty place, as in spec_kv_attention; it
 * limits nothing.
 * Limits: 1 <= groups <= B; other arguments, limits, outputs and statuses as in spec_kv_attention. */
sv_status spec_kv_attention_shared(const void* q, long long q_stride, const void* k_codes, const float* k_scale,
                                   const void* v_codes, const float* v_scale, const int32_t* seq_len,
                                   const int32_t* cu_tokens, const int32_t* page_table, const int32_t* cu_groups,
                                   const int32_t* shared_len, int B, int groups, int N, int max_tokens, int max_pages,
                                   int num_pages, int page_size, int q_heads, int kv_heads, int head_dim, float scale,
                                   void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_KV_H */

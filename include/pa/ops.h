/*
 * ops.h — operators of libpa.so around the attention of pa.h: rotary positions
 * and head norms with the cache write, 4-bit KV pools, and attention with a
 * sliding window.  The conventions of pa.h (ownership, streams, alignment,
 * pool layout, slots, block tables, GQA, supported shapes, errors) hold here.
 */
#ifndef PA_OPS_H_
#define PA_OPS_H_

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * pa_rope_and_cache — the step between the projections and the attention, in
 * one pass: an optional RMS norm of every query and key head, rotary
 * positions, and the write of K and V into the pools (as
 * pa_reshape_and_cache).  For token i and each head row x of q or key:
 *     x <- x / sqrt(mean(x^2) + eps) * weight       (weight NULL: no norm)
 *     (x_a, x_b) <- m (x_a cos t - x_b sin t, x_b cos t + x_a sin t)
 *                   t = positions[i] * inv_freq[j],  m = rope_scale
 * for the pairs j < rotary_dim / 2: (a, b) = (j, j + rotary_dim / 2), or with
 * interleaved != 0 (2j, 2j + 1); dims from rotary_dim on are not rotated.
 * Statistics and rotation in fp32, the angle's product in fp64 with whole
 * turns dropped (exact for far positions); each element rounded once to dtype.
 *
 *   q_out          [num_tokens][num_q_heads][head_dim], contiguous; may be q
 *                  itself where q is contiguous
 *   q, key, value  [num_tokens] rows of q_stride, k_stride, v_stride elements,
 *                  each row [heads][head_dim] contiguous (the three may be
 *                  slices of one fused projection); 16-byte aligned, strides
 *                  multiples of 16 bytes and at least a row
 *   positions      int64 [num_tokens], 8-byte aligned, |position| < 2^31
 *   slot_mapping   as in pa_reshape_and_cache; a token without a slot still
 *                  gets its q_out row
 *   inv_freq       fp32 [rotary_dim / 2], 4-byte aligned (NULL if rotary_dim is
 *                  0): a long-context scaling is a choice of these values and m
 *   q_weight,
 *   k_weight       [head_dim] in dtype, 16-byte aligned, or NULL (each apart)
 *   rotary_dim     a multiple of 16, at most head_dim (PA_ERR_UNSUPPORTED if
 *                  not a multiple)
 *   head_dim in {64, 128}, block_size in {8, 16, 32}; fp32, fp16 or bf16;
 *   num_tokens == 0 is a no-op.
 * pa_rope_and_cache_fp8 and pa_rope_and_cache_int4 write 8- and 4-bit pools:
 * every pool byte equals pa_reshape_and_cache_fp8 / _int4 of the rounded rows.
 */
pa_status pa_rope_and_cache(void* q_out, const void* q, const void* key, const void* value, void* k_cache,
                            void* v_cache, const int64_t* positions, const int64_t* slot_mapping,
                            const float* inv_freq, const void* q_weight, const void* k_weight, float eps,
                            float rope_scale, int interleaved, int rotary_dim, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, int64_t num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                            int block_size, int64_t num_blocks, pa_dtype dtype, void* stream);

pa_status pa_rope_and_cache_fp8(void* q_out, const void* q, const void* key, const void* value, void* k_cache,
                                void* v_cache, const float* k_scale, const float* v_scale, const int64_t* positions,
                                const int64_t* slot_mapping, const float* inv_freq, const void* q_weight,
                                const void* k_weight, float eps, float rope_scale, int interleaved, int rotary_dim,
                                int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t num_tokens,
                                int num_q_heads, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                                pa_dtype dtype, void* stream);

pa_status pa_rope_and_cache_int4(void* q_out, const void* q, const void* key, const void* value, void* k_cache,
                                 void* v_cache, const int64_t* positions, const int64_t* slot_mapping,
                                 const float* inv_freq, const void* q_weight, const void* k_weight, float eps,
                                 float rope_scale, int interleaved, int rotary_dim, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, int64_t num_tokens, int num_q_heads,
                                 int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, pa_dtype dtype,
                                 void* stream);

/*
 * 4-bit KV pools: 9/16 byte an element.  The 64 dims of a group (of one token
 * and kv head) share a scale and a zero, both bf16:
 *     zero  = the group's minimum rounded down to bf16
 *     scale = (maximum - zero) / 15 rounded up to bf16 (0 if that is 0, else at least 2^-126)
 *     code  = (x - zero) / scale rounded to the nearest whole number, ties to even, in 0..15 (0 where scale is 0)
 *     value = zero + scale * code
 * every step in fp32.  A group that is not finite, or whose span is not, reads
 * back as values that are not finite.  Pools are byte arrays of (block, kv head)
 * tiles of block_size * head_dim * 9 / 16 bytes:
 *   codes   block_size * head_dim / 2 bytes.  A byte holds dims d (low nibble)
 *           and d + 8 of one token, d % 16 < 8.  With u = token % 8,
 *           chunk = d / 64, m = d % 64 / 16, e = d % 8:
 *             K: lane = 4 u + e / 2, odd = e % 2;  V: lane = 4 e + u / 2, odd = u % 2
 *             byte = ((token / 16 * (head_dim / 64) + chunk) * 32 + lane) * 16
 *                    + 4 m + token % 16 / 8 + 2 odd
 *             (block_size 8: (chunk * 32 + lane) * 8 + m / 2 * 4 + m % 2 + 2 odd)
 *   groups  then block_size * head_dim / 64 words [token][group]: scale in the
 *           low half, zero in the high half.
 * pa_copy_blocks copies whole blocks of them as bytes: head_dim = tile bytes /
 * 2, block_size 1, dtype PA_F16.
 */

/* pa_reshape_and_cache_int4 — pa_reshape_and_cache into 4-bit pools (key and
 * value in fp32, fp16 or bf16).  The stored values are those of the definition
 * above, bit for bit. */
pa_status pa_reshape_and_cache_int4(const void* key, const void* value, void* k_cache, void* v_cache,
                                    const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads, int head_dim,
                                    int block_size, int64_t num_blocks, pa_dtype dtype, void* stream);

/* pa_gather_cache_int4 — the reverse: key and value [num_tokens][num_kv_heads]
 * [head_dim] get the values at the slots, rounded once to dtype (rows of
 * negative slots keep what they held).  For what has no 4-bit form of its own,
 * such as a prefill over cached tokens. */
pa_status pa_gather_cache_int4(void* key, void* value, const void* k_cache, const void* v_cache,
                               const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads, int head_dim,
                               int block_size, int64_t num_blocks, pa_dtype dtype, void* stream);

/*
 * Sliding window with first tokens that stay visible (sinks).  The query at
 * position p attends to the tokens t <= p with t > p - window or t <
 * num_sinks.  Blocks that hold no such token are not read, and their
 * block-table entries may hold anything; the others' tokens that no query of the
 * sequence sees do not count, whatever the pool holds there.
 * Scores, softmax and sums are fp32 as in pa.h.  For the product with V the
 * tensor cores take each weight rounded to the pools' 16-bit type, as in
 * pa_decode and pa_prefill (8-bit pools: to fp16; fp32 pools: not at all); in
 * one pass, a window that reaches past the context gives the same bits as they do.
 *
 * The decode entries below share a plan:
 *   partition_size  0: one thread block per (sequence, kv head); otherwise the
 *                   visible tokens are split into partitions of this many
 *                   (counted in whole blocks; 4-bit pools: in steps of 32
 *                   tokens) and the last thread block of a (sequence, kv head)
 *                   to finish merges them, as pa_decode_splitk does with
 *                   counters.  A multiple of 16 and of block_size (4-bit: of 32).
 *   workspace,
 *   counters        as in pa_decode_splitk with counters; not read where one
 *                   partition holds every visible token (NULL is fine there)
 * pa_decode_window_plan and pa_decode_int4_plan give the workspace's size in
 * *bytes (0: none needed) for *partition_size, or, where that is -1, choose
 * one for the current device first.  max_context_len, window and num_sinks
 * must be those of the call.
 */
pa_status pa_decode_window_plan(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                int max_context_len, int window, int num_sinks, int* partition_size, size_t* bytes);

pa_status pa_decode_int4_plan(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_context_len,
                              int window, int num_sinks, int* partition_size, size_t* bytes);

/*
 * pa_decode_window — pa_decode (key and value NULL) or pa_decode_append with a
 * sliding window: each sequence's newest token, at position L - 1, attends to
 * its newest `window` tokens (itself among them; window >= 1) and its first
 * num_sinks >= 0.  Other arguments as in pa_decode_append.
 */
pa_status pa_decode_window(void* out, const void* q, const void* key, const void* value, void* k_cache, void* v_cache,
                           const int32_t* block_tables, const int32_t* context_lens, float scale, int block_size,
                           int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                           int max_context_len, int64_t num_blocks, pa_dtype dtype, int window, int num_sinks,
                           int partition_size, void* workspace, size_t workspace_bytes, int32_t* counters,
                           int64_t num_counters, const int32_t* ref_counts, const int32_t* seq_order, void* stream);

/* pa_decode_window_fp8 — the same over 8-bit pools. */
pa_status pa_decode_window_fp8(void* out, const void* q, const void* key, const void* value, void* k_cache,
                               void* v_cache, const float* k_scale, const float* v_scale,
                               const int32_t* block_tables, const int32_t* context_lens, float scale, int block_size,
                               int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                               int max_context_len, int64_t num_blocks, pa_dtype dtype, int window, int num_sinks,
                               int partition_size, void* workspace, size_t workspace_bytes, int32_t* counters,
                               int64_t num_counters, const int32_t* ref_counts, const int32_t* seq_order,
                               void* stream);

/*
 * pa_decode_int4 — pa_decode over 4-bit pools (queries and outputs fp16 or
 * bf16; PA_ERR_UNSUPPORTED for fp32), whole (window 0) or with a sliding
 * window.  The codes are multiplied as whole numbers, scales and zeros applied
 * in fp32; each head's query (|q| < 2^114) is scaled by a power of two into
 * fp16's range first, exactly (elements below 2^-23 of the head's largest keep
 * 2^-34 of it).  A weight times its token's scale of V is rounded to fp16 (2^-11,
 * or 2^-30 of the largest weight times the context's largest scale).
 */
pa_status pa_decode_int4(void* out, const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* block_tables, const int32_t* context_lens, float scale, int block_size,
                         int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                         int max_context_len, int64_t num_blocks, pa_dtype dtype, int window, int num_sinks,
                         int partition_size, void* workspace, size_t workspace_bytes, int32_t* counters,
                         int64_t num_counters, const int32_t* seq_order, void* stream);

/*
 * pa_prefill_window — pa_prefill with a sliding window (window >= 1, num_sinks
 * >= 0) for every query; scale must be positive.  A token that some query of the
 * chunk attends to has to be finite: otherwise it may reach the others, as in
 * pa_prefill.  Other arguments and errors as in pa_prefill.  There is no form without a tensor map: PA_ERR_UNSUPPORTED
 * where 16- or 32-token blocks would need one that cannot be built.
 */
pa_status pa_prefill_window(void* out, const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
                            float scale, int block_size, int num_seqs, int num_q_heads, int num_kv_heads,
                            int head_dim, int max_blocks_per_seq, int max_context_len, int max_query_len,
                            int64_t num_blocks, pa_dtype dtype, int window, int num_sinks, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_OPS_H_ */

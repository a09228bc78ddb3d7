/*
 * msa_serving.h -- C ABI of what a serving step runs around the indexer
 * (msa_indexer.h) and the attention over its blocks (msa_attention.h): new
 * tokens enter the paged caches, a layer with full attention reads all of a
 * request's pages, and the step's tokens are answered with their log
 * probabilities.
 *
 * Shared conventions, paged caches, query heads and positions: as in
 * msa_attention.h.
 */
#ifndef MSA_SERVING_H
#define MSA_SERVING_H

#include "msa_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MSA_MAX_ALTERNATIVES 32  /* alternatives of one row in msa_token_logprobs */
#define MSA_MAX_GIVEN_TOKENS 256 /* given tokens of one row in msa_token_logprobs */

/*
 * Appends the keys and values of new tokens to the paged caches and, in the
 * same pass, prepares the new tokens' queries.  Keys and queries x (a head's 128
 * values) are normalised and rotated; values are taken as they are:
 *
 *     y = x * w / sqrt(mean(x^2) + eps)            (no weight w: y = x)
 *     (z_a, z_b) = (y_a cos - y_b sin, y_b cos + y_a sin),
 *                  angle = position * inv_freq[i], 0 <= i < rotary_dim / 2
 *
 * for the pairs (a, b) = (i, i + rotary_dim / 2), or (2 i, 2 i + 1) where
 * `interleaved`; dims from rotary_dim on stay y.  All of it in fp32 (angles by
 * exact integer arithmetic on fractions of a turn, so that positions up to
 * 2^31 lose nothing), rounded once to bf16.
 *
 * Row r is a token of request b: r = b * q_len + i, or, with cu_seqlens_q,
 * rows [cu_seqlens_q[b], cu_seqlens_q[b + 1]).  The n rows of a request are its
 * last n tokens: row i of them is token t = seq_lens[b] - n + i, which lies in
 * slot t % 128 of page block_table[b, t / 128].  A row whose t is negative (a
 * request shorter than q_len, a padded one of length 0) and rows behind
 * cu_seqlens_q[batch] are no tokens: their outputs are left as they were.
 *
 *   q, out_q     optional (both or neither): bf16 [total_rows, q_heads, 128], rows
 *                q_stride / out_q_stride elements apart; out_q may be q itself, in q's
 *                strides, and else overlaps none of the inputs (over rows of q, k or v:
 *                MSA_ERR_INVALID_ARG; it may lie between them).
 *   k, v         bf16 [total_rows, kv_heads, 128], rows k_stride / v_stride apart.
 *                v and v_cache may be NULL together: a cache of keys alone, such as
 *                the index-K cache (kv_heads 1).
 *                Base addresses and row strides are multiples of 16 bytes, heads of
 *                a row contiguous; values are finite, and below 2^60 where a norm
 *                squares them.
 *   q_weight, k_weight   optional fp32 [128]; NULL: no norm (of that tensor).
 *   eps          finite, >= 0.  (Where it is 0 a head of zeros stays one.)
 *   inv_freq     fp32 [rotary_dim / 2] (NULL where rotary_dim is 0), of at most 2^10 in
 *                magnitude (the angles of larger ones lose digits).
 *   rotary_dim   0..128, a multiple of 16.
 *   positions    optional int32 [total_rows]: the rows' rotary positions, where they
 *                are not t (after msa_cache_evict, keys keep the positions they were
 *                written with).  They need not be in order.
 *   total_rows   batch * q_len, or, with cu_seqlens_q, rows of the tensors.
 *   cu_seqlens_q optional int32 [batch + 1], non-decreasing from 0 on,
 *                cu_seqlens_q[batch] <= total_rows; no request has more rows than
 *                tokens.  (Where they break this MSA_FAULT_SEQ_LEN is set, and a row that is
 *                not within its request's is passed over.)  q_len is not used with it.
 *   workspace    at least 256 bytes (the fault word).
 *
 * A slot is written by one row: the pages that get new tokens are not shared, and
 * overlap neither the inputs nor out_q.
 */
msa_status msa_cache_append(const void *q, int64_t q_stride, int q_heads, void *out_q, int64_t out_q_stride,
                            const void *k, int64_t k_stride, const void *v, int64_t v_stride, int kv_heads,
                            const float *q_weight, const float *k_weight, float eps, const float *inv_freq,
                            int rotary_dim, int interleaved, const int32_t *positions, void *k_cache,
                            const int64_t *k_strides, void *v_cache, const int64_t *v_strides, int64_t num_pages,
                            const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                            const int32_t *cu_seqlens_q, int64_t total_rows, int batch, int q_len, int max_model_len,
                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * The same on an E4M3 cache: for every token and head scale = max|z| / 448 and
 * code = e4m3(z / scale), to the nearest (z times fp32's 1 / scale: within 2^-22
 * of the middle between two codes it may be either); a head whose largest value is
 * below 2^-117 has scale 0 and codes 0.  Scales fp32 [num_pages, kv_heads, 128],
 * contiguous, 16-byte aligned (an index-K cache's [num_pages, 128]).
 */
msa_status msa_cache_append_fp8(const void *q, int64_t q_stride, int q_heads, void *out_q, int64_t out_q_stride,
                                const void *k, int64_t k_stride, const void *v, int64_t v_stride, int kv_heads,
                                const float *q_weight, const float *k_weight, float eps, const float *inv_freq,
                                int rotary_dim, int interleaved, const int32_t *positions, void *k_cache,
                                const int64_t *k_strides, float *k_scale, void *v_cache, const int64_t *v_strides,
                                float *v_scale, int64_t num_pages, const int32_t *block_table, int64_t bt_stride,
                                const int32_t *seq_lens, const int32_t *cu_seqlens_q, int64_t total_rows, int batch,
                                int q_len, int max_model_len, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Attention over all of a request's tokens: msa_attention_sparse's formula, out
 * and out_lse with every block of the request selected.  out shares no memory with
 * a row of q (MSA_ERR_INVALID_ARG).  Both products accumulate in fp32; a token's
 * weight is rounded to bf16 for the second one, their sum is not.
 * q_len <= 64; batch x KV heads x tiles of 64 rows of a head x (pages of
 * max_model_len + 8) is at most 2^30.
 *
 *   workspace    at least msa_attention_paged_workspace_bytes(batch * q_len,
 *                kv_heads * group, kv_heads) bytes.
 */
size_t msa_attention_paged_workspace_bytes(int max_rows, int heads, int kv_heads);

msa_status msa_attention_paged(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                               const void *v, const int64_t *v_strides, int64_t num_pages,
                               const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens, int batch,
                               int q_len, int kv_heads, int group, int max_model_len, float scale, void *out,
                               float *out_lse, void *workspace, size_t workspace_bytes, void *stream);

/*
 * The same on an E4M3 cache with fp32 scales [num_pages, kv_heads, 128] (see
 * msa_attention_sparse_fp8).  Both products run on the codes as they are, with
 * fp32 accumulation: a query value is held exactly from 2^-14 of its row's largest
 * on, and to 2^-22 of that below; a product of weight and V scale to 2^-8 of
 * itself, or to 2^-21 of the largest such product of its row (a weight below
 * 2^-126 of the row's largest is 0, whatever its scale).
 */
msa_status msa_attention_paged_fp8(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                                   const float *k_scale, const void *v, const int64_t *v_strides,
                                   const float *v_scale, int64_t num_pages, const int32_t *block_table,
                                   int64_t bt_stride, const int32_t *seq_lens, int batch, int q_len, int kv_heads,
                                   int group, int max_model_len, float scale, void *out, float *out_lse,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Log probabilities of given tokens under p = softmax(logits[r] / temperature[r]),
 * the entropy of p and the likeliest alternatives:
 *
 *     out_logprobs[r, j]     = ln p(tokens[r, j])
 *     out_entropy[r]         = - sum_v p(v) ln p(v)
 *     out_top_ids[r, :]      = the top_n tokens of the largest logits, largest first,
 *                              equal ones by the lower token
 *     out_top_logprobs[r, :] = ln p of those
 *
 *   logits       fp32 (or bf16: logits_bf16 != 0) [rows, vocab], rows logits_stride
 *                elements apart.  Finite or -inf (NaN counts as -inf).
 *   tokens       int32 [rows, given], contiguous; a negative one is an unused slot (log
 *                probability 0), one past the vocabulary gives -inf and sets
 *                MSA_FAULT_TOKEN.
 *   temperature  optional fp32 [rows]; NULL: 1.  One that is not > 0 makes p one at
 *                the largest logit (the lowest token), as in msa_verify_draft.
 *   out_entropy  optional fp32 [rows], in nats.
 *   out_top_ids, out_top_logprobs   int32 and fp32 [rows, top_n], contiguous.  A row
 *                with fewer logits above -inf ends with -1 and -inf.
 *   workspace    at least 256 bytes (the fault word).
 *
 * A row without a logit above -inf has log probabilities of -inf and entropy 0.
 */
msa_status msa_token_logprobs(const void *logits, int logits_bf16, int64_t logits_stride, const int32_t *tokens,
                              int given, const float *temperature, int64_t rows, int vocab, int top_n,
                              float *out_logprobs, float *out_entropy, int32_t *out_top_ids, float *out_top_logprobs,
                              void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif

/*
 * msa_attention.h -- C ABI of the serving operators that follow the indexer
 * (msa_indexer.h): what reads its block ids.
 *
 * Shared conventions.  Pointers are device memory of the caller unless said
 * otherwise; work is enqueued on `stream` (a cudaStream_t as void*) and can be
 * captured in a CUDA graph; nothing is allocated and nothing synchronised.
 * Argument errors are returned before anything is enqueued.  A batch of 0 does
 * nothing and needs no pointers.  Bad device data (a length, page id, block id or
 * token out of range) never faults: the entry counts as absent and a bit is set in
 * the workspace fault word, read and cleared by msa_indexer_get_error().  Every
 * workspace is 256-byte aligned and zero-filled once before its first use; an
 * indexer workspace does where 256 bytes are asked for.  Calls that may overlap on
 * the GPU need their own.  Results do not depend on the order in which thread
 * blocks run.
 *
 * The paged K/V cache.  Pages of 128 tokens, `kv_heads` heads of dimension 128;
 * element (page, token, head, dim) of K lies at
 *     k + page * k_strides[0] + token * k_strides[1] + head * k_strides[2] + dim
 * (strides in elements; host array of 3), of V alike.  Head-major pages
 * [num_pages, kv_heads, 128, 128] make a page's tile of one head contiguous
 * and are the layout to prefer; token-major pages [num_pages, 128, kv_heads,
 * 128] work as well.  Base addresses and strides are multiples of 16 bytes.
 * Slots past a request's last token may hold anything, NaN included; the
 * tokens inside it are finite.
 *
 * Query heads: kv_heads * group; heads [h * group, (h + 1) * group) read KV
 * head h.  Positions: request b has q_len query rows b * q_len + i; position i
 * sees the first seq_lens[b] - (q_len - 1 - i) tokens.
 */
#ifndef MSA_ATTENTION_H
#define MSA_ATTENTION_H

#include "msa_indexer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MSA_MAX_GROUP 64 /* query heads of one KV head in msa_attention_sparse */

/* Further bits of the workspace fault word. */
#define MSA_FAULT_BLOCK_ID 0x10u /* a selected block past the position's last one, or past the weights (skipped) */
#define MSA_FAULT_TOKEN 0x20u    /* a drafted token outside [0, vocab) (refused) */

#define MSA_MAX_CACHE_BLOCKS 32768 /* blocks of one request that msa_cache_evict handles (2^22 tokens) */
#define MSA_MAX_DRAFT 63           /* drafted tokens of one request in msa_verify_draft */

/*
 * Attention over the selected blocks.  For query row r = b * q_len + i and head
 * h * group + g, over the visible tokens t of the blocks ids[r, h', :]:
 *
 *     s_t = scale * q . K_t,  lse = log sum_t e^(s_t),  out = sum_t e^(s_t - lse) V_t
 *
 * and for every slot j the mass the head group puts on that block:
 *
 *     mass[r, h, j] = sum_g sum_(t in block ids[r, h', j]) e^(s_t - lse_g)
 *
 *   q            bf16 [batch * q_len, kv_heads * group, 128], rows q_stride elements
 *                apart (a multiple of 8), 16-byte aligned.
 *   k, v         the bf16 cache, see above; 1 <= num_pages <= 2^24.
 *   block_table  int32 [batch, bt_stride]: physical page of a logical block.
 *   seq_lens     int32 [batch], in [0, min(max_model_len, 128 * bt_stride)].
 *   ids          int32 [batch * q_len, sel_heads, k], as msa_indexer_decode /
 *                _decode_mq write them (negative: unused); kv_heads is a multiple of
 *                sel_heads, KV head h reads row h' = h / (kv_heads / sel_heads).
 *                The blocks of one row are distinct.
 *   scale        finite, > 0.
 *   out          bf16 [batch * q_len, kv_heads * group, 128], contiguous; a row with no
 *                visible token is zero.
 *   out_lse      optional fp32 [batch * q_len, kv_heads * group]; -inf for such a row.
 *   out_mass     optional fp32 [batch * q_len, kv_heads, k]; 0 at unused slots.
 *   workspace    at least 256 bytes (the fault word).
 */
msa_status msa_attention_sparse(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                                const void *v, const int64_t *v_strides, int64_t num_pages,
                                const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                                int batch, int q_len, int kv_heads, int group, int max_model_len,
                                const int32_t *ids, int sel_heads, int topk, float scale, void *out,
                                float *out_lse, float *out_mass, void *workspace, size_t workspace_bytes,
                                void *stream);

/*
 * The same on an E4M3 cache: K[t] = e4m3(code) * k_scale[page, head, t], V alike;
 * scales fp32 [num_pages, kv_heads, 128], contiguous, 16-byte aligned, finite
 * and >= 0.  Both products run in f16 with fp32 accumulation: codes convert
 * exactly, a query row is brought to [2^13, 2^14) by a power of two, and a row's
 * products of weight and V scale are held relative to the largest of them: at 11
 * bits down to 2^-28 of it, at fewer down to 2^-38 (a weight below 2^-126 of the
 * row's largest is 0, whatever its scale).
 */
msa_status msa_attention_sparse_fp8(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                                    const float *k_scale, const void *v, const int64_t *v_strides,
                                    const float *v_scale, int64_t num_pages, const int32_t *block_table,
                                    int64_t bt_stride, const int32_t *seq_lens, int batch, int q_len,
                                    int kv_heads, int group, int max_model_len, const int32_t *ids,
                                    int sel_heads, int topk, float scale, void *out, float *out_lse,
                                    float *out_mass, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Decode attention of a batch whose requests share a prefix: position i of
 * request b sees the prefix's tokens and the first seq_lens[b] - (q_len - 1 - i)
 * tokens of its own (none where that is negative).  Same formula, same out and
 * out_lse as msa_attention_sparse, over all of these tokens.
 *
 *   prefix_table   int32 [ceil(max_prefix_len / 128)]: the prefix's pages (NULL where
 *                  max_prefix_len is 0).  Pages x KV heads x tiles of 256 rows of a head
 *                  are at most 2^30.
 *   prefix_len     device int32 [1], in [0, max_prefix_len] (outside: 0).
 *   block_table, seq_lens   each request's own pages and own tokens.
 *   workspace      at least msa_attention_prefix_workspace_bytes(batch * q_len,
 *                  kv_heads * group, kv_heads, max_prefix_len) bytes.
 */
size_t msa_attention_prefix_workspace_bytes(int max_rows, int heads, int kv_heads, int max_prefix_len);

msa_status msa_attention_prefix(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                                const void *v, const int64_t *v_strides, int64_t num_pages,
                                const int32_t *prefix_table, const int32_t *prefix_len, int max_prefix_len,
                                const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                                int batch, int q_len, int kv_heads, int group, int max_model_len, float scale,
                                void *out, float *out_lse, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Eviction from the cache by accumulated attention weight, in pages: the block
 * table is shared by the index-K cache and K/V, so a page leaves both at once.
 *
 * msa_cache_accumulate adds the mass of a step's positions to the weights, in
 * position order: for i < n_rows[b] and every used slot j (in fp32)
 *
 *     weights[b, h, ids[b * q_len + i, h', j]] += mass[b * q_len + i, h, j]
 *
 *   weights   fp32 [batch, kv_heads, cols], contiguous.
 *   ids, mass as msa_attention_sparse reads and writes them; equal ids in one row
 *             add up in slot order.
 *   n_rows    optional int32 [batch], in [0, q_len]: positions that count (a draft
 *             step's accepted ones); NULL: all.  Outside: none count.
 */
msa_status msa_cache_accumulate(float *weights, int64_t cols, const int32_t *ids, const float *mass,
                                const int32_t *n_rows, int batch, int q_len, int kv_heads, int sel_heads,
                                int topk, void *workspace, size_t workspace_bytes, void *stream);

/*
 * msa_cache_evict brings every request to at most `budget` blocks.  A request
 * with more keeps its first n_sink and last n_window blocks and, of the others,
 * those with the largest W[j] = (..(w[0][j] + w[1][j]) + ..) + w[kv_heads-1][j]
 * (fp32, in this order; -0 counts as 0, NaN as less than anything; of equal
 * ones the earlier block stays).  Kept blocks stay in order; keys keep the
 * positions they were written with.
 *
 *   block_table   int32 [batch, bt_stride], its first `cols` entries a row.
 *   seq_lens      int32 [batch], in [0, min(max_model_len, 128 * cols)].  Outside:
 *                 the request is passed through as it is.
 *   weights       fp32 [batch, kv_heads, cols], contiguous.
 *   budget        >= n_sink + n_window; n_window >= 1 (the last block, which is
 *                 being filled, stays).
 *   out_table     int32 [batch, out_stride]: the kept blocks' pages, then -1.  What lay
 *                 past a request's last block (pages allocated ahead, or left by
 *                 refused drafts) is in neither list: note it before writing in place.
 *   out_seq_lens  int32 [batch]: 128 less for each block that left.
 *   out_weights   fp32 [batch, kv_heads, cols]: the kept blocks' weights, then 0.
 *   out_freed     int32 [batch, cols]: the pages that left, in block order, then -1.
 *   out_n_freed   int32 [batch].
 * out_table, out_seq_lens and out_weights may be the inputs themselves (in place).
 */
msa_status msa_cache_evict(const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                           const float *weights, int64_t cols, int batch, int kv_heads, int max_model_len,
                           int budget, int n_sink, int n_window, int32_t *out_table, int64_t out_stride,
                           int32_t *out_seq_lens, float *out_weights, int32_t *out_freed,
                           int32_t *out_n_freed, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Verification of drafted tokens against the target's probabilities, from given
 * random numbers.  With p_i = softmax(logits[b, i] / temperature[b]) and
 * q_i = draft_probs[b, i], draft i is accepted while
 *
 *     uniforms[b, i] * q_i(x_i) < p_i(x_i).
 *
 * At the first refusal i the token is drawn from max(p_i - q_i, 0) (from p_i if
 * that is zero everywhere); with all n_draft[b] accepted it is drawn from
 * p_(n_draft).  The draw is the exponential race argmax_v r(v) / race[b, v], ties
 * to the lowest v, which picks v with probability r(v) / sum r.  A temperature
 * that is not > 0 makes p_i one at its largest logit (the lowest index).
 *
 *   logits        fp32 (or bf16: logits_bf16 != 0) [batch, max_draft + 1, vocab];
 *                 element (b, i, v) at b * logits_stride_b + i * logits_stride_i + v.
 *                 Finite or -inf (NaN counts as -inf).
 *   draft_probs   fp32 [batch, max_draft, vocab], contiguous, >= 0.
 *   draft_tokens  int32 [batch, max_draft], contiguous.
 *   uniforms      fp32 [batch, max_draft], in [0, 1).
 *   race          fp32 [batch, vocab], contiguous, > 0: draws of Exp(1).
 *   temperature   optional fp32 [batch]; NULL: 1.
 *   n_draft       optional int32 [batch], in [0, max_draft] (outside: 0); NULL: all.
 *   out_tokens    int32 [batch, max_draft + 1]: accepted drafts, the drawn token,
 *                 then -1.  A row of logits without a finite one draws -1.
 *   out_accepted  int32 [batch]: accepted drafts.
 *   out_logprobs  optional fp32 [batch, max_draft + 1]: ln p_i of each token given
 *                 out, 0 where there is none.
 */
msa_status msa_verify_draft(const void *logits, int logits_bf16, int64_t logits_stride_b,
                            int64_t logits_stride_i, const float *draft_probs, const int32_t *draft_tokens,
                            const float *uniforms, const float *race, const float *temperature,
                            const int32_t *n_draft, int batch, int max_draft, int vocab,
                            int32_t *out_tokens, int32_t *out_accepted, float *out_logprobs,
                            void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif

/*
 * msa_attention.h -- C ABI of the serving operators that follow the indexer
 * (msa_indexer.h): what reads its block ids.
 *
 * Shared conventions.  Pointers are device memory of the caller unless said
 * otherwise; work is enqueued on `stream` (a cudaStream_t as void*) and can be
 * captured in a CUDA graph; nothing is allocated and nothing synchronised.
 * Argument errors are returned before anything is enqueued.  Bad device data
 * (a length, page id, block id or token out of range) never faults: the entry
 * counts as absent and a bit is set in the workspace fault word, read and
 * cleared by msa_indexer_get_error().  Every workspace is 256-byte aligned and
 * zero-filled once before its first use; an indexer workspace does where 256
 * bytes are asked for.  Calls that may overlap on the GPU need their own.
 * Results do not depend on the order in which thread blocks run.
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
#define MSA_FAULT_BLOCK_ID 0x10u /* a selected block past the position's last one (skipped) */

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
 * exactly, a query row is brought to [2^13, 2^14) by a power of two, and the
 * weights are multiplied by V's scales relative to the largest one met.
 */
msa_status msa_attention_sparse_fp8(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                                    const float *k_scale, const void *v, const int64_t *v_strides,
                                    const float *v_scale, int64_t num_pages, const int32_t *block_table,
                                    int64_t bt_stride, const int32_t *seq_lens, int batch, int q_len,
                                    int kv_heads, int group, int max_model_len, const int32_t *ids,
                                    int sel_heads, int topk, float scale, void *out, float *out_lse,
                                    float *out_mass, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif

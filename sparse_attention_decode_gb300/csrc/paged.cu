// Attention over all of a request's tokens: argument checks and launches.
#include "overlap.h"
#include "paged_attn.cuh"

namespace msa {

bool test_withhold_pages();  // msa_indexer_test_withhold_pages
bool make_cache_map(CUtensorMap *map, const void *base, const int64_t *strides, int64_t pages, int heads, bool fp8);  // attention.cu
bool cache_ok(const void *base, const int64_t *strides, int64_t pages, int heads, bool fp8);
bool unaligned(const void *p, uintptr_t a);

// Rows of a unit: the GROUPS * N of the forms in launch_paged_rows.
static int paged_tile_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : kPagedMaxRows; }

// Two parts a CTA: a row of each is 516 bytes.
static size_t paged_workspace(int64_t max_rows, int group)
{
    return kHeaderBytes + 2 * kPagedMaxGrid * static_cast<size_t>(paged_tile_rows(max_rows * group)) * (kDim + 1) * sizeof(float);
}

// What a unit costs beside its pages (its query rows, its first page's references, its epilogue), in pages of the same type
// and rows: bf16, E4M3 up to 32 rows; E4M3 with 64, whose pages cost twice as much, counts as bf16.  64 requests of 1 to 3000
// tokens, 4 heads, with 0 / 4 / 8 / 12 / 16 pages: bf16 16 rows 52.8 us, 44.4, 45.2 with 8, 64 rows 90.2, 56.0, 57.3; E4M3 16
// rows 54.0, 29.3, 28.1, 29.2, 31.0, 32 rows 71.1, 37.8, 37.4, 39.5, 41.6, 64 rows 97.0, 54.9, 58.5, 62.0, 65.3.  24 requests of
// 2000 to 12000, E4M3: 38.5, 35.8, 36.3, 37.8, 39.1; 50.1, 45.6, 45.5, 47.7, 49.4; 75.9, 70.9, 74.0, 78.4, 82.3.
constexpr int kPagedLead[2] = {4, 8};

template <class F, int N, int WAYS, int GROUPS>
static msa_status launch_paged(const PagedParams &p, int dev, cudaStream_t st)
{
    static std::atomic<bool> allowed[kMaxDevices];
    auto *kernel = paged_attn_kernel<F, N, WAYS, GROUPS>;
    using L = PagedLayout<F, N, WAYS, GROUPS>;
    constexpr size_t smem = L::kBytes;
    if (!allow_smem(kernel, smem, dev, allowed))
        return MSA_ERR_CUDA;
    kernel<<<static_cast<unsigned>(p.grid), L::kThreads, smem, st>>>(p);
    if (cudaGetLastError() != cudaSuccess)
        return MSA_ERR_CUDA;
    if (p.grid < 2)
        return MSA_OK;
    // Few units have many parts each: blocks a unit, and 8 warps a row or 2.  Else a block for each range's end, where at most
    // one unit of 2 or 3 parts goes on.  With 8 / 2 / 0: one request of 131072 (E4M3, 4 units) 30.6 / 33.1 / 33.5 us, 8 ragged
    // ones (32 units) 64.5 / 57.0 / 59.6, 32 of 4000 (128) 59.9 / 51.6 / 49.4, 60 of 4000 (240) 99.7 / 86.3 / 83.1.
    const int rows = std::min(p.tile_rows, p.q_len * p.group);
    const int64_t units = static_cast<int64_t>(p.batch) * p.row_tiles * p.kv_heads;
    cudaLaunchAttribute attr[1];
    auto join = [&](auto *k, int64_t x, int wpr) {
        const cudaLaunchConfig_t cfg =
            pdl_config(dim3(static_cast<unsigned>(x), static_cast<unsigned>((rows * wpr + 7) / 8)), dim3(256), 0, st, attr);
        return cudaLaunchKernelEx(&cfg, k, p) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
    };
    return units * 8 <= p.grid   ? join(paged_join_kernel<8, true>, units, 8)
           : units * 2 <= p.grid ? join(paged_join_kernel<2, true>, units, 2)
                                 : join(paged_join_kernel<1, false>, p.grid - 1, 1);
}

template <class F>
static msa_status launch_paged_rows(const PagedParams &p, int dev, cudaStream_t st)
{
    // Up to 32 rows: two ways; 64: one.  E4M3 rows are worked on 16 a warpgroup, bf16 ones, which need no second and third
    // term, 32.  With 16 and 32: E4M3, 32 rows, 256 requests of 100 to 300 tokens 59.4 and 67.4 us, 64 of 1 to 3000 37.5 and
    // 40.9, 24 of 2000 to 12000 45.7 and 45.8, 32 of 31000 186.3 and 182.5; 64 rows, 32 of 31000 317 and 354, 1 of 131072 53.0
    // and 58.5; bf16, 8 of 32768, 32 rows 88.8 and 88.2, 64 rows 93.2 and 92.5.
    if (p.tile_rows == 16)
        return launch_paged<F, 16, 2, 1>(p, dev, st);
    if constexpr (F::kFp8)
        return p.tile_rows == 32 ? launch_paged<F, 16, 2, 2>(p, dev, st) : launch_paged<F, 16, 1, 4>(p, dev, st);
    else
        return p.tile_rows == 32 ? launch_paged<F, 32, 2, 1>(p, dev, st) : launch_paged<F, 32, 1, 2>(p, dev, st);
}

static msa_status paged_entry(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                              const float *k_scale, const void *v, const int64_t *v_strides, const float *v_scale,
                              int64_t num_pages, const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                              int batch, int q_len, int kv_heads, int group, int max_model_len, float scale, void *out,
                              float *out_lse, void *workspace, size_t workspace_bytes, void *stream, bool fp8)
{
    if (batch < 0 || q_len < 1 || kv_heads < 1 || group < 1 || num_pages < 1 || bt_stride < 1 || max_model_len < 1 ||
        !(scale > 0.0f) || !(scale < INFINITY))
        return MSA_ERR_INVALID_ARG;
    if (batch > MSA_MAX_BATCH || num_pages > (int64_t{1} << 24) || group > MSA_MAX_GROUP || kv_heads > 1024 ||
        q_len > 64 || static_cast<int64_t>(batch) * q_len * kv_heads * group > (int64_t{1} << 27))
        return MSA_ERR_UNSUPPORTED;
    if (batch == 0)  // (an empty tensor has no address)
        return MSA_OK;
    if (!q || !block_table || !seq_lens || !out || !workspace || !cache_ok(k, k_strides, num_pages, kv_heads, fp8) ||
        !cache_ok(v, v_strides, num_pages, kv_heads, fp8) || unaligned(q, 16) || q_stride % 8 ||
        q_stride < static_cast<int64_t>(kv_heads) * group * kDim || unaligned(out, 16) || unaligned(workspace, 256))
        return MSA_ERR_INVALID_ARG;
    if (fp8 && (!k_scale || !v_scale || unaligned(k_scale, 16) || unaligned(v_scale, 16)))
        return MSA_ERR_INVALID_ARG;
    if (workspace_bytes < paged_workspace(static_cast<int64_t>(batch) * q_len, group))
        return MSA_ERR_WORKSPACE_TOO_SMALL;
    // a unit's rows are read by every CTA that has pages of it, at any time
    const int64_t width = static_cast<int64_t>(kv_heads) * group * kDim * 2, q_rows = static_cast<int64_t>(batch) * q_len;
    if (rows_overlap(RowSpan(out, width, width, q_rows), RowSpan(q, q_stride * 2, width, q_rows)))
        return MSA_ERR_INVALID_ARG;
    PagedParams p;
    std::memset(&p, 0, sizeof p);
    p.tile_rows = paged_tile_rows(static_cast<int64_t>(q_len) * group);
    p.row_tiles = (q_len * group + p.tile_rows - 1) / p.tile_rows;
    p.seq_limit = static_cast<int>(std::min<int64_t>(max_model_len, kPage * bt_stride));
    p.lead = kPagedLead[fp8 && p.tile_rows < kPagedMaxRows];
    // the slots of all units are counted in 32 bits
    if (((static_cast<int64_t>(p.seq_limit) + kPage - 1) / kPage + p.lead) * batch * p.row_tiles * kv_heads > (1 << 30))
        return MSA_ERR_UNSUPPORTED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return MSA_ERR_CUDA;
    const int sms = device_sms(dev);
    if (sms <= 0 || !make_cache_map(&p.kmap, k, k_strides, num_pages, kv_heads, fp8) ||
        !make_cache_map(&p.vmap, v, v_strides, num_pages, kv_heads, fp8))
        return MSA_ERR_CUDA;
    p.q = static_cast<const uint16_t *>(q);
    p.kscale = k_scale;
    p.vscale = v_scale;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.out = static_cast<uint16_t *>(out);
    p.lse = out_lse;
    p.fault = &static_cast<WorkspaceHeader *>(workspace)->fault;
    p.q_stride = q_stride;
    p.bt_stride = bt_stride;
    p.num_pages = num_pages;
    p.batch = batch;
    p.q_len = q_len;
    p.kv_heads = kv_heads;
    p.group = group;
    p.grid = std::min(sms, kPagedMaxGrid);
    p.part_lse = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kHeaderBytes);
    p.part_o = p.part_lse + 2 * kPagedMaxGrid * p.tile_rows;
    p.scale_log2 = scale * kLog2e;
    p.withhold = test_withhold_pages();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return fp8 ? launch_paged_rows<PagedFp8>(p, dev, st) : launch_paged_rows<PagedBf16>(p, dev, st);
}

}  // namespace msa

using namespace msa;

extern "C" size_t msa_attention_paged_workspace_bytes(int max_rows, int heads, int kv_heads)
{
    if (max_rows < 0 || kv_heads < 1 || heads < kv_heads || heads % kv_heads)
        return 0;
    return paged_workspace(max_rows, heads / kv_heads);
}

extern "C" msa_status msa_attention_paged(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                                          const void *v, const int64_t *v_strides, int64_t num_pages,
                                          const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                                          int batch, int q_len, int kv_heads, int group, int max_model_len, float scale,
                                          void *out, float *out_lse, void *workspace, size_t workspace_bytes,
                                          void *stream)
{
    return paged_entry(q, q_stride, k, k_strides, nullptr, v, v_strides, nullptr, num_pages, block_table, bt_stride,
                       seq_lens, batch, q_len, kv_heads, group, max_model_len, scale, out, out_lse, workspace,
                       workspace_bytes, stream, false);
}

extern "C" msa_status msa_attention_paged_fp8(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                                              const float *k_scale, const void *v, const int64_t *v_strides,
                                              const float *v_scale, int64_t num_pages, const int32_t *block_table,
                                              int64_t bt_stride, const int32_t *seq_lens, int batch, int q_len,
                                              int kv_heads, int group, int max_model_len, float scale, void *out,
                                              float *out_lse, void *workspace, size_t workspace_bytes, void *stream)
{
    return paged_entry(q, q_stride, k, k_strides, k_scale, v, v_strides, v_scale, num_pages, block_table, bt_stride,
                       seq_lens, batch, q_len, kv_heads, group, max_model_len, scale, out, out_lse, workspace,
                       workspace_bytes, stream, true);
}

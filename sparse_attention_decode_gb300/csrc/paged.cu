// Attention over all of a request's tokens: argument checks and launches.
#include <cuda_fp16.h>

#include "block_attn.cuh"

#include "msa_serving.h"

namespace msa {

bool test_withhold_pages();  // msa_indexer_test_withhold_pages
bool cache_ok(const void *base, const int64_t *strides, int64_t pages, int heads, bool fp8);  // attention.cu
bool unaligned(const void *p, uintptr_t a);

struct PagedParams {
    const uint16_t *q;
    const uint8_t *k, *v;
    const float *kscale, *vscale;
    const int32_t *block_table, *seq_lens;
    uint16_t *out;
    float *lse;
    uint32_t *fault;
    int64_t q_stride, bt_stride, num_pages;
    int64_t ks[3], vs[3];
    int batch, q_len, kv_heads, group, seq_limit;
    float scale_log2;
};

__device__ __forceinline__ float e4m3_value(uint8_t c)
{
    return static_cast<float>(__half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(c) & 0xffffu))));
}

// A block a query head: thread t a token of the page, then a dim.
template <bool FP8>
__global__ void __launch_bounds__(128) paged_kernel(const __grid_constant__ PagedParams p)
{
    __shared__ float s_q[kDim], s_p[kPage], s_w[4];
    const int tid = threadIdx.x;
    const int heads = p.kv_heads * p.group;
    const int64_t row = blockIdx.x / heads;
    const int head = blockIdx.x % heads, h = head / p.group, b = static_cast<int>(row / p.q_len), i = static_cast<int>(row % p.q_len);
    const int L = p.seq_lens[b];
    const bool bad = L < 0 || L > p.seq_limit;
    if (bad && tid == 0)
        atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
    const int len = bad ? 0 : L, sees = max(0, len - (p.q_len - 1 - i));
    s_q[tid] = __uint_as_float(static_cast<uint32_t>(p.q[row * p.q_stride + head * kDim + tid]) << 16);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int base = 0; base < sees; base += kPage) {
        const int page = p.block_table[b * p.bt_stride + base / kPage];
        if (page < 0 || page >= p.num_pages) {
            if (tid == 0)
                atomicOr(p.fault, MSA_FAULT_PAGE_ID);
            continue;
        }
        const bool seen = base + tid < sees;
        const int64_t at = (static_cast<int64_t>(page) * p.kv_heads + h) * kPage;
        float s = -INFINITY;
        if (seen) {
            s = 0.0f;
            const int64_t from = page * p.ks[0] + tid * p.ks[1] + h * p.ks[2];
            for (int d = 0; d < kDim; ++d)
                s += s_q[d] * (FP8 ? e4m3_value(p.k[from + d])
                                   : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p.k)[from + d]) << 16));
            s *= p.scale_log2 * (FP8 ? p.kscale[at + tid] : 1.0f);
        }
        float top = s;
        for (int q = 16; q >= 1; q >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, q));
        if ((tid & 31) == 0)
            s_w[tid >> 5] = top;
        __syncthreads();
        const float n = fmaxf(m, fmaxf(fmaxf(s_w[0], s_w[1]), fmaxf(s_w[2], s_w[3])));
        const float f = rescale(m, n);
        m = n;
        s_p[tid] = seen ? exp2_approx(s - n) : 0.0f;
        __syncthreads();
        float sum = 0.0f, acc = 0.0f;
        const int64_t from = page * p.vs[0] + h * p.vs[2] + tid;
        for (int t = 0; t < min(kPage, sees - base); ++t) {
            sum += s_p[t];
            acc += s_p[t] * (FP8 ? e4m3_value(p.v[from + t * p.vs[1]]) * p.vscale[at + t]
                                 : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p.v)[from + t * p.vs[1]]) << 16));
        }
        l = l * f + sum;
        o = o * f + acc;
    }
    p.out[(row * heads + head) * kDim + tid] = static_cast<uint16_t>(f32x2_to_bf16x2(l > 0.0f ? o / l : 0.0f, 0.0f));
    if (tid == 0 && p.lse)
        p.lse[row * heads + head] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

static size_t paged_workspace(int64_t max_rows, int group, int kv_heads)
{
    (void)max_rows, (void)group, (void)kv_heads;
    return kHeaderBytes;
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
    if (workspace_bytes < paged_workspace(static_cast<int64_t>(batch) * q_len, group, kv_heads))
        return MSA_ERR_WORKSPACE_TOO_SMALL;
    PagedParams p;
    std::memset(&p, 0, sizeof p);
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint8_t *>(k);
    p.v = static_cast<const uint8_t *>(v);
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
    for (int i = 0; i < 3; ++i) {
        p.ks[i] = k_strides[i];
        p.vs[i] = v_strides[i];
    }
    p.batch = batch;
    p.q_len = q_len;
    p.kv_heads = kv_heads;
    p.group = group;
    p.seq_limit = static_cast<int>(std::min<int64_t>(max_model_len, kPage * bt_stride));
    p.scale_log2 = scale * kLog2e;
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(batch) * q_len * kv_heads * group);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (fp8)
        paged_kernel<true><<<grid, 128, 0, st>>>(p);
    else
        paged_kernel<false><<<grid, 128, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

}  // namespace msa

using namespace msa;

extern "C" size_t msa_attention_paged_workspace_bytes(int max_rows, int heads, int kv_heads)
{
    if (max_rows < 0 || kv_heads < 1 || heads < kv_heads || heads % kv_heads)
        return 0;
    return paged_workspace(max_rows, heads / kv_heads, kv_heads);
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

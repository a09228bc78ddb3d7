// Eviction from the paged cache by accumulated attention weight: the weights'
// update and the choice of the pages that leave.
#include "host_util.cuh"
#include "keys.cuh"
#include "layout.cuh"
#include "ptx.cuh"

#include "msa_attention.h"

namespace msa {

// ---------------------------------------------------------------------------
// weights[b, h, id] += mass, one warp per (request, KV head), lane = slot.
// Positions go one after the other and equal ids of a row add up in slot order
// in their first lane, so the sums do not depend on scheduling and need no
// atomics.  Latency-bound: q_len dependent read-modify-writes.
__global__ void __launch_bounds__(128) accumulate_kernel(float *weights, int64_t cols, const int32_t *ids,
                                                         const float *mass, const int32_t *n_rows, int batch,
                                                         int q_len, int kv_heads, int sel_heads, int topk,
                                                         uint32_t *fault)
{
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (w >= static_cast<int64_t>(batch) * kv_heads)
        return;
    const int b = static_cast<int>(w / kv_heads), h = static_cast<int>(w % kv_heads);
    int n = n_rows ? n_rows[b] : q_len;
    if (n < 0 || n > q_len) {
        if (lane == 0)
            atomicOr(fault, MSA_FAULT_SEQ_LEN);
        n = 0;
    }
    float *row = weights + w * cols;
    const int sel = h / (kv_heads / sel_heads);
    for (int i = 0; i < n; ++i) {
        const int64_t r = static_cast<int64_t>(b) * q_len + i;
        int id = -1;
        float m = 0.0f;
        if (lane < topk) {
            id = ids[(r * sel_heads + sel) * topk + lane];
            m = mass[(r * kv_heads + h) * topk + lane];
        }
        if (id >= cols) {
            atomicOr(fault, MSA_FAULT_BLOCK_ID);
            id = -1;
        }
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        const bool first = (same & ((1u << lane) - 1u)) == 0;
        float sum = id >= 0 && first ? row[id] : 0.0f;
        const bool alone = __all_sync(0xffffffffu, id < 0 || same == (1u << lane));
        if (alone) {
            sum += m;
        } else {
            for (int j = 0; j < 32; ++j) {
                const float x = __shfl_sync(0xffffffffu, m, j);
                if ((same >> j) & 1u)
                    sum += x;
            }
        }
        if (id >= 0 && first)
            row[id] = sum;
        __syncwarp();
    }
}

// ---------------------------------------------------------------------------
struct EvictParams {
    const int32_t *table;
    const int32_t *seq_lens;
    const float *weights;
    int32_t *out_table;
    int32_t *out_seq;
    float *out_weights;
    int32_t *freed;
    int32_t *n_freed;
    uint32_t *fault;
    int64_t bt_stride, out_stride;
    int cols, kv_heads, seq_limit, budget, n_sink, n_window;
};

constexpr int kEvictThreads = 512;

// A block's key, ordered as its weight: NaN lowest, then -inf .. inf, pinned blocks highest.
__device__ __forceinline__ uint32_t evict_key(float w)
{
    return w != w ? 0u : float_order_bits(w == 0.0f ? 0.0f : w);
}

// Exclusive prefix sum over the block's threads; *total gets the sum.
__device__ __forceinline__ int block_exclusive_sum(int v, int *scratch, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    if (lane == 31)
        scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = lane < kEvictThreads / 32 ? scratch[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o)
                y += z;
        }
        scratch[lane] = y;
    }
    __syncthreads();
    const int before = warp ? scratch[warp - 1] : 0;
    *total = scratch[31];
    __syncthreads();
    return before + x - v;
}

// One CTA per request.  Keys in shared memory; the budget-th largest by four
// 8-bit radix passes; equal keys at the threshold go by index through one prefix
// sum, a second one numbers the kept and the freed blocks; then table and
// weights are copied in increasing destination order (every read of a tile
// before its writes, and a source never lies below its destination), so outputs
// may be the inputs.
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const __grid_constant__ EvictParams p)
{
    extern __shared__ uint32_t evict_smem[];
    uint32_t *keys = evict_smem;
    uint16_t *list = reinterpret_cast<uint16_t *>(keys + p.cols);  // kept blocks, then the freed ones
    __shared__ int scratch[32];
    __shared__ int hist[256];
    __shared__ uint32_t s_prefix;
    __shared__ int s_want;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int L = p.seq_lens[b];
    const bool bad = L < 0 || L > p.seq_limit;
    if (bad && tid == 0)
        atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
    const int nb = bad ? p.cols : (L + kPage - 1) / kPage;
    const int keep = bad ? p.cols : min(nb, p.budget);
    const float *w = p.weights + static_cast<int64_t>(b) * p.kv_heads * p.cols;
    const int32_t *table = p.table + b * p.bt_stride;
    const int per = (nb + kEvictThreads - 1) / kEvictThreads;
    const int j0 = min(nb, tid * per), j1 = min(nb, j0 + per);

    if (keep < nb) {
        for (int j = tid; j < nb; j += kEvictThreads) {
            float sum = w[j];
            for (int h = 1; h < p.kv_heads; ++h)
                sum += w[static_cast<int64_t>(h) * p.cols + j];
            keys[j] = j < p.n_sink || j >= nb - p.n_window ? 0xffffffffu : evict_key(sum);
        }
        if (tid == 0) {
            s_prefix = 0;
            s_want = keep;
        }
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kEvictThreads)
                hist[i] = 0;
            __syncthreads();
            const uint32_t prefix = s_prefix;
            const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int j = tid; j < nb; j += kEvictThreads)
                if ((keys[j] & mask) == prefix)
                    atomicAdd(&hist[(keys[j] >> shift) & 255], 1);
            __syncthreads();
            // the bin, from the top, in which the want-th largest lies
            if (tid < 256) {
                int above = 0;
                for (int i = tid + 1; i < 256; ++i)
                    above += hist[i];
                const int want = s_want;
                if (above < want && above + hist[tid] >= want)
                    scratch[0] = tid, scratch[1] = want - above;
            }
            __syncthreads();
            if (tid == 0) {
                s_prefix = prefix | static_cast<uint32_t>(scratch[0]) << shift;
                s_want = scratch[1];
            }
            __syncthreads();
        }
    }
    const bool all = keep == nb;
    const uint32_t bound = all ? 0u : s_prefix;
    const int want = all ? 0 : s_want;  // blocks at the bound that stay
    int total;
    int ties = 0;
    if (!all)
        for (int j = j0; j < j1; ++j)
            ties += keys[j] == bound;
    const int tie0 = block_exclusive_sum(ties, scratch, &total);
    // stays(j, rank): rank counts the thread's blocks at the bound in block order
    auto stays = [&](int j, int &rank) {
        return all || keys[j] > bound || (keys[j] == bound && rank++ < want);
    };
    int mine = 0, rank = tie0;
    for (int j = j0; j < j1; ++j)
        mine += stays(j, rank);
    int at = block_exclusive_sum(mine, scratch, &total);
    int gone = keep + (j0 - at);  // freed blocks are listed after the kept ones
    rank = tie0;
    for (int j = j0; j < j1; ++j)
        list[stays(j, rank) ? at++ : gone++] = static_cast<uint16_t>(j);
    __syncthreads();

    int32_t *freed = p.freed + static_cast<int64_t>(b) * p.cols;
    for (int i = tid; i < p.cols; i += kEvictThreads)
        freed[i] = i < nb - keep ? table[list[keep + i]] : -1;
    if (tid == 0) {
        p.n_freed[b] = nb - keep;
        p.out_seq[b] = L - (nb - keep) * kPage;
    }
    __syncthreads();  // the freed pages are read before any entry is overwritten
    int32_t *out_table = p.out_table + b * p.out_stride;
    for (int i0 = 0; i0 < p.cols; i0 += kEvictThreads) {
        const int i = i0 + tid;
        const int32_t v = i < keep ? table[list[i]] : -1;
        __syncthreads();
        if (i < p.cols)
            out_table[i] = v;
    }
    float *out_w = p.out_weights + static_cast<int64_t>(b) * p.kv_heads * p.cols;
    for (int h = 0; h < p.kv_heads; ++h) {
        const float *from = w + static_cast<int64_t>(h) * p.cols;
        float *to = out_w + static_cast<int64_t>(h) * p.cols;
        for (int i0 = 0; i0 < p.cols; i0 += kEvictThreads) {
            const int i = i0 + tid;
            const float v = i < keep ? from[list[i]] : 0.0f;
            __syncthreads();
            if (i < p.cols)
                to[i] = v;
        }
    }
}

}  // namespace msa

using namespace msa;

extern "C" msa_status msa_cache_accumulate(float *weights, int64_t cols, const int32_t *ids, const float *mass,
                                           const int32_t *n_rows, int batch, int q_len, int kv_heads, int sel_heads,
                                           int topk, void *workspace, size_t workspace_bytes, void *stream)
{
    if (batch < 0 || q_len < 1 || kv_heads < 1 || sel_heads < 1 || topk < 1 || cols < 1 || kv_heads % sel_heads ||
        !weights || !ids || !mass || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return MSA_ERR_INVALID_ARG;
    if (batch > MSA_MAX_BATCH || topk > MSA_MAX_TOPK || kv_heads > 1024 || q_len > 64 || cols > (int64_t{1} << 30))
        return MSA_ERR_UNSUPPORTED;
    if (workspace_bytes < kHeaderBytes)
        return MSA_ERR_WORKSPACE_TOO_SMALL;
    if (batch == 0)
        return MSA_OK;
    const int64_t warps = static_cast<int64_t>(batch) * kv_heads;
    accumulate_kernel<<<static_cast<unsigned>((warps + 3) / 4), 128, 0, static_cast<cudaStream_t>(stream)>>>(
        weights, cols, ids, mass, n_rows, batch, q_len, kv_heads, sel_heads, topk,
        &static_cast<WorkspaceHeader *>(workspace)->fault);
    return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

extern "C" msa_status msa_cache_evict(const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                                      const float *weights, int64_t cols, int batch, int kv_heads, int max_model_len,
                                      int budget, int n_sink, int n_window, int32_t *out_table, int64_t out_stride,
                                      int32_t *out_seq_lens, float *out_weights, int32_t *out_freed,
                                      int32_t *out_n_freed, void *workspace, size_t workspace_bytes, void *stream)
{
    if (batch < 0 || kv_heads < 1 || cols < 1 || max_model_len < 1 || n_sink < 0 || n_window < 1 ||
        static_cast<int64_t>(n_sink) + n_window > budget || bt_stride < cols || out_stride < cols || !block_table ||
        !seq_lens || !weights || !out_table || !out_seq_lens || !out_weights || !out_freed || !out_n_freed ||
        !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return MSA_ERR_INVALID_ARG;
    if (batch > MSA_MAX_BATCH || kv_heads > 1024 || cols > MSA_MAX_CACHE_BLOCKS)
        return MSA_ERR_UNSUPPORTED;
    if (workspace_bytes < kHeaderBytes)
        return MSA_ERR_WORKSPACE_TOO_SMALL;
    if (batch == 0)
        return MSA_OK;
    EvictParams p;
    std::memset(&p, 0, sizeof p);
    p.table = block_table;
    p.seq_lens = seq_lens;
    p.weights = weights;
    p.out_table = out_table;
    p.out_seq = out_seq_lens;
    p.out_weights = out_weights;
    p.freed = out_freed;
    p.n_freed = out_n_freed;
    p.fault = &static_cast<WorkspaceHeader *>(workspace)->fault;
    p.bt_stride = bt_stride;
    p.out_stride = out_stride;
    p.cols = static_cast<int>(cols);
    p.kv_heads = kv_heads;
    p.seq_limit = static_cast<int>(std::min<int64_t>(max_model_len, kPage * cols));
    p.budget = budget;
    p.n_sink = n_sink;
    p.n_window = n_window;
    const size_t smem = static_cast<size_t>(cols) * 6 + 8;
    if (cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
        cudaSuccess)
        return MSA_ERR_CUDA;
    evict_kernel<<<batch, kEvictThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

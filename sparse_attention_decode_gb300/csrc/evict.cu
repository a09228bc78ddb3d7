// Eviction from the paged cache by accumulated attention weight: the weights'
// update and the choice of the pages that leave.
#include <algorithm>

#include "attn_ptx.cuh"
#include "host_util.cuh"
#include "keys.cuh"
#include "layout.cuh"

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
    griddep_launch_dependents();  // an eviction that follows may take its place
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
    int apart;  // the outputs are not the inputs
};

// A block's key, ordered as its weight: NaN lowest, then -inf .. inf, pinned blocks highest.
__device__ __forceinline__ uint32_t evict_key(float w)
{
    return w != w ? 0u : float_order_bits(w == 0.0f ? 0.0f : w);
}

// Block sums W[j] = ((w_0 + w_1) + ..)[j] of N consecutive blocks, the loads of four heads at a time in flight.
template <int N>
__device__ __forceinline__ void block_sums(const float *w, int64_t cols, int heads, int j, float (&sum)[N])
{
    for (int h0 = 0; h0 < heads; h0 += 4) {
        float v[4][N];
#pragma unroll
        for (int h = 0; h < 4; ++h)
            if (h0 + h < heads) {
                const float *at = w + (h0 + h) * cols + j;
                if (N == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(at);
                    v[h][0] = x.x, v[h][1 % N] = x.y, v[h][2 % N] = x.z, v[h][3 % N] = x.w;
                } else {
                    v[h][0] = *at;
                }
            }
#pragma unroll
        for (int h = 0; h < 4; ++h)
            if (h0 + h < heads)
#pragma unroll
                for (int k = 0; k < N; ++k)
                    sum[k] = h0 + h == 0 ? v[h][k] : sum[k] + v[h][k];
    }
}

// One CTA per request.  Keys in shared memory; the budget-th largest by three
// radix passes of 11, 11 and 10 bits, the first one's counts taken as the keys are
// made (adding up a warp's equal digits by match before they are counted was
// slower; four passes of 8 bits took 1 us more).  A warp then takes a run of
// blocks, 32 at a time by ballot: how many lie above the threshold and how many on
// it, one prefix sum over the warps, and the blocks' places follow (blocks on the
// threshold stay in index order until it is met).  Table and weights are copied in
// increasing destination order, kCopy entries a thread at a time: every read of a
// piece before its writes, and a source never lies below its destination, so
// outputs may be the inputs.  VEC: rows start on 16 bytes.  T threads, two CTAs an
// SM: 1024 for long contexts, whose rounds over the blocks are then few (with the
// first digit counted apart: 35 us against 38 with 512), 256 for short ones.
//
// Bound by latency.  256 requests x 8192 blocks x 4 heads, accumulation included: 29
// us.  By the clock, from accumulation's start: 2.3 until it has ended; then, in the
// slowest CTA (in the median one), 11 us for the keys (7), 6 for the three passes (3.6),
// 1 for the counts, 1.9 for the places, 1.7 for the freed pages and 1.1 for the copies,
// 25 in all; the launch and the end are the rest.  104 SMs carry two requests, 48 one.
// DRAM is busy for 14 % of the time, the issue slots for 36; stalls are loads (4.1 a
// issued instruction), barriers (3.8) and turns not got (3.3); 32 registers a thread
// spill 28 bytes.  What carries it are wide loads with several heads in flight and few
// barriers (with a barrier every 512 entries and a load at a time: 62 us).
// 4 x 68 blocks: 4.9.
constexpr int kCopy = 2;
constexpr int kBins = 2048;  // of a radix pass: digits of 11, 11 and 10 bits

template <bool VEC, int T>
__global__ void __launch_bounds__(T, 2) evict_kernel(const __grid_constant__ EvictParams p)
{
    constexpr int kWarps = T / 32;
    extern __shared__ uint32_t evict_smem[];
    uint32_t *keys = evict_smem;
    uint16_t *list = reinterpret_cast<uint16_t *>(keys + (p.cols + 3) / 4 * 4);  // kept blocks, then the freed ones
    __shared__ int2 hist2[kBins / 2];
    int *hist = reinterpret_cast<int *>(hist2);
    __shared__ int above_of[kWarps], ties_of[kWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int s_want;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();  // the weights of a call to accumulate just before
    const int L = p.seq_lens[b];
    const bool bad = L < 0 || L > p.seq_limit;
    if (bad && tid == 0)
        atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
    const int nb = bad ? p.cols : (L + kPage - 1) / kPage;
    const int keep = bad ? p.cols : min(nb, p.budget);
    const bool all = keep == nb;
    const float *w = p.weights + static_cast<int64_t>(b) * p.kv_heads * p.cols;
    const int32_t *table = p.table + b * p.bt_stride;

    int32_t *out_table = p.out_table + b * p.out_stride;
    float *out_w = p.out_weights + static_cast<int64_t>(b) * p.kv_heads * p.cols;
    // what lies past the kept blocks
    auto clear = [&] {
#pragma unroll 4
        for (int i = keep + tid; i < p.cols; i += T)
            out_table[i] = -1;
        for (int h = 0; h < p.kv_heads; ++h) {
            float *row = out_w + static_cast<int64_t>(h) * p.cols;
            const int first = VEC ? min(p.cols, (keep + 3) / 4 * 4) : p.cols;
#pragma unroll 4
            for (int i = keep + tid; i < first; i += T)
                row[i] = 0.0f;
#pragma unroll 4
            for (int i = first + tid * 4; i < p.cols; i += T * 4)
                *reinterpret_cast<float4 *>(row + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    };
    if (p.apart)  // beside the loads; in place, it would clear what is still to be read
        clear();

    uint32_t bound = 0;  // the key of the last block that stays
    int want = all ? 0 : keep;
    if (!all) {
        constexpr int N = VEC ? 4 : 1;
        for (int i = tid; i < kBins; i += T)
            hist[i] = 0;
        __syncthreads();
#pragma unroll 2
        for (int j = tid * N; j < nb; j += T * N) {  // VEC: a row is at least nb rounded up to 4 long
            float sum[N];
            block_sums<N>(w, p.cols, p.kv_heads, j, sum);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const uint32_t key = j + k < p.n_sink || j + k >= nb - p.n_window ? 0xffffffffu : evict_key(sum[k]);
                keys[j + k] = key;
                if (j + k < nb)
                    atomicAdd(&hist[key >> 21], 1);  // the first digit's count
            }
        }
        uint32_t mask = 0;
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            if (pass > 0) {
#pragma unroll 4
                for (int j = tid; j < nb; j += T)
                    if ((keys[j] & mask) == bound)
                        atomicAdd(&hist[(keys[j] >> shift) & (pass == 2 ? 1023 : 2047)], 1);
            }
            __syncthreads();
            // the digit, from the top, in which the want-th largest lies: thread 0 has the highest ones
            constexpr int kMine = kBins / T;
            int mine[kMine], sum = 0;
#pragma unroll
            for (int k = 0; k < kMine; k += 2) {
                const int at = (kBins - 2 - k) / 2 - tid * (kMine / 2);
                const int2 two = hist2[at];
                hist2[at] = make_int2(0, 0);  // for the next pass
                mine[k] = two.y;
                mine[k + 1] = two.x;
                sum += two.x + two.y;
            }
            int above = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, above, o);
                if (lane >= o)
                    above += y;
            }
            if (lane == 31)
                above_of[warp] = above;
            above -= sum;
            __syncthreads();
            above += __reduce_add_sync(0xffffffffu, lane < warp ? above_of[lane] : 0);
#pragma unroll
            for (int k = 0; k < kMine; ++k) {
                if (above < want && above + mine[k] >= want) {
                    s_prefix = bound | static_cast<uint32_t>(kBins - 1 - tid * kMine - k) << shift;
                    s_want = want - above;
                }
                above += mine[k];
            }
            __syncthreads();
            bound = s_prefix;
            want = s_want;  // how many of the blocks that share the digits so far stay
            mask |= (pass == 2 ? 1023u : 2047u) << shift;
        }
    }
    // a warp's run: rows of 32 blocks
    const int rows = (nb + 31) / 32, per = (rows + kWarps - 1) / kWarps;
    const int r0 = min(rows, warp * per), r1 = min(rows, r0 + per);
    int above = 0, ties = 0;
    for (int r = r0; r < r1; ++r) {
        const int j = r * 32 + lane;
        const uint32_t key = j < nb && !all ? keys[j] : 0u;
        above += __popc(__ballot_sync(0xffffffffu, j < nb && (all || key > bound)));
        ties += __popc(__ballot_sync(0xffffffffu, j < nb && !all && key == bound));
    }
    if (lane == 0) {
        above_of[warp] = above;
        ties_of[warp] = ties;
    }
    __syncthreads();
    above = __reduce_add_sync(0xffffffffu, lane < warp ? above_of[lane] : 0);  // before the warp's run
    ties = __reduce_add_sync(0xffffffffu, lane < warp ? ties_of[lane] : 0);
    for (int r = r0; r < r1; ++r) {
        const int j = r * 32 + lane;
        const uint32_t lower = (1u << lane) - 1u;
        const uint32_t key = j < nb && !all ? keys[j] : 0u;
        const uint32_t on = __ballot_sync(0xffffffffu, j < nb && !all && key == bound);
        const bool stays = j < nb && (all || key > bound || (key == bound && ties + __popc(on & lower) < want));
        const uint32_t kept = __ballot_sync(0xffffffffu, stays);
        const int at = above + min(want, ties) + __popc(kept & lower);  // kept blocks before j
        if (j < nb)
            list[stays ? at : keep + j - at] = static_cast<uint16_t>(j);
        ties += __popc(on);
        above += __popc(__ballot_sync(0xffffffffu, j < nb && (all || key > bound)));
    }
    __syncthreads();

    // Every read of a piece before its writes; the first piece's loads are under way beside those of the freed pages.
    int from[kCopy];
    int32_t page[kCopy];
    float v[4][kCopy];
    auto ask = [&](int i0, int h0) {
#pragma unroll
        for (int k = 0; k < kCopy; ++k) {
            const int i = i0 + k * T + tid;
            if (h0 == 0) {
                from[k] = i < keep ? list[i] : -1;
                page[k] = from[k] >= 0 ? table[from[k]] : -1;
            }
#pragma unroll
            for (int h = 0; h < 4; ++h)
                if (h0 + h < p.kv_heads && from[k] >= 0)
                    v[h][k] = w[static_cast<int64_t>(h0 + h) * p.cols + from[k]];
        }
    };
    ask(0, 0);
    int32_t *freed = p.freed + static_cast<int64_t>(b) * p.cols;
#pragma unroll 4
    for (int i = tid; i < p.cols; i += T)
        freed[i] = i < nb - keep ? table[list[keep + i]] : -1;
    if (tid == 0) {
        p.n_freed[b] = nb - keep;
        p.out_seq[b] = L - (nb - keep) * kPage;
    }
    for (int i0 = 0; i0 < keep; i0 += T * kCopy) {
        if (i0 > 0)
            ask(i0, 0);
        for (int h0 = 0; h0 < p.kv_heads; h0 += 4) {
            if (h0 > 0)
                ask(i0, h0);
            __syncthreads();  // what the piece and, before the first, the freed list come from is read
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int k = 0; k < kCopy; ++k)
                    if (h0 + h < p.kv_heads && from[k] >= 0)
                        out_w[static_cast<int64_t>(h0 + h) * p.cols + i0 + k * T + tid] = v[h][k];
        }
#pragma unroll
        for (int k = 0; k < kCopy; ++k)
            if (from[k] >= 0)
                out_table[i0 + k * T + tid] = page[k];
    }
    if (!p.apart) {
        __syncthreads();  // the last piece's sources are read before the rest is cleared
        clear();
    }
}

}  // namespace msa

using namespace msa;

// Keys of all blocks, then the list of their numbers.
static size_t evict_smem_bytes(int64_t cols) { return (static_cast<size_t>(cols) + 3) / 4 * 16 + static_cast<size_t>(cols) * 2; }

extern "C" msa_status msa_cache_accumulate(float *weights, int64_t cols, const int32_t *ids, const float *mass,
                                           const int32_t *n_rows, int batch, int q_len, int kv_heads, int sel_heads,
                                           int topk, void *workspace, size_t workspace_bytes, void *stream)
{
    if (batch < 0 || q_len < 1 || kv_heads < 1 || sel_heads < 1 || topk < 1 || cols < 1 || kv_heads % sel_heads)
        return MSA_ERR_INVALID_ARG;
    if (batch > 0 && (!weights || !ids || !mass || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)))
        return MSA_ERR_INVALID_ARG;
    if (batch > MSA_MAX_BATCH || topk > MSA_MAX_TOPK || kv_heads > 1024 || q_len > 64 || cols > (int64_t{1} << 30))
        return MSA_ERR_UNSUPPORTED;
    if (batch == 0)  // (an empty tensor has no address)
        return MSA_OK;
    if (workspace_bytes < kHeaderBytes)
        return MSA_ERR_WORKSPACE_TOO_SMALL;
    const int64_t warps = static_cast<int64_t>(batch) * kv_heads;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>((warps + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = static_cast<cudaStream_t>(stream);
    return cudaLaunchKernelEx(&cfg, accumulate_kernel, weights, cols, ids, mass, n_rows, batch, q_len, kv_heads, sel_heads,
                              topk, &static_cast<WorkspaceHeader *>(workspace)->fault) == cudaSuccess
               ? MSA_OK
               : MSA_ERR_CUDA;
}

extern "C" msa_status msa_cache_evict(const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                                      const float *weights, int64_t cols, int batch, int kv_heads, int max_model_len,
                                      int budget, int n_sink, int n_window, int32_t *out_table, int64_t out_stride,
                                      int32_t *out_seq_lens, float *out_weights, int32_t *out_freed,
                                      int32_t *out_n_freed, void *workspace, size_t workspace_bytes, void *stream)
{
    if (batch < 0 || kv_heads < 1 || cols < 1 || max_model_len < 1 || n_sink < 0 || n_window < 1 ||
        static_cast<int64_t>(n_sink) + n_window > budget || bt_stride < cols || out_stride < cols)
        return MSA_ERR_INVALID_ARG;
    if (batch > 0 && (!block_table || !seq_lens || !weights || !out_table || !out_seq_lens || !out_weights ||
                      !out_freed || !out_n_freed || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)))
        return MSA_ERR_INVALID_ARG;
    if (batch > MSA_MAX_BATCH || kv_heads > 1024 || cols > MSA_MAX_CACHE_BLOCKS)
        return MSA_ERR_UNSUPPORTED;
    if (batch == 0)
        return MSA_OK;
    if (workspace_bytes < kHeaderBytes)
        return MSA_ERR_WORKSPACE_TOO_SMALL;
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
    p.apart = out_table != block_table && out_weights != weights;
    const size_t smem = evict_smem_bytes(cols);
    const bool vec = cols % 4 == 0 && ((reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(out_weights)) & 15) == 0;
    const bool wide = cols > 1024;
    auto *kernel = wide ? (vec ? evict_kernel<true, 1024> : evict_kernel<false, 1024>)
                        : (vec ? evict_kernel<true, 256> : evict_kernel<false, 256>);
    // (up to 1024 blocks need 6 KiB, which is always granted)
    static std::atomic<bool> allowed[2][kMaxDevices];
    int dev = 0;
    if (wide && (cudaGetDevice(&dev) != cudaSuccess ||
                 !allow_smem(kernel, evict_smem_bytes(MSA_MAX_CACHE_BLOCKS), dev, allowed[vec])))
        return MSA_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg =
        pdl_config(dim3(batch), dim3(wide ? 1024 : 256), smem, static_cast<cudaStream_t>(stream), attr);
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

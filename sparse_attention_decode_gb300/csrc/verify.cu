// Verification of drafted tokens against the target's probabilities.
//
// With m the row's largest logit, c = log2 e / T and Z = sum 2^(c (l - m)):
// p(v) = 2^(c (l_v - m)) / Z and ln p(v) = (l_v - m) / T - ln Z.  The draw is an
// exponential race: the argmax of r(v) / e(v) over independent e ~ Exp(1) is v
// with probability r(v) / sum r, so it needs no normalised cumulative sum, and
// its argmax is the same however the vocabulary is split.
//
// What bounds it: every logit is used once for m and Z and those of one row
// once more for the draw, so the stream of logits does.  One cluster a request:
// its CTAs take slices of the vocabulary, exchange (m, Z) and the best key
// through distributed shared memory, and decide alike; one launch.
#include "host_util.cuh"
#include "keys.cuh"
#include "layout.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

#include "msa_attention.h"

namespace msa {

struct VerifyParams {
    const void *logits;
    const float *draft;
    const int32_t *tokens;
    const float *uniforms;
    const float *race;
    const float *temperature;
    const int32_t *n_draft;
    int32_t *out;
    int32_t *accepted;
    float *logprobs;
    uint32_t *fault;
    int64_t stride_b, stride_i;
    int max_draft, vocab;
};

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyRows = MSA_MAX_DRAFT + 1;
constexpr float kVLog2e = 1.4426950408889634f;

struct VerifySmem {
    float wm[kVerifyRows][kVerifyWarps], ws[kVerifyRows][kVerifyWarps];
    uint64_t wk[kVerifyRows][kVerifyWarps];
    float m[kVerifyRows], s[kVerifyRows];  // the CTA's slice of each row, read by the cluster
    uint64_t key[kVerifyRows];             // greedy: its largest logit and where
    float gm[kVerifyRows], gs[kVerifyRows];
    uint64_t gkey[kVerifyRows];
    int ok[kVerifyRows];
    float lp[kVerifyRows];
    uint64_t best[2];  // the CTA's draw: from the residual, from p
    uint64_t wbest[2][kVerifyWarps];
};

__device__ __forceinline__ uint64_t dsmem_ld_u64(uint32_t addr)
{
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float dsmem_ld_float(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t verify_cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ float logit(const float *p, int v) { return p[v]; }
__device__ __forceinline__ float logit(const uint16_t *p, int v) { return __uint_as_float(static_cast<uint32_t>(p[v]) << 16); }

// (larger value, lower index) as one key; 0: none.
__device__ __forceinline__ uint64_t value_key(float x, int v)
{
    return (static_cast<uint64_t>(float_order_bits(x == 0.0f ? 0.0f : x)) << 32) | (0xffffffffu - static_cast<uint32_t>(v));
}

__device__ __forceinline__ uint64_t warp_max(uint64_t k)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        k = umax64(k, __shfl_xor_sync(0xffffffffu, k, o));
    return k;
}

// Adds a part (m2, s2) to (m, s): sums of 2^(c (l - max)).
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2, float c)
{
    const float n = fmaxf(m, m2);
    if (n == -INFINITY)
        return;
    s = s * exp2_approx(c * (m - n)) + s2 * exp2_approx(c * (m2 - n));
    m = n;
}

template <class T>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const __grid_constant__ VerifyParams p)
{
    __shared__ VerifySmem sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = static_cast<int>(verify_cluster_size()), crank = static_cast<int>(cluster_ctarank());
    const int b = blockIdx.x / C;
    const int V = p.vocab, S = p.max_draft;
    const T *logits = static_cast<const T *>(p.logits) + b * p.stride_b;
    int n = p.n_draft ? p.n_draft[b] : S;
    if (n < 0 || n > S) {
        if (tid == 0)
            atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
        n = 0;
    }
    const float temp = p.temperature ? p.temperature[b] : 1.0f;
    const bool greedy = !(temp > 0.0f);
    const float c = greedy ? 0.0f : kVLog2e / temp;
    const int step = C * kVerifyThreads;

    // ---- each row's maximum and sum over this CTA's slice ----
    for (int i = 0; i <= n; ++i) {
        const T *row = logits + i * p.stride_i;
        float m = -INFINITY, s = 0.0f;
        uint64_t key = 0;
        for (int v = crank * kVerifyThreads + tid; v < V; v += step) {
            float x = logit(row, v);
            x = x == x ? x : -INFINITY;
            if (greedy) {
                if (x > -INFINITY)
                    key = umax64(key, value_key(x, v));
            } else if (x > m) {
                s = s * exp2_approx(c * (m - x)) + 1.0f;
                m = x;
            } else if (x > -INFINITY) {
                s += exp2_approx(c * (x - m));
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            join(m, s, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o), c);
        key = warp_max(key);
        if (lane == 0) {
            sm.wm[i][warp] = m;
            sm.ws[i][warp] = s;
            sm.wk[i][warp] = key;
        }
    }
    __syncthreads();
    if (tid <= n) {
        float m = -INFINITY, s = 0.0f;
        uint64_t key = 0;
        for (int w = 0; w < kVerifyWarps; ++w) {
            join(m, s, sm.wm[tid][w], sm.ws[tid][w], c);
            key = umax64(key, sm.wk[tid][w]);
        }
        sm.m[tid] = m;
        sm.s[tid] = s;
        sm.key[tid] = key;
    }
    __syncwarp();
    cluster_sync_all();
    // ---- every CTA: the rows' totals and the drafts' fate ----
    if (tid <= n) {
        float m = -INFINITY, s = 0.0f;
        uint64_t key = 0;
        for (int r = 0; r < C; ++r) {
            join(m, s, dsmem_ld_float(mapa_shared(smem_addr(&sm.m[tid]), r)),
                 dsmem_ld_float(mapa_shared(smem_addr(&sm.s[tid]), r)), c);
            key = umax64(key, dsmem_ld_u64(mapa_shared(smem_addr(&sm.key[tid]), r)));
        }
        sm.gm[tid] = m;
        sm.gs[tid] = s;
        sm.gkey[tid] = key;
        int ok = 0;
        float lp = 0.0f;
        if (tid < n) {
            const int x = p.tokens[static_cast<int64_t>(b) * S + tid];
            if (x < 0 || x >= V) {
                atomicOr(p.fault, MSA_FAULT_TOKEN);
            } else if (greedy) {
                ok = key != 0 && static_cast<uint32_t>(x) == 0xffffffffu - static_cast<uint32_t>(key);
            } else if (s > 0.0f) {
                const float l = logit(logits + tid * p.stride_i, x);
                const float px = l > -INFINITY ? exp2_approx(c * (l - m)) / s : 0.0f;
                const float qx = p.draft[(static_cast<int64_t>(b) * S + tid) * V + x];
                ok = p.uniforms[static_cast<int64_t>(b) * S + tid] * qx < px;
                lp = (l - m) / temp - logf(s);
            }
        }
        sm.ok[tid] = ok;
        sm.lp[tid] = lp;
    }
    __syncthreads();
    int at = 0;
    while (at < n && sm.ok[at])
        ++at;
    // ---- the drawn token ----
    const bool residual = at < n && !greedy;
    const float m = sm.gm[at], inv = sm.gs[at] > 0.0f ? 1.0f / sm.gs[at] : 0.0f;
    if (!greedy && inv > 0.0f) {
        const T *row = logits + at * p.stride_i;
        const float *q = p.draft + (static_cast<int64_t>(b) * S + at) * V;
        const float *e = p.race + static_cast<int64_t>(b) * V;
        uint64_t kr = 0, kp = 0;
        for (int v = crank * kVerifyThreads + tid; v < V; v += step) {
            const float l = logit(row, v);
            if (!(l > -INFINITY))
                continue;
            const float pv = exp2_approx(c * (l - m)) * inv;
            const float ev = e[v];
            const float a = pv / ev;
            if (a > 0.0f)
                kp = umax64(kp, value_key(a, v));
            if (residual) {
                const float r = (pv - q[v]) / ev;
                if (r > 0.0f)
                    kr = umax64(kr, value_key(r, v));
            }
        }
        kr = warp_max(kr);
        kp = warp_max(kp);
        if (lane == 0) {
            sm.wbest[0][warp] = kr;
            sm.wbest[1][warp] = kp;
        }
    } else if (lane == 0) {
        sm.wbest[0][warp] = sm.wbest[1][warp] = 0;
    }
    __syncthreads();
    if (tid < 2) {
        uint64_t k = 0;
        for (int w = 0; w < kVerifyWarps; ++w)
            k = umax64(k, sm.wbest[tid][w]);
        sm.best[tid] = k;
    }
    __syncthreads();
    cluster_sync_all();
    if (crank == 0 && warp == 0) {
        uint64_t kr = 0, kp = 0;
        for (int r = 0; r < C; ++r) {
            kr = umax64(kr, dsmem_ld_u64(mapa_shared(smem_addr(&sm.best[0]), r)));
            kp = umax64(kp, dsmem_ld_u64(mapa_shared(smem_addr(&sm.best[1]), r)));
        }
        const uint64_t k = greedy ? sm.gkey[at] : (kr ? kr : kp);
        const int x = k ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)) : -1;
        float lp = 0.0f;
        if (x >= 0 && !greedy)
            lp = (logit(logits + at * p.stride_i, x) - m) / temp - logf(sm.gs[at]);
        for (int i = lane; i <= S; i += 32) {
            const int64_t o = static_cast<int64_t>(b) * (S + 1) + i;
            p.out[o] = i < at ? p.tokens[static_cast<int64_t>(b) * S + i] : i == at ? x : -1;
            if (p.logprobs)
                p.logprobs[o] = i < at ? sm.lp[i] : i == at ? lp : 0.0f;
        }
        if (lane == 0)
            p.accepted[b] = at;
    }
    __syncwarp();
    cluster_sync_all();  // no CTA ends while its shared memory is read
}

template <class T>
static msa_status launch_verify(const VerifyParams &p, int batch, int cluster, cudaStream_t st)
{
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(batch * cluster));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T>, p) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

}  // namespace msa

using namespace msa;

extern "C" msa_status msa_verify_draft(const void *logits, int logits_bf16, int64_t logits_stride_b,
                                       int64_t logits_stride_i, const float *draft_probs, const int32_t *draft_tokens,
                                       const float *uniforms, const float *race, const float *temperature,
                                       const int32_t *n_draft, int batch, int max_draft, int vocab,
                                       int32_t *out_tokens, int32_t *out_accepted, float *out_logprobs,
                                       void *workspace, size_t workspace_bytes, void *stream)
{
    if (batch < 0 || max_draft < 0 || vocab < 1 || !logits || !race || !out_tokens || !out_accepted || !workspace ||
        (max_draft > 0 && (!draft_probs || !draft_tokens || !uniforms)) || logits_stride_i < vocab ||
        logits_stride_b < vocab || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return MSA_ERR_INVALID_ARG;
    const uintptr_t size = logits_bf16 ? 2 : 4;
    if ((reinterpret_cast<uintptr_t>(logits) & (size - 1)) ||
        ((reinterpret_cast<uintptr_t>(draft_probs) | reinterpret_cast<uintptr_t>(race)) & 3))
        return MSA_ERR_INVALID_ARG;
    if (batch > MSA_MAX_BATCH || max_draft > MSA_MAX_DRAFT || vocab > (1 << 24))
        return MSA_ERR_UNSUPPORTED;
    if (workspace_bytes < kHeaderBytes)
        return MSA_ERR_WORKSPACE_TOO_SMALL;
    if (batch == 0)
        return MSA_OK;
    VerifyParams p;
    std::memset(&p, 0, sizeof p);
    p.logits = logits;
    p.draft = draft_probs;
    p.tokens = draft_tokens;
    p.uniforms = uniforms;
    p.race = race;
    p.temperature = temperature;
    p.n_draft = n_draft;
    p.out = out_tokens;
    p.accepted = out_accepted;
    p.logprobs = out_logprobs;
    p.fault = &static_cast<WorkspaceHeader *>(workspace)->fault;
    p.stride_b = logits_stride_b;
    p.stride_i = logits_stride_i;
    p.max_draft = max_draft;
    p.vocab = vocab;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int cluster = 8;
    return logits_bf16 ? launch_verify<uint16_t>(p, batch, cluster, st) : launch_verify<float>(p, batch, cluster, st);
}

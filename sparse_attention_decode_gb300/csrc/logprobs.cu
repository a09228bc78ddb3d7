// Log probabilities of given tokens, entropy and the likeliest alternatives, one
// pass over each row of logits.
//
// Mathematics.  With c = log2 e / T, m = max l, y_v = c (l_v - m): s = sum 2^y,
// h = sum 2^y y, and
//     ln p(v) = (l_v - m) / T - ln s,   H = ln s - ln2 h / s.
// A part at maximum m joins one at n >= m by d = c (m - n): s -> 2^d s and
// h -> 2^d (h + d s).  s and h stay in fp32; y is taken no lower than -200 in h, where
// 2^y is 0 (-inf times 0 would be NaN).
//
// Alternatives.  Every warp keeps its 32 largest (logit, token) pairs so far, one a lane,
// as 64-bit keys that order equal logits by the lower token.  A logit below the n-th of
// them cannot count, so 16 logits a lane cost one comparison of their maximum, which the
// sums want anyway; the few that pass go to a buffer, and 32 of them at a time are sorted
// and merged into the list.  The first bound is the CTA's: each warp sorts the maxima of
// its lanes' first 16 logits, and the least of the warps' ceil(n / 8)-th is passed by n.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "attn_ptx.cuh"
#include "host_util.cuh"
#include "keys.cuh"
#include "layout.cuh"
#include "logits.cuh"
#include "tcgen05.cuh"

#include "msa_serving.h"

namespace msa {

struct LogprobParams {
    const void *logits;
    const int32_t *tokens;
    const float *temperature;
    float *out, *entropy, *top_out;
    int32_t *top_ids;
    uint32_t *fault;
    int64_t stride;
    int given, vocab, top_n;
    int keep;  // alternatives that are tracked: top_n, and one for a row whose temperature may ask for the largest
};

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpGroup = 16;                    // logits of a lane that share a comparison
constexpr int kLpBuffer = 31 + 32 * kLpGroup;   // candidates of a warp before they are merged

struct LogprobSmem {
    uint64_t buffer[kLpWarps][kLpBuffer];
    uint64_t list[kLpWarps][32];
    uint64_t best[32];  // the CTA's, read by the cluster
    float m[kLpWarps], s[kLpWarps], h[kLpWarps];
    float cm, cs, ch;
    float bound[kLpWarps];
    float gm, gs;
    uint64_t first;
};

struct LogSum {
    float m, s, h;
    __device__ __forceinline__ void move(float to, float c)
    {
        if (s > 0.0f) {
            const float d = (m - to) * c, f = exp2_approx(d);
            h = f * fmaf(fmaxf(d, -200.0f), s, h);
            s *= f;
        }
        m = to;
    }
    __device__ __forceinline__ void join(LogSum o, float c)
    {
        const float n = fmaxf(m, o.m);
        if (n == -INFINITY)
            return;
        move(n, c);
        o.move(n, c);
        s += o.s;
        h += o.h;
    }
};

// The same for the same parts, in whatever lanes: pairwise in lane order.
template <int LANES>
__device__ __forceinline__ void lanes_join(LogSum &r, float c)
{
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
        const LogSum other{__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o),
                           __shfl_xor_sync(0xffffffffu, r.h, o)};
        r.join(other, c);
    }
}

__device__ __forceinline__ uint64_t logit_key(float l, int v)
{
    return (static_cast<uint64_t>(float_order_bits(l == 0.0f ? 0.0f : l)) << 32) | (0xffffffffu - static_cast<uint32_t>(v));
}

__device__ __forceinline__ uint64_t sort32_desc(uint64_t v, int lane)
{
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k / 2; j >= 1; j >>= 1) {
            const uint64_t o = __shfl_xor_sync(0xffffffffu, v, j);
            const bool larger = ((lane & j) == 0) == ((lane & k) == 0);
            v = larger ? umax64(v, o) : umin64(v, o);
        }
    return v;
}

// A warp's candidates: its list, what a candidate has to exceed, and the buffer.
struct Candidates {
    uint64_t *buffer;
    uint64_t list;    // this lane's, in descending order
    uint64_t bound;   // warp-uniform
    float at_least;   // its logit
    int fill;
    __device__ __forceinline__ void raise(uint64_t to)
    {
        bound = umax64(bound, to);
        at_least = float_from_order_bits(static_cast<uint32_t>(bound >> 32));
    }
    // the first 32 candidates (or what there is) join the list
    __device__ __noinline__ void merge(int keep, int lane)
    {
        __syncwarp();
        const uint64_t mine = lane < fill ? buffer[lane] : 0;
        const uint64_t rest = 32 + lane < fill ? buffer[32 + lane] : 0;
        (void)rest;
        const uint64_t sorted = sort32_desc(mine, lane);
        list = merge_top<32>(list, __shfl_sync(0xffffffffu, sorted, 31 - lane), lane);
        raise(__shfl_sync(0xffffffffu, list, keep - 1));
        // the others move up, those that still count
        int to = 0;
        for (int i = 32; i < fill; i += 32) {
            const uint64_t k = i + lane < fill ? buffer[i + lane] : 0;
            const uint32_t stay = __ballot_sync(0xffffffffu, k > bound);
            __syncwarp();
            if (k > bound)
                buffer[to + __popc(stay & ((1u << lane) - 1u))] = k;
            to += __popc(stay);
            __syncwarp();
        }
        fill = to;
    }
    __device__ __forceinline__ void push(uint64_t key, int lane)
    {
        const uint32_t who = __ballot_sync(0xffffffffu, key > bound);
        if (key > bound)
            buffer[fill + __popc(who & ((1u << lane) - 1u))] = key;
        fill += __popc(who);
    }
};

// ALIGNED: rows start on 16 bytes; else the elements before a row's first 16-byte boundary are taken one by one, as the
// ones behind its last.
template <class T>
__global__ void __launch_bounds__(kLpThreads, 3) logprobs_kernel(const __grid_constant__ LogprobParams p)
{
    extern __shared__ uint8_t smem_raw[];
    auto &sm = *reinterpret_cast<LogprobSmem *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = static_cast<int>(cluster_nctarank()), crank = static_cast<int>(cluster_ctarank());
    const int64_t r = blockIdx.x / C;
    const int V = p.vocab, keep = p.keep;
    const T *row = static_cast<const T *>(p.logits) + r * p.stride;
    constexpr int N = Logits<T>::kVec;
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int head = min(V, skew ? N - skew : 0);  // elements before the first vector
    const int nv = (V - head) / N;
    const uint4 *vectors = reinterpret_cast<const uint4 *>(row + head);
    const float temp = p.temperature ? p.temperature[r] : 1.0f;
    const bool greedy = !(temp > 0.0f);
    const float c = greedy ? 1.0f : fminf(fmaxf(kLog2e / temp, FLT_MIN), FLT_MAX);
    // the given tokens' logits, on their way beside the row
    int token = -1;
    float given = 0.0f;
    if (crank == 0 && tid < p.given) {
        token = p.tokens[r * p.given + tid];
        if (token >= V) {
            atomicOr(p.fault, MSA_FAULT_TOKEN);
            given = -INFINITY;
        } else if (token >= 0) {
            given = Logits<T>::one(row + token);
        }
    }

    const int rank = crank * kLpThreads + tid, ranks = C * kLpThreads;
    LogSum part{-INFINITY, 0.0f, 0.0f};
    Candidates cand{sm.buffer[warp], 0, logit_key(-INFINITY, 0), -INFINITY, 0};
    if (keep == 0) {
        cand.bound = ~uint64_t{0};
        cand.at_least = INFINITY;
    }
    constexpr int kLoads = 4;
    constexpr int H = kLpGroup / N;  // vectors of a group
    constexpr uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
    uint4 qa[kLoads], qb[kLoads];
    int v0 = rank;
    auto load = [&](uint4 (&q)[kLoads], int from) {
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
            q[u] = from + u * ranks < nv ? vectors[from + u * ranks] : make_uint4(none, none, none, none);
    };
    auto work = [&](const uint4 (&q)[kLoads]) {
#pragma unroll
        for (int u0 = 0; u0 < kLoads; u0 += H) {
            float l[H][N];
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < H; ++w) {
                Logits<T>::unpack(q[u0 + w], l[w]);
#pragma unroll
                for (int e = 0; e < N; ++e)
                    top = fmaxf(top, l[w][e]);
            }
            if (__any_sync(0xffffffffu, top >= cand.at_least && top > -INFINITY)) {
#pragma unroll
                for (int w = 0; w < H; ++w)
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (__any_sync(0xffffffffu, l[w][e] >= cand.at_least))
                            cand.push(logit_key(l[w][e], head + (v0 + (u0 + w) * ranks) * N + e), lane);
                while (cand.fill >= 32)
                    cand.merge(keep, lane);
            }
            if (top > part.m)  // rarer and rarer along the row
                part.move(top, c);
            const float ref = part.m == -INFINITY ? 0.0f : part.m;
            const uint64_t c2 = pack2(c, c), r2 = pack2(-ref, -ref);
            uint64_t s2[2] = {0, 0}, h2[2] = {0, 0};
#pragma unroll
            for (int w = 0; w < H; ++w)
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    float y, z;
                    unpack2(mul2(add2(pack2(l[w][e], l[w][e + 1]), r2), c2), y, z);
                    y = fmaxf(y, -200.0f);
                    z = fmaxf(z, -200.0f);
                    const uint64_t x = pack2(exp2_approx(y), exp2_approx(z));
                    s2[(e / 2) & 1] = add2(s2[(e / 2) & 1], x);
                    h2[(e / 2) & 1] = fma2(x, pack2(y, z), h2[(e / 2) & 1]);
                }
            float a, b;
            unpack2(add2(s2[0], s2[1]), a, b);
            part.s += a + b;
            unpack2(add2(h2[0], h2[1]), a, b);
            part.h += a + b;
        }
        v0 += kLoads * ranks;
    };
    load(qa, v0);
    if (keep > 0) {
        // the first bound, from the maxima of the lanes' first vectors
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < H; ++u) {
            float l[N];
            Logits<T>::unpack(qa[u], l);
#pragma unroll
            for (int e = 0; e < N; ++e)
                top = fmaxf(top, l[e]);
        }
        const uint64_t sorted = sort32_desc(static_cast<uint64_t>(float_order_bits(top)), lane);
        const uint64_t mine = __shfl_sync(0xffffffffu, sorted, (keep + kLpWarps - 1) / kLpWarps - 1);
        if (lane == 0)
            sm.bound[warp] = float_from_order_bits(static_cast<uint32_t>(mine));
        __syncthreads();
        float least = sm.bound[0];
#pragma unroll
        for (int w = 1; w < kLpWarps; ++w)
            least = fminf(least, sm.bound[w]);
        if (least > -INFINITY)
            cand.raise(logit_key(least, 0x7fffffff) - 1);  // that logit itself still counts, at every token
    }
    // all lanes of a warp together (they vote): as far as its first lane
    const int warp0 = rank - lane;
    int w0 = warp0;
    while (w0 < nv) {
        load(qb, v0 + kLoads * ranks);
        work(qa);
        w0 += kLoads * ranks;
        if (w0 >= nv)
            break;
        load(qa, v0 + kLoads * ranks);
        work(qb);
        w0 += kLoads * ranks;
    }
    // the elements before the first vector and behind the last one: fewer than 2 N, by the last CTA's first warp
    if (crank == C - 1 && warp == 0) {
        const int tail = head + nv * N;
        const int v = lane < head ? lane : tail + lane - head;
        const float l = lane < head || v < V ? Logits<T>::one(row + v) : -INFINITY;
        part.join(LogSum{l, l > -INFINITY ? 1.0f : 0.0f, 0.0f}, c);
        if (keep > 0)
            cand.push(l > -INFINITY ? logit_key(l, v) : 0, lane);
    }
    while (cand.fill > 0)
        cand.merge(keep, lane);
    lanes_join<32>(part, c);
    if (lane == 0) {
        sm.m[warp] = part.m;
        sm.s[warp] = part.s;
        sm.h[warp] = part.h;
    }
    sm.list[warp][lane] = cand.list;
    __syncthreads();
    if (warp == 0) {
        LogSum all{-INFINITY, 0.0f, 0.0f};
        if (lane < kLpWarps)
            all = LogSum{sm.m[lane], sm.s[lane], sm.h[lane]};
        lanes_join<kLpWarps>(all, c);
        uint64_t list = cand.list;
        if (keep > 0) {
#pragma unroll 1
            for (int w = 1; w < kLpWarps; ++w)
                list = merge_top<32>(list, sm.list[w][31 - lane], lane);
        }
        sm.best[lane] = list;
        if (lane == 0) {
            sm.cm = all.m;
            sm.cs = all.s;
            sm.ch = all.h;
        }
        __syncwarp();
    }
    if (C > 1)
        cluster_sync_all();
    if (crank == 0) {
        if (warp == 0) {
            LogSum all{-INFINITY, 0.0f, 0.0f};
            if (lane < C)
                all = LogSum{dsmem_ld_f32(mapa_shared(smem_addr(&sm.cm), lane)),
                             dsmem_ld_f32(mapa_shared(smem_addr(&sm.cs), lane)),
                             dsmem_ld_f32(mapa_shared(smem_addr(&sm.ch), lane))};
            lanes_join<8>(all, c);
            all = LogSum{__shfl_sync(0xffffffffu, all.m, 0), __shfl_sync(0xffffffffu, all.s, 0),
                         __shfl_sync(0xffffffffu, all.h, 0)};
            uint64_t list = sm.best[lane];
            if (keep > 0) {
#pragma unroll 1
                for (int q = 1; q < C; ++q)
                    list = merge_top<32>(list, dsmem_ld_u64(mapa_shared(smem_addr(&sm.best[31 - lane]), q)), lane);
            }
            const bool some = all.m > -INFINITY;
            const float ln_s = some ? logf(all.s) : 0.0f;
            if (lane < p.top_n) {
                const bool is = list != 0;
                const int v = is ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(list)) : -1;
                const float l = float_from_order_bits(static_cast<uint32_t>(list >> 32));
                p.top_ids[r * p.top_n + lane] = v;
                p.top_out[r * p.top_n + lane] = !is ? -INFINITY
                                                : greedy ? (lane == 0 ? 0.0f : -INFINITY)
                                                         : (l - all.m) / temp - ln_s;
            }
            if (lane == 0) {
                if (p.entropy)
                    p.entropy[r] = some && !greedy ? fmaxf(ln_s - kLn2 * (all.h / all.s), 0.0f) : 0.0f;
                sm.gm = all.m;
                sm.gs = ln_s;
                sm.first = list;
            }
        }
        __syncthreads();
        if (tid < p.given) {
            float lp = 0.0f;
            if (token >= 0) {
                if (given == -INFINITY || sm.gm == -INFINITY)
                    lp = -INFINITY;
                else if (greedy)
                    lp = static_cast<uint32_t>(token) == 0xffffffffu - static_cast<uint32_t>(sm.first) ? 0.0f : -INFINITY;
                else
                    lp = (given - sm.gm) / temp - sm.gs;
            }
            p.out[r * p.given + tid] = lp;
        }
    }
    if (C > 1)
        cluster_sync_all();  // no CTA ends while its shared memory is read
}

template <class T>
static msa_status launch_logprobs(const LogprobParams &p, int64_t rows, int cluster, int dev, cudaStream_t st)
{
    static std::atomic<bool> allowed[kMaxDevices];
    if (!allow_smem(logprobs_kernel<T>, sizeof(LogprobSmem), dev, allowed))
        return MSA_ERR_CUDA;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = sizeof(LogprobSmem);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, p) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

}  // namespace msa

using namespace msa;

extern "C" msa_status msa_token_logprobs(const void *logits, int logits_bf16, int64_t logits_stride,
                                         const int32_t *tokens, int given, const float *temperature, int64_t rows,
                                         int vocab, int top_n, float *out_logprobs, float *out_entropy,
                                         int32_t *out_top_ids, float *out_top_logprobs, void *workspace,
                                         size_t workspace_bytes, void *stream)
{
    if (rows < 0 || vocab < 1 || given < 0 || top_n < 0 || (rows > 1 && logits_stride < vocab))
        return MSA_ERR_INVALID_ARG;
    if (rows > (int64_t{1} << 27) || vocab > (1 << 24) || given > MSA_MAX_GIVEN_TOKENS || top_n > MSA_MAX_ALTERNATIVES)
        return MSA_ERR_UNSUPPORTED;
    if (rows == 0)  // (an empty tensor has no address)
        return MSA_OK;
    if (!logits || !workspace || (given > 0 && (!tokens || !out_logprobs)) ||
        (top_n > 0 && (!out_top_ids || !out_top_logprobs)) || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
        (reinterpret_cast<uintptr_t>(logits) & (logits_bf16 ? 1 : 3)))
        return MSA_ERR_INVALID_ARG;
    if (workspace_bytes < kHeaderBytes)
        return MSA_ERR_WORKSPACE_TOO_SMALL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return MSA_ERR_CUDA;
    const int sms = device_sms(dev);
    if (sms <= 0)
        return MSA_ERR_CUDA;
    LogprobParams p;
    std::memset(&p, 0, sizeof p);
    p.logits = logits;
    p.tokens = tokens;
    p.temperature = temperature;
    p.out = out_logprobs;
    p.entropy = out_entropy;
    p.top_ids = out_top_ids;
    p.top_out = out_top_logprobs;
    p.fault = &static_cast<WorkspaceHeader *>(workspace)->fault;
    p.stride = rows > 1 ? logits_stride : 0;
    p.given = given;
    p.vocab = vocab;
    p.top_n = top_n;
    p.keep = std::max(top_n, temperature && given > 0 ? 1 : 0);
    int cluster = 8;
    while (cluster > 1 && rows * cluster > 3 * sms)
        cluster /= 2;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return logits_bf16 ? launch_logprobs<uint16_t>(p, rows, cluster, dev, st)
                       : launch_logprobs<float>(p, rows, cluster, dev, st);
}

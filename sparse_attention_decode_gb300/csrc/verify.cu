// Verification of drafted tokens against the target's probabilities.
//
// With c = log2 e / T, m = max l and Z = sum 2^(c (l - m)):
// p(v) = 2^(c (l_v - m)) / Z and ln p(v) = (c (l_v - m) - log2 Z) ln 2.  m is a logit
// itself, so the largest term is exactly 1 whatever c is: c l - c m in one fused
// operation would leave the rounding of c m in the exponent, 1e-3 for l = 30000 and
// more than an exponent holds at temperatures below 1e-7.  The draw is an
// exponential race: the argmax of r(v) / e(v) over independent e ~ Exp(1) is v
// with probability r(v) / sum r, so it needs no normalised cumulative sum, and
// its argmax is the same however the vocabulary is split.
//
// What bounds it: the stream of logits (every one is read once for m and Z, those
// of one row again for the draw).  256 requests x 163840 fp32, 3 drafts of which 1.5
// are accepted: 670 MB that have to be read and 170 of the drawn rows again, which L2
// no longer holds: 840 MB in 143 us, 0.87 of the copy rate.  Rows off 16 bytes are
// bound by their loads' shape: each thread reads its vector word by word, so that a
// warp's load touches 21 sectors where 4 would hold the data (32 x 100003 bf16: 22 us
// for 38 MB; aligned, 32 x 100000: 15.8).  One cluster a request: its CTAs take
// slices of the vocabulary in 16-byte loads, several in flight a thread, exchange
// (m, Z) and the best key through distributed shared memory and decide alike; one
// launch.  A row past the first refusal has no part in the result.  Where there
// are requests enough to fill the GPU, rows are therefore taken one at a time, each
// decided before the next is read; a few requests take all rows at once, since a
// decision (two cluster barriers) would cost more than the rows it could save.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "attn_ptx.cuh"
#include "host_util.cuh"
#include "keys.cuh"
#include "layout.cuh"
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
    int rows_a_round;  // rows summed between two decisions
};

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyRows = MSA_MAX_DRAFT + 1;

struct VerifySmem {
    float wm[kVerifyRows][kVerifyWarps], ws[kVerifyRows][kVerifyWarps];
    int wi[kVerifyRows][kVerifyWarps];
    float m[kVerifyRows], s[kVerifyRows];  // the CTA's slice of each row, read by the cluster
    int i[kVerifyRows];                    // greedy: where its largest logit lies
    float gm[kVerifyRows], gs[kVerifyRows];
    int gi[kVerifyRows];
    int x[kVerifyRows];  // the drafts: token, its logit and draft probability, the uniform number
    float lx[kVerifyRows], qx[kVerifyRows], u[kVerifyRows];
    int ok[kVerifyRows];
    float lp[kVerifyRows];
    uint64_t best[2];  // the CTA's draw: from the residual, from p
    uint64_t wbest[kVerifyWarps];
};

// Logits in 16-byte vectors; NaN counts as -inf.
template <class T>
struct Logits;
template <>
struct Logits<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float one(const float *p) { return fmaxf(*p, -INFINITY); }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&x)[4])
    {
        x[0] = fmaxf(__uint_as_float(v.x), -INFINITY);
        x[1] = fmaxf(__uint_as_float(v.y), -INFINITY);
        x[2] = fmaxf(__uint_as_float(v.z), -INFINITY);
        x[3] = fmaxf(__uint_as_float(v.w), -INFINITY);
    }
};
template <>
struct Logits<uint16_t> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float one(const uint16_t *p)
    {
        return fmaxf(__uint_as_float(static_cast<uint32_t>(*p) << 16), -INFINITY);
    }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&x)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = fmaxf(__uint_as_float(w[i] << 16), -INFINITY);
            x[2 * i + 1] = fmaxf(__uint_as_float(w[i] & 0xffff0000u), -INFINITY);
        }
    }
};

// A part of a row: m = max l and s = sum 2^(c (l - m)).  Greedy: where the largest logit first occurs.
struct RowPart {
    float m, s;
    int i;
    __device__ __forceinline__ void join(const RowPart &o, float c)
    {
        const float n = fmaxf(m, o.m);
        if (n == -INFINITY)
            return;
        i = m > o.m ? i : o.m > m ? o.i : min(i, o.i);
        s = s * exp2_approx((m - n) * c) + o.s * exp2_approx((o.m - n) * c);
        m = n;
    }
};

// The join of all lanes' parts, in lane order pairwise: the same for the same parts.
__device__ __forceinline__ void warp_join(RowPart &r, float c)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const RowPart other{__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o),
                            __shfl_xor_sync(0xffffffffu, r.i, o)};
        r.join(other, c);
    }
}

// Vector v of a row (elements [v * N, v * N + N)) wherever the row starts, so that a
// row's sums are grouped by index alone, not by address: one 16-byte load where
// every row is aligned to it, else word by word (five words that hold the eight
// 2-byte elements, shifted into place when they are used; the outer two each hold a
// byte of the vector).
template <class T, bool ALIGNED>
struct RawVec {
    uint32_t w[ALIGNED || sizeof(T) == 4 ? 4 : 5];
    __device__ __forceinline__ void load(const T *row, int v)
    {
        const uint8_t *at = reinterpret_cast<const uint8_t *>(row) + static_cast<int64_t>(v) * 16;
        if (ALIGNED) {
            const uint4 x = *reinterpret_cast<const uint4 *>(at);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
            const uint32_t odd = sizeof(T) == 4 ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 2);
            const uint32_t *word = reinterpret_cast<const uint32_t *>(at - odd);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = word[i];
            if (sizeof(T) != 4)
                w[sizeof(w) / 4 - 1] = odd ? word[4] : 0u;
        }
    }
    __device__ __forceinline__ uint4 get(const T *row) const
    {
        if (ALIGNED || sizeof(T) == 4)
            return make_uint4(w[0], w[1], w[2], w[3]);
        const uint32_t bits = (reinterpret_cast<uintptr_t>(row) & 2) * 8;
        return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                          __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[sizeof(w) / 4 - 1], bits));
    }
};

constexpr int kBatch = 4;  // vectors a thread loads at a time

// A batch of a thread's share of a row: vectors v0 + u * ranks.
template <class T, bool ALIGNED>
__device__ __forceinline__ void load_batch(RawVec<T, ALIGNED> (&q)[kBatch], const T *row, int nv, int v0, int ranks)
{
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
        const int v = v0 + u * ranks;
        if (v < nv)
            q[u].load(row, v);
    }
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One CTA's best of max(p - q, 0) / e (Q) or p / e over its slice, as (value, lowest index); 0: none.
// p = 2^(c (l - m)) * inv.
template <bool ALIGNED, class T, bool Q>
__device__ __forceinline__ uint64_t race_part(const T *row, const float *q, const float *e, int V, int rank, int ranks,
                                              float m, float inv, float c)
{
    constexpr int N = Logits<T>::kVec;
    float best = 0.0f;
    int at = -1;
    auto value = [&](float l, float qv, float ev) {
        const float pv = exp2_approx((l - m) * c) * inv;
        return (Q ? pv - qv : pv) * rcp_approx(ev);
    };
    const int nv = V / N;
#pragma unroll 2
    for (int v = rank; v < nv; v += ranks) {
        float l[N], r[N];
        RawVec<T, ALIGNED> lv;
        RawVec<float, ALIGNED> ev[N / 4], qv[N / 4];
        lv.load(row, v);
#pragma unroll
        for (int k = 0; k < N / 4; ++k) {
            ev[k].load(e, v * (N / 4) + k);
            if (Q)
                qv[k].load(q, v * (N / 4) + k);
        }
        Logits<T>::unpack(lv.get(row), l);
#pragma unroll
        for (int k = 0; k < N; ++k)
            r[k] = value(l[k], Q ? __uint_as_float(qv[k / 4].w[k & 3]) : 0.0f, __uint_as_float(ev[k / 4].w[k & 3]));
        float top = r[0];
#pragma unroll
        for (int k = 1; k < N; ++k)
            top = fmaxf(top, r[k]);
        if (top > best) {  // rarer and rarer; a thread's indices grow
            best = top;
#pragma unroll
            for (int k = N - 1; k >= 0; --k)
                at = r[k] == top ? v * N + k : at;
        }
    }
    const int v = nv * N + rank;
    if (v < V) {
        const float r = value(Logits<T>::one(row + v), Q ? q[v] : 0.0f, e[v]);
        if (r > best) {
            best = r;
            at = v;
        }
    }
    return at < 0 ? 0 : (static_cast<uint64_t>(__float_as_uint(best)) << 32) | (0xffffffffu - static_cast<uint32_t>(at));
}

__device__ __forceinline__ uint64_t warp_max(uint64_t k)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        k = umax64(k, __shfl_xor_sync(0xffffffffu, k, o));
    return k;
}

__device__ __forceinline__ void async_word(void *dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

// ALIGNED: every row of every input starts on 16 bytes.  BLOCKS: CTAs an SM.  3, without
// spills, where the work of one thread sets the time: few requests, and many whose bf16
// rows are shifted into place (32 x 100003 bf16: 22 us, 29 with 4; 120: 67 and 81; 256:
// 107 and 133).  4 (64 registers, some spills) where the number of loads in flight does:
// many requests otherwise (256 x 163840 fp32: 143 us, 175 with 3; 256 x 100003 fp32: 118
// and 128; 256 x 100000 bf16: 67 and 81).
template <class T, bool ALIGNED, int BLOCKS>
__global__ void __launch_bounds__(kVerifyThreads, BLOCKS) verify_kernel(const __grid_constant__ VerifyParams p)
{
    __shared__ VerifySmem sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = static_cast<int>(cluster_nctarank()), crank = static_cast<int>(cluster_ctarank());
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
    // positive and finite, so that c times a difference of logits is 0 or of its sign, also at the ends of the range
    const float c = greedy ? 1.0f : fminf(fmaxf(kLog2e / temp, FLT_MIN), FLT_MAX);
    constexpr int N = Logits<T>::kVec;
    const int nv = V / N;
    // the drafts' tokens and numbers, on their way to shared memory beside the first rows
    if (tid < n) {
        async_word(&sm.x[tid], p.tokens + static_cast<int64_t>(b) * S + tid);
        async_word(&sm.u[tid], p.uniforms + static_cast<int64_t>(b) * S + tid);
    }

    int at = 0;  // the row that the last token comes from: the first refusal, or n
    for (int i0 = 0; i0 <= n; i0 += p.rows_a_round) {
        const int i1 = min(n + 1, i0 + p.rows_a_round), R = i1 - i0;
        // several CTAs to a row, or several rows to a CTA; neighbouring threads read neighbouring vectors
        const bool share = R <= C;
        const int first = i0 + (share ? crank * R / C : crank);
        const int c0 = share ? ((first - i0) * C + R - 1) / R : crank;
        const int c1 = share ? ((first - i0 + 1) * C + R - 1) / R : crank + 1;
        const int rank = (crank - c0) * kVerifyThreads + tid, ranks = (c1 - c0) * kVerifyThreads;
        for (int i = i0 + tid; i < i1; i += kVerifyThreads) {  // rows of other CTAs: an empty part
            sm.m[i] = -INFINITY;
            sm.s[i] = 0.0f;
            sm.i[i] = 0x7fffffff;
        }
        for (int i = first; i < (share ? first + 1 : i1); i += C) {
            const T *row = logits + i * p.stride_i;
            RowPart part{-INFINITY, 0.0f, 0x7fffffff};
            int v0 = rank;  // the thread's first vector of the batch at hand
            auto work = [&](const RawVec<T, ALIGNED> (&q)[kBatch]) {
                constexpr uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
                constexpr int H = 16 / N;  // vectors of 16 elements, which share a maximum and a branch
#pragma unroll
                for (int u0 = 0; u0 < kBatch; u0 += H) {
                    float l[H][N];
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < H; ++w) {
                        const bool have = v0 + (u0 + w) * ranks < nv;
                        Logits<T>::unpack(have ? q[u0 + w].get(row) : make_uint4(none, none, none, none), l[w]);
#pragma unroll
                        for (int e = 0; e < N; ++e)
                            top = fmaxf(top, l[w][e]);
                    }
                    if (top > part.m) {  // rarer and rarer along the row
                        if (greedy) {
#pragma unroll
                            for (int w = H - 1; w >= 0; --w)
#pragma unroll
                                for (int e = N - 1; e >= 0; --e)
                                    part.i = l[w][e] == top ? (v0 + (u0 + w) * ranks) * N + e : part.i;
                        }
                        part.s *= exp2_approx((part.m - top) * c);
                        part.m = top;
                    }
                    if (!greedy) {
                        const float ref = part.m == -INFINITY ? 0.0f : part.m;
                        const uint64_t c2 = pack2(c, c), r2 = pack2(-ref, -ref);
                        float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int w = 0; w < H; ++w)
#pragma unroll
                            for (int e = 0; e < N; e += 2) {
                                float y, z;
                                unpack2(mul2(add2(pack2(l[w][e], l[w][e + 1]), r2), c2), y, z);
                                a[e & 3] += exp2_approx(y);
                                a[(e + 1) & 3] += exp2_approx(z);
                            }
                        part.s += (a[0] + a[1]) + (a[2] + a[3]);
                    }
                }
                v0 += kBatch * ranks;
            };
            // the next batch in flight while one is summed
            RawVec<T, ALIGNED> qa[kBatch], qb[kBatch];
            load_batch(qa, row, nv, v0, ranks);
            while (v0 < nv) {
                load_batch(qb, row, nv, v0 + kBatch * ranks, ranks);
                work(qa);
                if (v0 >= nv)
                    break;
                load_batch(qa, row, nv, v0 + kBatch * ranks, ranks);
                work(qb);
            }
            const int v = nv * N + rank;  // the elements that fill no vector
            if (v < V) {
                const float y = Logits<T>::one(row + v);
                part.join(RowPart{y, y > -INFINITY ? 1.0f : 0.0f, v}, c);
            }
            warp_join(part, c);
            if (lane == 0) {
                sm.wm[i][warp] = part.m;
                sm.ws[i][warp] = part.s;
                sm.wi[i][warp] = part.i;
            }
        }
        if (i0 == 0 && tid < n) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            const int x = sm.x[tid];
            const bool ok = x >= 0 && x < V;
            if (!ok)
                atomicOr(p.fault, MSA_FAULT_TOKEN);
            sm.lx[tid] = ok ? Logits<T>::one(logits + tid * p.stride_i + x) : 0.0f;
            sm.qx[tid] = ok ? p.draft[(static_cast<int64_t>(b) * S + tid) * V + x] : 0.0f;
            sm.x[tid] = ok ? x : -1;
        }
        __syncthreads();
        for (int r = first + C * warp; r < (share ? first + 1 : i1); r += C * kVerifyWarps) {
            RowPart q{-INFINITY, 0.0f, 0x7fffffff};
            if (lane < kVerifyWarps)
                q = RowPart{sm.wm[r][lane], sm.ws[r][lane], sm.wi[r][lane]};
            warp_join(q, c);
            if (lane == 0) {
                sm.m[r] = q.m;
                sm.s[r] = q.s;
                sm.i[r] = q.i;
            }
        }
        __syncwarp();
        cluster_sync_all();
        // every CTA: the rows' totals and the drafts' fate
        for (int r = i0 + warp; r < i1; r += kVerifyWarps) {
            RowPart q{-INFINITY, 0.0f, 0x7fffffff};
            if (lane < C)
                q = RowPart{dsmem_ld_f32(mapa_shared(smem_addr(&sm.m[r]), lane)),
                            dsmem_ld_f32(mapa_shared(smem_addr(&sm.s[r]), lane)),
                            dsmem_ld_s32(mapa_shared(smem_addr(&sm.i[r]), lane))};
            warp_join(q, c);
            if (lane == 0) {
                int ok = 0;
                float lp = 0.0f;
                if (r < n && sm.x[r] >= 0 && q.m > -INFINITY) {
                    if (greedy) {
                        ok = sm.x[r] == q.i;
                    } else {
                        const float e = (sm.lx[r] - q.m) * c;
                        ok = sm.u[r] * sm.qx[r] < exp2_approx(e) / q.s;
                        lp = (e - log2f(q.s)) * kLn2;
                    }
                }
                sm.gm[r] = q.m;
                sm.gs[r] = q.s;
                sm.gi[r] = q.m > -INFINITY ? q.i : -1;
                sm.ok[r] = ok;
                sm.lp[r] = lp;
            }
        }
        __syncthreads();
        while (at < i1 && at < n && sm.ok[at])
            ++at;
        if (at < i1)  // refused, or the row behind the last draft
            break;
    }
    // ---- the drawn token ----
    const int rank = crank * kVerifyThreads + tid, ranks = C * kVerifyThreads;
    const bool draws = !greedy && sm.gm[at] > -INFINITY;
    bool residual = draws && at < n;
    const float m0 = sm.gm[at], inv = draws ? 1.0f / sm.gs[at] : 0.0f;
    const T *row = logits + at * p.stride_i;
    uint64_t key = 0;
    for (int round = 0; draws && round < 2; ++round) {
        const float *q = residual ? p.draft + (static_cast<int64_t>(b) * S + at) * V : nullptr;
        const float *e = p.race + static_cast<int64_t>(b) * V;
        uint64_t k = warp_max(residual ? race_part<ALIGNED, T, true>(row, q, e, V, rank, ranks, m0, inv, c)
                                       : race_part<ALIGNED, T, false>(row, nullptr, e, V, rank, ranks, m0, inv, c));
        if (lane == 0)
            sm.wbest[warp] = k;
        __syncthreads();
        if (warp == 0) {
            k = warp_max(lane < kVerifyWarps ? sm.wbest[lane] : 0);
            if (lane == 0)
                sm.best[round] = k;
        }
        __syncwarp();
        cluster_sync_all();
        key = warp_max(lane < C ? dsmem_ld_u64(mapa_shared(smem_addr(&sm.best[round]), lane)) : 0);
        if (key || !residual)
            break;
        residual = false;  // p <= q everywhere: the draw is from p
    }
    if (crank == 0 && warp == 0) {
        const int x = greedy ? sm.gi[at] : key ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
        float lp = 0.0f;
        if (x >= 0 && !greedy)
            lp = ((Logits<T>::one(row + x) - m0) * c - log2f(sm.gs[at])) * kLn2;
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

template <class T, bool ALIGNED, int BLOCKS>
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
    return cudaLaunchKernelEx(&cfg, verify_kernel<T, ALIGNED, BLOCKS>, p) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
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
    if (batch < 0 || max_draft < 0 || vocab < 1 || logits_stride_i < vocab || logits_stride_b < vocab)
        return MSA_ERR_INVALID_ARG;
    if (batch > 0 && (!logits || !race || !out_tokens || !out_accepted || !workspace ||
                      (max_draft > 0 && (!draft_probs || !draft_tokens || !uniforms)) ||
                      (reinterpret_cast<uintptr_t>(workspace) & 255)))
        return MSA_ERR_INVALID_ARG;
    const uintptr_t size = logits_bf16 ? 2 : 4;
    if ((reinterpret_cast<uintptr_t>(logits) & (size - 1)) ||
        ((reinterpret_cast<uintptr_t>(draft_probs) | reinterpret_cast<uintptr_t>(race)) & 3))
        return MSA_ERR_INVALID_ARG;
    if (batch > MSA_MAX_BATCH || max_draft > MSA_MAX_DRAFT || vocab > (1 << 24))
        return MSA_ERR_UNSUPPORTED;
    if (batch == 0)  // (an empty tensor has no address)
        return MSA_OK;
    if (workspace_bytes < kHeaderBytes)
        return MSA_ERR_WORKSPACE_TOO_SMALL;
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
    // Few requests: clusters of 8, all rows at once (24 x 131072 fp32, 3 drafts: 23.9 us, against 41.2 with 4 CTAs
    // and a row at a time).  Many: a row at a time and smaller clusters, which wait less for one another (128: 67
    // against 80 us; 192: 104 with 2 CTAs, 105 with 4, 110 with 8).
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return MSA_ERR_CUDA;
    const int sms = device_sms(dev);
    if (sms <= 0)
        return MSA_ERR_CUDA;
    const bool many = batch * 8 > 5 * sms;
    const int cluster = !many ? 8 : batch <= sms ? 4 : 2;
    p.rows_a_round = many ? 1 : max_draft + 1;
    const bool aligned = ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(draft_probs) |
                           reinterpret_cast<uintptr_t>(race) | static_cast<uintptr_t>(logits_stride_b) * size |
                           static_cast<uintptr_t>(logits_stride_i) * size | static_cast<uintptr_t>(vocab) * 4) &
                          15) == 0;
    const auto run = [&](auto one) {
        using T = decltype(one);
        constexpr int kShifted = sizeof(T) == 2 ? 3 : 4;
        if (many)
            return aligned ? launch_verify<T, true, 4>(p, batch, cluster, st)
                           : launch_verify<T, false, kShifted>(p, batch, cluster, st);
        return aligned ? launch_verify<T, true, 3>(p, batch, cluster, st)
                       : launch_verify<T, false, 3>(p, batch, cluster, st);
    };
    return logits_bf16 ? run(uint16_t{}) : run(float{});
}

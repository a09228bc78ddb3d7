// Log probabilities of given tokens, entropy and the likeliest alternatives, one
// pass over each row of logits.
//
// Mathematics.  With c = log2 e / T, a reference m near the largest logit, y_v = c (l_v - m):
// s = sum 2^y, h = sum 2^y y, and
//     ln p(v) = (l_v - m) / T - ln s,   H = ln s - ln2 h / s.
// A part at reference m moves to n by d = c (m - n): s -> 2^d s and h -> 2^d (h + d s).  s
// and h stay in fp32.  y is one fused operation, c l - M with M = c m rounded; what M is
// off by, d = c m - M, is the same for all terms of a part, known exactly, and taken
// out of its sums: 2^-d s', 2^-d (h' - d s').  (Where |c m| passes 2^12, y is c (l - m).)
// y is taken no lower than -200 (bf16: l no lower than 400 / c below m, two logits an
// instruction), where 2^y is 0: -inf times 0 would be NaN.  A warp's reference is the
// largest logit of its first ones, and moves when one passes it by 2^8.
//
// What bounds it: the stream of logits (1024 x 163840 fp32, 671 MB, one alternative: 116 us,
// 5.8 TB/s; bf16 the instructions, 0.6 of the issue slots: 79 us).  Slices of a row come into a ring in
// shared memory by bulk copies, so that a thread's registers hold one group of 16 logits and
// the loop is short: 4.5 instructions a bf16 logit.  Where a CTA has one slice of a row, what
// follows one after the other: 128 x 100003 bf16, 20 alternatives, take 14.7 us, of which the
// stream is 4; first stage and bound 2, the others 6, noted places 0.7, order and sums in the
// CTA 1.9, clusters' barrier and lists 1.2, what is left 1.
//
// Alternatives.  16 logits a lane cost one comparison of their maximum with a bound that n
// logits of the CTA are known to reach; where it passes, the lane's place is noted (a
// few instructions: looking for the logit at once cost as much as the sums).  At the row's
// end the noted places are read again, with the bound as it is then, and the few logits
// that reach it become 64-bit keys that order equal logits by the lower token; a key's
// place is the number of larger ones.  The bound comes from the lanes' running maxima,
// which are logits of their own: the n-th of the warps' four largest each.  It is brought
// up to date after stages 1, 5, 13, 29, .., without a barrier: old numbers make a bound as
// well.
// (Where logits rise along a row, every place is noted for a while: 64 of them are then
// read at once, and 32 keys at a time sorted and merged into a list of the warp's 32
// largest, which raises the bound.)
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "attn_common.cuh"
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
    int64_t stride, rows;
    int given, vocab, top_n;
    int keep;  // alternatives that are tracked: top_n, and one for a row whose temperature may ask for the largest
};

constexpr int kLpThreads = 256;  // eight warps that sum; a ninth issues the copies
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpGroup = 16;     // logits of a lane that share a comparison
constexpr int kLpBlocks = 2;     // CTAs an SM: with 3, and 72 registers, the sums' loop spills (1024 x 163840 bf16 90 us, 71)
constexpr int kLpStages = 5;     // 160 KB an SM under way; 6 leave less of L1 to the noted places (20 alternatives: 142 us, 135)
constexpr int kLpVectors = 1024;  // of a stage: 16 KiB
constexpr int kLpBuffer = 64;    // keys of a warp: 32 that wait, and one a lane
constexpr int kLpNoted = 128;    // places of a warp: 64 that wait, and a stage's

struct LogprobSmem {
    uint4 ring[kLpStages][kLpVectors];
    uint64_t full[kLpStages], empty[kLpStages];
    uint64_t buffer[kLpWarps][kLpBuffer];
    uint64_t list[kLpWarps][32];         // a warp's largest in order, where its buffer has been full
    int noted[kLpWarps][kLpNoted];       // first vectors of groups that hold a candidate
    uint64_t all[kLpWarps * kLpBuffer];  // the CTA's candidates
    uint64_t reach[kLpWarps];            // the warps' bounds
    uint64_t best[32];                   // the CTA's largest, in order, read by the cluster
    uint32_t tops[32];                   // the warps' four largest lane maxima, in the order of the keys
    float m[kLpWarps], s[kLpWarps], h[kLpWarps];
    float cm, cs, ch;  // the CTA's sums
    float gm, gs;
    uint64_t first;
    int count;
    int abort_flag;
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

// All lanes' parts in every lane: the same for the same parts, whatever lanes they are in.
__device__ __forceinline__ LogSum lanes_join(LogSum r, float c)
{
    const float m = float_from_order_bits(__reduce_max_sync(0xffffffffu, float_order_bits(r.m)));
    if (m > -INFINITY)
        r.move(m, c);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
        r.h += __shfl_xor_sync(0xffffffffu, r.h, o);
    }
    r.m = m;
    return r;
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

__device__ __forceinline__ uint32_t sort32_desc(uint32_t v, int lane)
{
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k / 2; j >= 1; j >>= 1) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, v, j);
            v = ((lane & j) == 0) == ((lane & k) == 0) ? max(v, o) : min(v, o);
        }
    return v;
}

// The lanes' four largest values to tops[0..3].
__device__ __forceinline__ void lanes_tops(uint32_t v, volatile uint32_t *tops, int lane)
{
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, v);
        mine = lane == i ? top : mine;
        if (lane == __ffs(__ballot_sync(0xffffffffu, v == top)) - 1)
            v = 0;
    }
    if (lane < 4)
        tops[lane] = mine;
}

// A warp's candidates: what a key has to exceed, and how many wait in the buffer.  (The list stays in shared memory: the
// sums' loop has no registers for it.)
struct Candidates {
    uint64_t bound;
    float at_least;  // its logit
    int fill;
    bool listed;
    __device__ __forceinline__ void raise(uint64_t to)
    {
        bound = umax64(bound, to);
        at_least = float_from_order_bits(static_cast<uint32_t>(bound >> 32));
    }
    // every logit from this one on still counts, at every token
    __device__ __forceinline__ void raise_to(uint32_t order)
    {
        const float l = float_from_order_bits(order);
        if (l > -INFINITY)
            raise(logit_key(l, 0x7fffffff) - 1);
    }
    __device__ __forceinline__ void push(uint64_t *buffer, uint64_t key, int lane)
    {
        const uint32_t who = __ballot_sync(0xffffffffu, key > bound);
        if (key > bound)
            buffer[fill + __popc(who & ((1u << lane) - 1u))] = key;
        fill += __popc(who);
    }
};

// The first 32 candidates (or what there is) join the list.
__device__ __noinline__ Candidates merge_candidates(Candidates c, uint64_t *buffer, uint64_t *list, int keep, int lane)
{
    __syncwarp();
    const uint64_t sorted = sort32_desc(lane < c.fill ? buffer[lane] : uint64_t{0}, lane);
    const uint64_t mine = merge_top<32>(c.listed ? list[lane] : 0, __shfl_sync(0xffffffffu, sorted, 31 - lane), lane);
    list[lane] = mine;
    c.listed = true;
    c.raise(__shfl_sync(0xffffffffu, mine, keep - 1));
    // the others move up, those that still count
    int to = 0;
    for (int i = 32; i < c.fill; i += 32) {
        const uint64_t k = i + lane < c.fill ? buffer[i + lane] : 0;
        const uint32_t stay = __ballot_sync(0xffffffffu, k > c.bound);
        __syncwarp();
        if (k > c.bound)
            buffer[to + __popc(stay & ((1u << lane) - 1u))] = k;
        to += __popc(stay);
        __syncwarp();
    }
    c.fill = to;
    return c;
}

// Logits as they are: NaN passes no comparison, and its term of the sums is taken at the floor of y, where it is 0.
__device__ __forceinline__ void raw_logits(const uint4 &v, float (&x)[4])
{
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void raw_logits(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// 16 logits a lane, of which some reach the bound: `stride` tokens from one vector of N to the next.
template <int N>
__device__ __forceinline__ Candidates push_group(Candidates c, uint64_t *buffer, uint64_t *list, int keep, int lane, int v,
                                                 int stride, uint4 a, uint4 b, uint4 d, uint4 e)
{
    float x[16 / N][N];
    const uint4 in[4] = {a, b, d, e};
#pragma unroll
    for (int w = 0; w < 16 / N; ++w)
        raw_logits(in[w], x[w]);
    for (;;) {  // each lane its largest, as long as one has one that counts
        float top = -INFINITY;
        int at = 0;
#pragma unroll
        for (int i = 15; i >= 0; --i) {
            const bool larger = x[i / N][i % N] >= top;  // (the first of equal ones; NaN never)
            top = larger ? x[i / N][i % N] : top;
            at = larger ? i : at;
        }
        const bool counts = top >= c.at_least && top > -INFINITY;
        if (!__any_sync(0xffffffffu, counts))
            break;
        c.push(buffer, counts ? logit_key(top, v + at / N * stride + at % N) : 0, lane);
        if (c.fill >= 32)
            c = merge_candidates(c, buffer, list, keep, lane);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i / N][i % N] = i == at ? -INFINITY : x[i / N][i % N];
    }
    return c;
}

// The noted places' logits: those that reach the bound by now become keys.  `row`: the row's first vector, of `to`.
template <int N>
__device__ __noinline__ Candidates read_noted(Candidates c, uint64_t *buffer, uint64_t *list, const int *noted, int count, int keep, int lane,
                                              const uint4 *row, int to, int head)
{
    constexpr int H = kLpGroup / N;
    constexpr uint32_t none = N == 4 ? 0xff800000u : 0xff80ff80u;
    __syncwarp();
    for (int i = 0; i < count; i += 32) {
        const int v = i + lane < count ? noted[i + lane] : to;
        uint4 q[4];
#pragma unroll
        for (int w = 0; w < 4; ++w)
            q[w] = w < H && v + w * kLpThreads < to ? row[v + w * kLpThreads] : make_uint4(none, none, none, none);
        c = push_group<N>(c, buffer, list, keep, lane, head + v * N, kLpThreads * N, q[0], q[1], q[2], q[3]);
    }
    __syncwarp();
    return c;
}

// The larger of two bf16 each; of a NaN and a number the number.
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The largest of some vectors' logits; NaN where all are.
template <int N, int H>
__device__ __forceinline__ float top_of(const uint4 (&q)[H])
{
    if (N == 8) {
        uint32_t m = bf16x2_max(bf16x2_max(q[0].x, q[0].y), bf16x2_max(q[0].z, q[0].w));
#pragma unroll
        for (int i = 1; i < H; ++i)
            m = bf16x2_max(m, bf16x2_max(bf16x2_max(q[i].x, q[i].y), bf16x2_max(q[i].z, q[i].w)));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < H; ++i)
        top = max3(top, max3(__uint_as_float(q[i].x), __uint_as_float(q[i].y), __uint_as_float(q[i].z)), __uint_as_float(q[i].w));
    return top;
}

__device__ __forceinline__ void sums_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kLpThreads) : "memory"); }

// A cluster a row at a time, each CTA a slice of it.  Rows may start anywhere: the logits before a row's first 16-byte
// boundary are taken one by one, as the ones behind its last.
template <class T>
__global__ void __launch_bounds__(kLpThreads + 32, kLpBlocks) logprobs_kernel(const __grid_constant__ LogprobParams p)
{
    extern __shared__ uint8_t smem_raw[];
    auto &sm = *reinterpret_cast<LogprobSmem *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int C = static_cast<int>(cluster_nctarank()), crank = static_cast<int>(cluster_ctarank());
    const int64_t r0 = blockIdx.x / C, clusters = gridDim.x / C;
    const int V = p.vocab, keep = p.keep;
    constexpr int N = Logits<T>::kVec;
    constexpr int H = kLpGroup / N;  // vectors of a group
    if (tid == 0) {
        for (int s = 0; s < kLpStages; ++s) {
            mbar_init(smem_addr(&sm.full[s]), 1);
            mbar_init(smem_addr(&sm.empty[s]), kLpWarps);
        }
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    // row r: elements before its first vector, and this CTA's vectors [from, to)
    struct Slice {
        const T *row;
        int head, from, to, nv;
    };
    auto slice = [&](int64_t r) {
        Slice x;
        x.row = static_cast<const T *>(p.logits) + r * p.stride;
        const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(x.row) & 15) / sizeof(T));
        x.head = min(V, skew ? N - skew : 0);
        x.nv = (V - x.head) / N;
        const int each = (x.nv + C - 1) / C;
        x.from = min(x.nv, crank * each);
        x.to = min(x.nv, x.from + each);
        return x;
    };
    uint32_t it = 0;  // stages so far
    if (warp == kLpWarps) {
        bool alive = true;
        for (int64_t r = r0; r < p.rows && alive; r += clusters) {
            const Slice x = slice(r);
            for (int v = x.from; v < x.to && alive; v += kLpVectors, ++it) {
                const int s = static_cast<int>(it % kLpStages);
                if (it >= kLpStages)
                    alive = attn_wait(&sm.abort_flag, p.fault, smem_addr(&sm.empty[s]), (it / kLpStages + 1) & 1, 0);
                if (alive && lane == 0) {
                    const uint32_t bytes = static_cast<uint32_t>(min(kLpVectors, x.to - v)) * 16u, bar = smem_addr(&sm.full[s]);
                    mbar_arrive_expect_tx(bar, bytes);
                    bulk_load(smem_addr(sm.ring[s]), reinterpret_cast<const uint4 *>(x.row + x.head) + v, bytes, bar);
                }
                __syncwarp();
            }
        }
        // the copies in flight land before the CTA may end
        const uint32_t issued = alive ? it : it - 1;
        for (uint32_t j = issued >= kLpStages ? issued - kLpStages : 0; j < issued; ++j)
            mbar_wait(smem_addr(&sm.full[j % kLpStages]), (j / kLpStages) & 1);
        if (C > 1) {  // a cluster of several has one row: its barriers
            cluster_sync_all();
            cluster_sync_all();
        }
        return;
    }
    uint64_t *buffer = sm.buffer[warp];
    for (int64_t r = r0; r < p.rows; r += clusters) {
        const Slice x = slice(r);
        const float temp = p.temperature ? p.temperature[r] : 1.0f;
        const bool greedy = !(temp > 0.0f);
        const float c = greedy ? 1.0f : fminf(fmaxf(kLog2e / temp, FLT_MIN), FLT_MAX);
        const float lag = 8.0f / c, floor_at = 400.0f / c;
        // the given tokens' logits, on their way beside the row
        int token = -1;
        float given = 0.0f;
        if (crank == 0 && tid < p.given) {
            token = p.tokens[r * p.given + tid];
            if (token >= V) {
                atomicOr(p.fault, MSA_FAULT_TOKEN);
                given = -INFINITY;
            } else if (token >= 0) {
                given = Logits<T>::one(x.row + token);
            }
        }
        if (tid == 0)
            sm.count = 0;
        if (tid < 32)
            sm.best[tid] = 0;
        LogSum part{-INFINITY, 0.0f, 0.0f};
        Candidates cand{logit_key(-INFINITY, 0), -INFINITY, 0, false};
        if (keep == 0) {
            cand.bound = ~uint64_t{0};
            cand.at_least = INFINITY;
        }
        // of the warp's reference part.m: -M, what M is off by, 2^-off, the least logit that is told apart (two of them),
        // and the one that moves it
        float minus_m = 0.0f, off = 0.0f, undo = 1.0f, moves = -INFINITY;
        uint32_t least2 = 0xff80ff80u;
        bool far = true;  // (no reference yet)
        float run = -INFINITY;  // the lane's largest logit
        int stage = 0, noted = 0, update = 0;
        const uint4 *vectors = reinterpret_cast<const uint4 *>(x.row + x.head);
        // the CTA's bound by the lanes' largest logits so far
        auto raise = [&](float top, bool together) {
            volatile uint32_t *tops = sm.tops;
            if (keep == 1) {
                const uint32_t mine = __reduce_max_sync(0xffffffffu, float_order_bits(top));
                if (lane < 4)
                    tops[warp * 4 + lane] = mine;
            } else {
                lanes_tops(float_order_bits(top), tops + warp * 4, lane);
            }
            if (together)
                sums_barrier();
            else
                __syncwarp();
            if (keep == 1)
                cand.raise_to(__reduce_max_sync(0xffffffffu, tops[lane]));
            else
                cand.raise_to(__shfl_sync(0xffffffffu, sort32_desc(tops[lane], lane), keep - 1));
        };
        for (int v0 = x.from; v0 < x.to || stage == 0; v0 += kLpVectors, ++stage) {
            const int s = static_cast<int>(it % kLpStages), left = x.to - v0;
            const uint4 *ring = sm.ring[s];
            constexpr uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
            auto vector = [&](int i) { return i < left ? ring[i] : make_uint4(none, none, none, none); };
            if (left > 0)
                attn_wait(&sm.abort_flag, p.fault, smem_addr(&sm.full[s]), (it / kLpStages) & 1, 0);
            if (keep > 0 && stage == update) {
                update = 2 * stage + 4;
                float top = run;
#pragma unroll
                for (int u = 0; u < kLpVectors / kLpThreads; ++u) {
                    const uint4 q[1] = {vector(u * kLpThreads + tid)};
                    top = fmaxf(top, top_of<N>(q));
                }
                raise(top, stage == 0);
            }
#pragma unroll 1
            for (int u0 = 0; u0 < kLpVectors / kLpThreads; u0 += H) {
                if (u0 * kLpThreads + warp * 32 >= left)
                    break;
                uint4 q[H];
                if (left >= kLpVectors) {
#pragma unroll
                    for (int w = 0; w < H; ++w)
                        q[w] = ring[(u0 + w) * kLpThreads + tid];
                } else {
#pragma unroll
                    for (int w = 0; w < H; ++w)
                        q[w] = vector((u0 + w) * kLpThreads + tid);
                }
                const float top = top_of<N>(q);
                run = fmaxf(run, top);
                if (__any_sync(0xffffffffu, top >= fminf(cand.at_least, moves))) {
                    const bool passes = top >= cand.at_least && top > -INFINITY;
                    const uint32_t who = __ballot_sync(0xffffffffu, passes);
                    if (passes)
                        sm.noted[warp][noted + __popc(who & ((1u << lane) - 1u))] = v0 + u0 * kLpThreads + tid;
                    noted += __popc(who);
                    if (__any_sync(0xffffffffu, top > moves)) {
                        const float m = float_from_order_bits(__reduce_max_sync(0xffffffffu, float_order_bits(fmaxf(top, -INFINITY))));
                        part.move(m, c);
                        const float at = m * c;
                        far = !(fabsf(at) < 4096.0f && floor_at < 1e37f);
                        minus_m = -at;
                        off = fmaf(m, c, -at);
                        undo = exp2_approx(-off);
                        moves = m + lag;
                        const uint32_t least = __float_as_uint(m - floor_at) >> 16;
                        least2 = least | least << 16;
                    }
                }
                if (!far) {
                    uint64_t s2[2] = {0, 0}, h2[2] = {0, 0};
                    const uint64_t c2 = pack2(c, c), m2 = pack2(minus_m, minus_m);
#pragma unroll
                    for (int w = 0; w < H; ++w) {
                        float l[N];
                        if (N == 8)
                            raw_logits(make_uint4(bf16x2_max(q[w].x, least2), bf16x2_max(q[w].y, least2),
                                                  bf16x2_max(q[w].z, least2), bf16x2_max(q[w].w, least2)), l);
                        else
                            raw_logits(q[w], l);
#pragma unroll
                        for (int e = 0; e < N; e += 2) {
                            float y, z;
                            unpack2(fma2(pack2(l[e], l[e + 1]), c2, m2), y, z);
                            if (N == 4) {
                                y = fmaxf(y, -200.0f);
                                z = fmaxf(z, -200.0f);
                            }
                            const uint64_t t = pack2(exp2_approx(y), exp2_approx(z));
                            s2[(e / 2) & 1] = add2(s2[(e / 2) & 1], t);
                            h2[(e / 2) & 1] = fma2(t, pack2(y, z), h2[(e / 2) & 1]);
                        }
                    }
                    float a, b;
                    unpack2(add2(s2[0], s2[1]), a, b);
                    const float sum = a + b;
                    unpack2(add2(h2[0], h2[1]), a, b);
                    part.s = fmaf(undo, sum, part.s);
                    part.h = fmaf(undo, fmaf(-off, sum, a + b), part.h);
                } else {
                    const float ref = part.m == -INFINITY ? 0.0f : part.m;
#pragma unroll
                    for (int w = 0; w < H; ++w) {
                        float l[N];
                        raw_logits(q[w], l);
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            const float y = fmaxf((l[e] - ref) * c, -200.0f), t = exp2_approx(y);
                            part.s += t;
                            part.h = fmaf(t, y, part.h);
                        }
                    }
                }
            }
            if (noted > kLpNoted - 64) {  // (a stage notes 64 at most)
                cand = read_noted<N>(cand, buffer, sm.list[warp], sm.noted[warp], noted, keep, lane, vectors, x.to, x.head);
                noted = 0;
            }
            if (left > 0) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&sm.empty[s]));
                ++it;
            }
        }
        // the elements before the first vector and behind the last one: fewer than 2 N, by the last CTA's first warp
        if (crank == C - 1 && warp == 0) {
            const int tail = x.head + x.nv * N;
            const int v = lane < x.head ? lane : tail + lane - x.head;
            const float l = lane < x.head || v < V ? Logits<T>::one(x.row + v) : -INFINITY;
            part.join(LogSum{l, l > -INFINITY ? 1.0f : 0.0f, 0.0f}, c);
            if (keep > 0) {
                cand.push(buffer, l > -INFINITY ? logit_key(l, v) : 0, lane);
                if (cand.fill >= 32)  // (the next push has room for 32)
                    cand = merge_candidates(cand, buffer, sm.list[warp], keep, lane);
            }
        }
        part = lanes_join(part, c);
        if (noted > 0)
            cand = read_noted<N>(cand, buffer, sm.list[warp], sm.noted[warp], noted, keep, lane, vectors, x.to, x.head);
        if (cand.listed) {  // a list that was needed, and what waits
            while (cand.fill > 0)
                cand = merge_candidates(cand, buffer, sm.list[warp], keep, lane);
            buffer[lane] = sm.list[warp][lane];
            cand.fill = __popc(__ballot_sync(0xffffffffu, sm.list[warp][lane] != 0));  // (in order, so without gaps)
        }
        __syncwarp();
        if (lane == 0) {
            sm.m[warp] = part.m;
            sm.s[warp] = part.s;
            sm.h[warp] = part.h;
            sm.reach[warp] = cand.bound;
        }
        sums_barrier();
        if (keep > 0) {
            uint64_t reach = sm.reach[0];
#pragma unroll
            for (int w = 1; w < kLpWarps; ++w)
                reach = umax64(reach, sm.reach[w]);
            for (int i = 0; i < cand.fill; i += 32) {
                const uint64_t k = i + lane < cand.fill ? buffer[i + lane] : 0;
                const uint32_t who = __ballot_sync(0xffffffffu, k >= reach);
                int at = 0;
                if (lane == 0 && who)
                    at = atomicAdd(&sm.count, __popc(who));
                at = __shfl_sync(0xffffffffu, at, 0);
                if (k >= reach)
                    sm.all[at + __popc(who & ((1u << lane) - 1u))] = k;
            }
            sums_barrier();
            const int count = sm.count;
            for (int i = tid; i < count; i += kLpThreads) {
                const uint64_t k = sm.all[i];
                int place = 0;
                for (int o = 0; o < count; ++o)
                    place += sm.all[o] > k;
                if (place < 32)
                    sm.best[place] = k;
            }
        }
        if (warp == 0) {
            LogSum all{-INFINITY, 0.0f, 0.0f};
            if (lane < kLpWarps)
                all = LogSum{sm.m[lane], sm.s[lane], sm.h[lane]};
            all = lanes_join(all, c);
            if (lane == 0) {
                sm.cm = all.m;
                sm.cs = all.s;
                sm.ch = all.h;
            }
        }
        sums_barrier();
        if (C > 1)
            cluster_sync_all();
        if (crank == 0) {
            if (C > 1 && keep > 0) {  // the CTAs' lists: a warp each, a key's place by search in the others
                if (warp < C)
                    sm.all[tid] = dsmem_ld_u64(mapa_shared(smem_addr(&sm.best[lane]), warp));
                sums_barrier();
                if (warp < C) {
                    const uint64_t k = sm.all[tid];
                    int place = lane;
                    for (int o = 0; o < C; ++o) {
                        int larger = 0;  // of list o's keys
#pragma unroll
                        for (int step = 16; step >= 1; step >>= 1)
                            larger += sm.all[o * 32 + larger + step - 1] > k ? step : 0;
                        larger += sm.all[o * 32 + larger] > k;
                        place += o == warp ? 0 : larger;
                    }
                    if (k != 0 && place < 32)
                        sm.best[place] = k;
                }
                sums_barrier();
            }
            if (warp == 0) {
                LogSum all{-INFINITY, 0.0f, 0.0f};
                uint64_t list = sm.best[lane];
                int bad = 0;
                if (lane < C) {
                    all = LogSum{dsmem_ld_f32(mapa_shared(smem_addr(&sm.cm), lane)),
                                 dsmem_ld_f32(mapa_shared(smem_addr(&sm.cs), lane)),
                                 dsmem_ld_f32(mapa_shared(smem_addr(&sm.ch), lane))};
                    bad = dsmem_ld_s32(mapa_shared(smem_addr(&sm.abort_flag), lane));
                }
                all = lanes_join(all, c);
                if (__any_sync(0xffffffffu, bad)) {  // a wait that ran out: nothing
                    list = 0;
                    all = LogSum{-INFINITY, 0.0f, 0.0f};
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
            sums_barrier();
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
        sums_barrier();  // the row's numbers have been read
        if (C > 1)
            cluster_sync_all();
    }
}

template <class T>
static msa_status launch_logprobs(const LogprobParams &p, int cluster, int sms, int dev, cudaStream_t st)
{
    static std::atomic<bool> allowed[kMaxDevices];
    if (!allow_smem(logprobs_kernel<T>, sizeof(LogprobSmem), dev, allowed))
        return MSA_ERR_CUDA;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(cluster > 1 ? p.rows * cluster : std::min<int64_t>(p.rows, kLpBlocks * sms)));
    cfg.blockDim = dim3(kLpThreads + 32);
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
    p.rows = rows;
    // CTAs a row: as many as there is room for, two an SM for pairs, one an SM for larger clusters, which do not fit so densely.
    // fp32, 5 alternatives, with 8 / 4 / 2 / 1 of them: 1 x 163840 9.2 / 10.9 / 15.0 / 21.4 us, 16 x 131072 9.9 / 10.7 / 14.2 /
    // 19.1, 38 rows 18.3 / 11.7 / 14.3 / 19.2, 76 - / 23.5 / 16.4 / 20.3, 152 - / - / 21.6 / 21.8.
    int cluster = 8;
    while (cluster > 1 && rows * cluster > (cluster > 2 ? sms : 2 * sms))
        cluster /= 2;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return logits_bf16 ? launch_logprobs<uint16_t>(p, cluster, sms, dev, st)
                       : launch_logprobs<float>(p, cluster, sms, dev, st);
}

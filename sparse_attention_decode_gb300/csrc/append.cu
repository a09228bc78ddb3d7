// New tokens enter the paged caches: keys normalised, rotated and, for an E4M3
// cache, quantised on the way; the queries of the same tokens beside them.
//
// Mathematics.  A head's 128 values x, weights w, n = 1 / sqrt(mean x^2 + eps) and
// the angle a_i of pair i: every output is n (x_j A_j + x_p B_j), with j's partner p
// in its pair, A_j = w_j cos a, B_j = -+ w_p sin a.  A and B are a token's, the same
// for all heads of one kind, so a head costs two multiply-adds a value beside its sum of
// squares; where nothing turns, A = w and B = 0.
//
// Angles.  position * inv_freq is wanted modulo one turn.  Turns are counted in units of
// 2^-64 in a 64-bit integer, which wraps where a turn ends: F = inv_freq 2^64 / (2 pi)
// once, from the bits of the fp32 value and a 64-bit 1 / (2 pi), then position * F.
// That is exact but for F's own rounding (position * 2^-64 turns, or that times inv_freq / 4 where it is more: below 2^-22
// rad up to an inv_freq of 2^10 and any position); an fp32 product
// would be off by 0.06 rad at a position of 10^6, and 64-bit floating-point products run
// at a 64th of the rate.  (Integer work of one thread a pair: nothing beside the heads.)
//
// What bounds it: with many rows the stream in and out (4 requests of 2048 new tokens, 64 query and 8 key and value heads,
// 237 MB: 43.2 us, 5.5 TB/s, where copying the same rows through the same ring takes 40.7); with few the launch and one
// row's chain of loads, its place, its page, its heads (a token of one request 3.2 us, 128 rows of E4M3 keys and values 5.6).
// In fp32; q, keys and values are rounded once, to bf16 or, relative to the head's largest, to E4M3, the caches' types.
#include <algorithm>
#include <cmath>

#include "attn_common.cuh"
#include "attn_ptx.cuh"
#include "host_util.cuh"
#include "layout.cuh"
#include "overlap.h"

#include "msa_serving.h"

namespace msa {

bool cache_ok(const void *base, const int64_t *strides, int64_t pages, int heads, bool fp8);  // attention.cu
bool unaligned(const void *p, uintptr_t a);

struct AppendParams {
    const uint16_t *q, *k, *v;
    uint16_t *out_q;
    uint8_t *k_cache, *v_cache;
    float *k_scale, *v_scale;
    const float *q_weight, *k_weight, *inv_freq;
    const int32_t *positions, *block_table, *seq_lens, *cu;
    uint32_t *fault;
    int64_t q_stride, out_q_stride, k_stride, v_stride;
    int64_t kc_stride[3], vc_stride[3];  // elements (page, token, head)
    int64_t bt_stride, num_pages, rows;
    int batch, q_len, q_heads, kv_heads, rot, seq_limit;
    float eps;
};

constexpr int kAppendThreads = 128;
constexpr int kAppendBatch = 4;                    // heads of a lane under way together
constexpr float kTinyEps = 8.271806125530277e-25f;  // 2^-80: from there on what underflows of a head's squares is nothing beside it
constexpr uint64_t kInverseTurn = 11743562013128004906ull;  // 2^66 / (2 pi)

// inv_freq in units of 2^-64 turns a position, modulo a turn: m 2^e with an integer m of 24 bits.
__device__ __forceinline__ uint64_t turns_of(float f)
{
    const uint32_t u = __float_as_uint(f), field = (u >> 23) & 255u;
    const uint64_t m = (u & 0x7fffffu) | (field ? 0x800000u : 0u);
    const int e = static_cast<int>(field ? field : 1u) - 150 - 2;  // times 2^66 / (2 pi): units of 2^-64 after 2^(e - 2)
    const uint64_t lo = m * kInverseTurn, hi = __umul64hi(m, kInverseTurn);
    uint64_t r;
    if (e >= 64)
        r = 0;  // (none of the digits that count are among the 64)
    else if (e >= 0)
        r = lo << e;
    else if (e > -64)
        r = (lo >> -e) | (hi << (64 + e));
    else
        r = e > -128 ? hi >> (-e - 64) : 0;
    return u >> 31 ? 0 - r : r;
}

__device__ __forceinline__ void turn(uint64_t f, int position, float &cs, float &sn)
{
    const uint64_t at = static_cast<uint64_t>(static_cast<int64_t>(position)) * f;
    // the nearest of 2^32 fractions of a turn in [-1/2, 1/2), and in half turns
    const int32_t part = static_cast<int32_t>((at + 0x80000000ull) >> 32);
    sincospif(static_cast<float>(part) * 4.656612873077393e-10f, &sn, &cs);
}


__device__ __forceinline__ float half_warp_sum(float x)
{
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float half_warp_max(float x)
{
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1)
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// Where a row goes: its request's token, or nowhere (live false; page -1: its key and value).
struct RowPlace {
    bool live;
    int position, page, slot;
};

// Row `row` of request b, whose rows are [lo, lo + n).
__device__ __forceinline__ RowPlace row_place(const AppendParams &p, int64_t row, int b, int lo, int n, bool bad)
{
    const int len = p.seq_lens[b];
    bad |= len < 0 || len > p.seq_limit || (p.cu && n > len);
    RowPlace x{false, 0, -1, 0};
    if (bad) {
        atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
        return x;
    }
    const int token = len - n + static_cast<int>(row - lo);
    if (token < 0)
        return x;
    x.live = true;
    x.position = p.positions ? p.positions[row] : token;
    x.page = p.block_table[b * p.bt_stride + token / kPage];
    x.slot = token % kPage;
    if (x.page < 0 || x.page >= p.num_pages) {
        atomicOr(p.fault, MSA_FAULT_PAGE_ID);
        x.page = -1;
    }
    return x;
}

// Rows of requests that do not follow one another.
__device__ __forceinline__ void check_rows(const AppendParams &p)  // by one block
{
    if (p.cu)
        for (int b = threadIdx.x; b < p.batch; b += blockDim.x)
            if (p.cu[b + 1] < p.cu[b] || p.cu[b + 1] > p.rows)
                atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
}

// The row's request looked up; cu: the first b with cu[b + 1] > row.
__device__ __forceinline__ RowPlace row_place(const AppendParams &p, int64_t row)
{
    if (!p.cu) {
        const int b = static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(p.q_len));  // (rows are below 2^27)
        return row_place(p, row, b, b * p.q_len, p.q_len, false);
    }
    int b = 0, end = p.batch;
    while (b < end) {
        const int mid = (b + end) >> 1;
        if (p.cu[mid + 1] > row)
            end = mid;
        else
            b = mid + 1;
    }
    if (b == p.batch)
        return RowPlace{false, 0, -1, 0};
    const int lo = p.cu[b], hi = p.cu[b + 1];
    return row_place(p, row, b, lo, hi - lo, lo < 0 || lo > row || hi > p.rows);
}

// A lane's part in heads: the row's line of heads (queries, keys, values), the lane's coefficients of one kind of them.
// LIFT: eps is next to nothing (below kTinyEps).  (As a branch of one kernel 237 MB of prompts took 45.6 us for 43.4.)
template <bool FP8, bool INTER, bool LIFT>
struct HeadLane {
    const AppendParams &p;
    int nq, nk, all;   // heads before the keys, before the values, and all
    int sub, lane;
    int half, partner; // lanes of a head that hold a first half of the rotated dims (pairs apart); who holds the others
    int kind = -1;
    bool norm = false;
    uint64_t A[4], B[4];  // two values each

    __device__ __forceinline__ explicit HeadLane(const AppendParams &p_) : p(p_)
    {
        nq = p.q ? p.q_heads : 0;
        nk = nq + p.kv_heads;
        all = p.v ? nk + p.kv_heads : nk;
        lane = threadIdx.x & 31;
        sub = lane & 15;
        half = p.rot / 16;
        partner = INTER ? sub : sub < half ? sub + half : sub < 2 * half ? sub - half : sub;
    }
    // the lane's weights of kind `is`, and its partner's
    __device__ __forceinline__ void weights(int is, float (&w)[8], float (&wp)[8]) const
    {
        const float *weight = is == 0 ? p.q_weight : is == 1 ? p.k_weight : nullptr;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = weight ? weight[sub * 8 + j] : 1.0f;
            wp[j] = weight ? weight[INTER ? sub * 8 + (j ^ 1) : partner * 8 + j] : 1.0f;
        }
    }
    __device__ __forceinline__ void coefficients(int is, const float (&w)[8], const float (&wp)[8], const float *cosines,
                                                 const float *sines)
    {
        kind = is;
        norm = (is == 0 ? p.q_weight : is == 1 ? p.k_weight : nullptr) != nullptr;
        const bool turns = is < 2 && sub < 2 * half;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float a[2], c[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int pair = INTER ? sub * 4 + j / 2 : (turns && sub >= half ? sub - half : sub) * 8 + j + e;
                const bool first = INTER ? e == 0 : sub < half;
                a[e] = turns ? w[j + e] * cosines[pair] : w[j + e];
                c[e] = turns ? wp[j + e] * (first ? -sines[pair] : sines[pair]) : 0.0f;
            }
            A[j / 2] = pack2(a[0], a[1]);
            B[j / 2] = pack2(c[0], c[1]);
        }
    }
    // Where next to nothing is added to them, a head's squares must not underflow: a small one is normalised 2^90 times as
    // large, which is exact in bf16.  A head of zeros is to stay one.
    __device__ __forceinline__ void lift(uint32_t (&w)[4], float &eps) const
    {
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            top = max3(top, fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u)));
        top = half_warp_max(top);
        if (norm && top < 8.881784197001252e-16f) {  // 2^-50
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w[j]) : "r"(0x6c806c80u));  // 2^90, two
            eps = top > 0.0f ? eps * 1.2379400392853803e27f * 1.2379400392853803e27f : 1.0f;  // 2^180
        }
    }
    // the lane's 8 values of a head of the kind at hand, normalised and rotated; all lanes of the warp together
    __device__ __forceinline__ void turned(const uint4 &raw, float (&f)[8]) const
    {
        uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        float eps = p.eps;
        if (LIFT)
            lift(w, eps);
        uint64_t x[4], sum2 = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = pack2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
            sum2 = fma2(x[j], x[j], sum2);
        }
        float inv = 1.0f;
        if (p.q_weight || p.k_weight) {
            float s0, s1;
            unpack2(sum2, s0, s1);
            const float r = rsqrtf(half_warp_sum(s0 + s1) * (1.0f / kDim) + eps);
            inv = norm ? r : 1.0f;
        }
        const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint64_t t = 0;
            if (p.rot) {
                const uint32_t o = INTER ? __byte_perm(w[j], 0, 0x1032) : __shfl_sync(0xffffffffu, w[j], (lane & 16) | partner);
                t = mul2(pack2(__uint_as_float(o << 16), __uint_as_float(o & 0xffff0000u)), B[j]);
            }
            unpack2(mul2(fma2(x[j], A[j], t), inv2), f[2 * j], f[2 * j + 1]);
        }
    }
    static __device__ __forceinline__ uint4 packed(const float (&f)[8])
    {
        return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                          f32x2_to_bf16x2(f[6], f[7]));
    }
    // head `at` of the line, of any kind
    __device__ __forceinline__ void head(int at, const uint4 &raw, int64_t row, int page, int slot, const float *cosines,
                                         const float *sines)
    {
        const bool have = at < all;
        const int is = at < nq ? 0 : at < nk ? 1 : 2;
        float f[8];
        if (is != kind) {
            float wp[8];
            weights(is, f, wp);
            coefficients(is, f, wp, cosines, sines);
        }
        turned(raw, f);
        const bool write = have && (is == 0 || page >= 0);
        if ((!FP8 || is == 0) && write) {
            uint16_t *dst;
            if (is == 0) {
                dst = p.out_q + row * p.out_q_stride + at * kDim;
            } else {
                const int64_t *st = is == 1 ? p.kc_stride : p.vc_stride;
                dst = reinterpret_cast<uint16_t *>(is == 1 ? p.k_cache : p.v_cache) + page * st[0] + slot * st[1] +
                      (at - (is == 1 ? nq : nk)) * st[2];
            }
            *reinterpret_cast<uint4 *>(dst + sub * 8) = is == 2 ? raw : packed(f);
        }
        if (!FP8 || !__any_sync(0xffffffffu, is != 0))
            return;
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            top = max3(top, fabsf(f[j]), fabsf(f[j + 1]));
        top = half_warp_max(top);
        const float unit = top < 6.018531076210112e-36f ? 0.0f : top / 448.0f;  // 2^-117: the quotient is normal
        const float up = unit > 0.0f ? 1.0f / unit : 0.0f;
        if (write && is != 0) {
            const int64_t *st = is == 1 ? p.kc_stride : p.vc_stride;
            const int g = at - (is == 1 ? nq : nk);
            uint32_t c[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                c[j] = e4m3_pair(f[4 * j] * up, f[4 * j + 1] * up) |
                       static_cast<uint32_t>(e4m3_pair(f[4 * j + 2] * up, f[4 * j + 3] * up)) << 16;
            *reinterpret_cast<uint2 *>((is == 1 ? p.k_cache : p.v_cache) + page * st[0] + slot * st[1] + g * st[2] + sub * 8) =
                unit > 0.0f ? make_uint2(c[0], c[1]) : make_uint2(0u, 0u);
            if (sub == 0)
                (is == 1 ? p.k_scale : p.v_scale)[(static_cast<int64_t>(page) * p.kv_heads + g) * kPage + slot] = unit;
        }
    }
};

// Few rows, or short ones: a row a warp, or a share of its heads (`shares` warps a row, which take its heads two at a time
// in turn).  A lane's first heads are asked for before the row's place is looked up.
template <bool FP8, bool INTER, bool LIFT>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p, int shares)
{
    __shared__ float s_cos[kAppendThreads / 32][kDim / 2], s_sin[kAppendThreads / 32][kDim / 2];
    const int warp = threadIdx.x >> 5;
    const int64_t at_warp = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + warp, row = at_warp / shares;
    if (blockIdx.x == 0)
        check_rows(p);
    if (row >= p.rows)
        return;
    HeadLane<FP8, INTER, LIFT> x(p);
    const int first = static_cast<int>(at_warp - row * shares) * 2, h0 = first + (x.lane >> 4), step = 2 * shares;
    auto load = [&](int h) {
        const uint16_t *from = h < x.nq   ? p.q + row * p.q_stride + h * kDim
                               : h < x.nk ? p.k + row * p.k_stride + (h - x.nq) * kDim
                                          : p.v + row * p.v_stride + (h - x.nk) * kDim;
        return h < x.all ? reinterpret_cast<const uint4 *>(from)[x.sub] : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 in[kAppendBatch];
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i)
        in[i] = load(h0 + i * step);
    const RowPlace at = row_place(p, row);  // (every lane: one address, one answer)
    if (!at.live)
        return;
#pragma unroll
    for (int i = x.lane; i < kDim / 2; i += 32)
        if (i < p.rot / 2)
            turn(turns_of(p.inv_freq[i]), at.position, s_cos[warp][i], s_sin[warp][i]);
    __syncwarp();
    for (int h = 0; first + h < x.all; h += kAppendBatch * step) {
#pragma unroll
        for (int u = 0; u < kAppendBatch; ++u) {
            if (first + h + u * step >= x.all)
                break;
            const uint4 raw = in[u];
            in[u] = load(h0 + h + (u + kAppendBatch) * step);
            x.head(h0 + h + u * step, raw, row, at.page, at.slot, s_cos[warp], s_sin[warp]);
        }
    }
}

// Many rows: blocks that stay, and take rows in turn.  A warp looks up the places of the block's next 32 rows at a time,
// a lane a row, has the rows copied into a ring in shared memory and works out their sines and cosines; four warps turn
// the heads.  What has to be on its way for the copy rate does not depend on registers then.
struct AppendRow {
    float cosines[kDim / 2], sines[kDim / 2];
    int live, page, slot, pad;
};
constexpr int kRowsThreads = 128;
constexpr int kRowsHeads = kRowsThreads / 16;
constexpr int kAppendStages = 2;
constexpr int kAppendBlocks = 5;  // an SM (4 with 3 rows each: 48.8 us for 237 MB, 43.2)
constexpr int kAppendSmBytes = 233472;
constexpr int append_block_bytes(int row_bytes)  // with the static shared memory and what the system takes
{
    return kAppendStages * (row_bytes + static_cast<int>(sizeof(AppendRow))) + 128 + 1024;
}

template <bool FP8, bool INTER, bool LIFT>
__global__ void __launch_bounds__(kRowsThreads + 32, kAppendBlocks) append_rows_kernel(const __grid_constant__ AppendParams p, int row_bytes)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kAppendStages], empty[kAppendStages];
    __shared__ AppendRow places[kAppendStages];
    __shared__ int abort_flag;
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 15) & ~uintptr_t(15));
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        for (int s = 0; s < kAppendStages; ++s) {
            mbar_init(smem_addr(&full[s]), 2);  // the copies, and the row's place
            mbar_init(smem_addr(&empty[s]), kRowsThreads / 32);
        }
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    HeadLane<FP8, INTER, LIFT> x(p);
    const int64_t step = gridDim.x;
    if (blockIdx.x == 0)
        check_rows(p);
    if (warp == kRowsThreads / 32) {
        const uint64_t turns[2] = {lane < p.rot / 2 ? turns_of(p.inv_freq[lane]) : 0,
                                   lane + 32 < p.rot / 2 ? turns_of(p.inv_freq[lane + 32]) : 0};
        uint32_t it = 0;
        bool alive = true;
        for (int64_t r0 = blockIdx.x; r0 < p.rows && alive; r0 += 32 * step) {
            RowPlace mine{false, 0, -1, 0};
            bool looked = false;
            for (int i = 0; i < 32 && r0 + i * step < p.rows && alive; ++i, ++it) {
                const int64_t row = r0 + i * step;
                const int s = static_cast<int>(it % kAppendStages);
                if (it >= kAppendStages)
                    alive = attn_wait(&abort_flag, p.fault, smem_addr(&empty[s]), (it / kAppendStages + 1) & 1, 0);
                if (!alive)
                    break;
                if (lane == 0) {
                    const uint32_t bar = smem_addr(&full[s]), to = smem_addr(ring + s * row_bytes);
                    mbar_arrive_expect_tx(bar, x.all * kDim * 2);
                    if (x.nq)
                        bulk_load(to, p.q + row * p.q_stride, x.nq * kDim * 2, bar);
                    bulk_load(to + x.nq * kDim * 2, p.k + row * p.k_stride, p.kv_heads * kDim * 2, bar);
                    if (p.v)
                        bulk_load(to + x.nk * kDim * 2, p.v + row * p.v_stride, p.kv_heads * kDim * 2, bar);
                }
                __syncwarp();
                if (!looked) {  // beside the first copies
                    if (r0 + lane * step < p.rows)
                        mine = row_place(p, r0 + lane * step);
                    looked = true;
                }
                AppendRow &to = places[s];
                const int position = __shfl_sync(0xffffffffu, mine.position, i);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (lane + 32 * k < p.rot / 2)
                        turn(turns[k], position, to.cosines[lane + 32 * k], to.sines[lane + 32 * k]);
                if (lane == i) {
                    to.live = mine.live;
                    to.page = mine.page;
                    to.slot = mine.slot;
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&full[s]));
            }
        }
        // the copies in flight land before the block may end
        for (uint32_t j = it >= kAppendStages ? it - kAppendStages : 0; j < it; ++j)
            mbar_wait(smem_addr(&full[j % kAppendStages]), (j / kAppendStages) & 1);
        return;
    }
    float w[8], wp[8];  // the queries' weights
    x.weights(0, w, wp);
    uint32_t it = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += step, ++it) {
        const int s = static_cast<int>(it % kAppendStages);
        if (!attn_wait(&abort_flag, p.fault, smem_addr(&full[s]), (it / kAppendStages) & 1, 0))
            return;
        const AppendRow &at = places[s];
        if (at.live) {
            const uint4 *from = reinterpret_cast<const uint4 *>(ring + s * row_bytes) + x.sub;
            x.kind = -1;
            int h = 0;
            if (x.nq >= kRowsHeads) {  // queries, as far as every half warp has one
                x.coefficients(0, w, wp, at.cosines, at.sines);
                uint16_t *dst = p.out_q + row * p.out_q_stride + (tid / 16) * kDim + x.sub * 8;
                const uint4 *src = from + (tid / 16) * 16;
#pragma unroll 2
                for (; h + kRowsHeads <= x.nq; h += kRowsHeads) {
                    float f[8];
                    x.turned(src[h * 16], f);
                    *reinterpret_cast<uint4 *>(dst + h * kDim) = x.packed(f);
                }
            }
            for (; h < x.all; h += kRowsHeads) {
                const int mine = h + tid / 16;
                x.head(mine, mine < x.all ? from[mine * 16] : make_uint4(0u, 0u, 0u, 0u), row, at.page, at.slot, at.cosines, at.sines);
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_addr(&empty[s]));
    }
}

template <bool FP8, bool INTER, bool LIFT>
static msa_status launch_append(const AppendParams &p, int sms, int dev, cudaStream_t st)
{
    const int heads = (p.q ? p.q_heads : 0) + (p.v ? 2 : 1) * p.kv_heads;
    const int64_t bytes = static_cast<int64_t>(heads) * kDim * 2;
    const int blocks = bytes < kAppendSmBytes / 4 ? std::min(kAppendBlocks, kAppendSmBytes / append_block_bytes(static_cast<int>(bytes))) : 0;
    // The ring: more rows than SMs (160 rows of 72 heads 5.9 us with it, 6.2 without), lines of 24 heads and more, where a
    // row is enough to hide its set-up, that fit twice an SM.  With it and without, 6440 rows of 40 / 32 / 24 / 20 / 16 heads:
    // 31.1 and 39.2, 28.3 and 33.2, 25.1 and 27.2, 23.9 and 24.1, 20.9 and 21.1 us; a quarter of the rows: 11.9 and 13.1, 10.8
    // and 11.1, 9.5 and 9.6, 9.2 and 8.3, 8.2 and 7.6; E4M3, 6440 rows: 36.5 and 51.1, 32.9 and 42.9, 29.3 and 36.7, 28.3 and
    // 31.0, 24.5 and 27.7, 200 rows: 5.7 and 5.9, 5.5 and 5.7, 5.2 and 4.6, 5.1 and 4.6, 4.8 and 4.3.
    if (p.rows > sms && heads >= 24 && blocks >= 2) {
        static std::atomic<bool> allowed[kMaxDevices];
        auto *kernel = append_rows_kernel<FP8, INTER, LIFT>;
        if (!allow_smem(kernel, kAppendSmBytes / 2 - 1024 - kAppendStages * sizeof(AppendRow) - 128, dev, allowed))
            return MSA_ERR_CUDA;
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>(p.rows, blocks * sms));
        kernel<<<grid, kRowsThreads + 32, static_cast<size_t>(kAppendStages * bytes + 16), st>>>(p, static_cast<int>(bytes));
    } else {
        // 16 warps an SM (64 rows of 72 heads 4.2 us, with 8 4.7; 128 E4M3 rows 5.6, with 32 7.6)
        const int shares = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((heads + 1) / 2, (16 * sms + p.rows - 1) / p.rows)));
        const int64_t blocks_of = (p.rows * shares + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
        append_kernel<FP8, INTER, LIFT><<<static_cast<unsigned>(blocks_of), kAppendThreads, 0, st>>>(p, shares);
    }
    return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

template <bool LIFT>
static msa_status launch_append_kind(const AppendParams &p, bool fp8, bool interleaved, int sms, int dev, cudaStream_t st)
{
    if (fp8)
        return interleaved ? launch_append<true, true, LIFT>(p, sms, dev, st) : launch_append<true, false, LIFT>(p, sms, dev, st);
    return interleaved ? launch_append<false, true, LIFT>(p, sms, dev, st) : launch_append<false, false, LIFT>(p, sms, dev, st);
}

static msa_status append_entry(AppendParams &p, const int64_t *k_strides, const int64_t *v_strides, int interleaved,
                               int64_t total_rows, int batch, int max_model_len, void *workspace,
                               size_t workspace_bytes, void *stream, bool fp8)
{
    const bool values = p.v || p.v_cache;
    if (batch < 0 || total_rows < 0 || p.kv_heads < 1 || p.num_pages < 1 || p.bt_stride < 1 || max_model_len < 1 ||
        (!p.cu && (p.q_len < 1 || total_rows != static_cast<int64_t>(batch) * p.q_len)) || !(p.eps >= 0.0f) ||
        !(p.eps < INFINITY) || p.rot < 0 || (p.rot > 0 && !p.inv_freq) || (p.q == nullptr) != (p.out_q == nullptr) ||
        (p.q && p.q_heads < 1))
        return MSA_ERR_INVALID_ARG;
    if (batch > MSA_MAX_BATCH || p.num_pages > (int64_t{1} << 24) || p.kv_heads > 1024 || (p.q && p.q_heads > 65536) ||
        p.rot > kDim || p.rot % 16 || total_rows > (int64_t{1} << 27))
        return MSA_ERR_UNSUPPORTED;
    if (batch == 0 || total_rows == 0)  // (an empty tensor has no address)
        return MSA_OK;
    const int64_t kv = static_cast<int64_t>(p.kv_heads) * kDim, qd = static_cast<int64_t>(p.q_heads) * kDim;
    if (!p.k || !p.block_table || !p.seq_lens || !workspace || (values && (!p.v || !p.v_cache)) ||
        !cache_ok(p.k_cache, k_strides, p.num_pages, p.kv_heads, fp8) ||
        (values && !cache_ok(p.v_cache, v_strides, p.num_pages, p.kv_heads, fp8)) || unaligned(p.q, 16) ||
        unaligned(p.out_q, 16) || unaligned(p.k, 16) || unaligned(p.v, 16) || unaligned(workspace, 256) ||
        p.k_stride % 8 || p.k_stride < kv || (values && (p.v_stride % 8 || p.v_stride < kv)) ||
        (p.q && (p.q_stride % 8 || p.q_stride < qd || p.out_q_stride % 8 || p.out_q_stride < qd)) ||
        (p.q && p.out_q == p.q && p.out_q_stride != p.q_stride))
        return MSA_ERR_INVALID_ARG;
    if (fp8 && (!p.k_scale || (values && !p.v_scale) || unaligned(p.k_scale, 16) || unaligned(p.v_scale, 16)))
        return MSA_ERR_INVALID_ARG;
    // Heads are read by who writes them, so out_q may be q itself; any other overlap is a race between rows or heads.
    const bool in_place = p.out_q == p.q;
    auto rows_of = [&](const uint16_t *x, int64_t stride, int64_t width) { return RowSpan(x, stride * 2, width * 2, total_rows); };
    auto over = [&](const uint16_t *x, int64_t stride, int64_t width) {
        return p.q && x && rows_overlap(rows_of(p.out_q, p.out_q_stride, qd), rows_of(x, stride, width));
    };
    if (!in_place && (over(p.q, p.q_stride, qd) || over(p.k, p.k_stride, kv) || over(p.v, p.v_stride, kv)))
        return MSA_ERR_INVALID_ARG;
    if (workspace_bytes < kHeaderBytes)
        return MSA_ERR_WORKSPACE_TOO_SMALL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return MSA_ERR_CUDA;
    const int sms = device_sms(dev);
    if (sms <= 0)
        return MSA_ERR_CUDA;
    if (in_place && (over(p.k, p.k_stride, kv) || over(p.v, p.v_stride, kv)))
        return MSA_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
        p.kc_stride[i] = k_strides[i];
        p.vc_stride[i] = values ? v_strides[i] : 0;
    }
    p.fault = &static_cast<WorkspaceHeader *>(workspace)->fault;
    p.rows = total_rows;
    p.batch = batch;
    p.seq_limit = static_cast<int>(std::min<int64_t>(max_model_len, kPage * p.bt_stride));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((p.q_weight || p.k_weight) && p.eps < kTinyEps)
        return launch_append_kind<true>(p, fp8, interleaved != 0, sms, dev, st);
    return launch_append_kind<false>(p, fp8, interleaved != 0, sms, dev, st);
}

static AppendParams append_params(const void *q, int64_t q_stride, int q_heads, void *out_q, int64_t out_q_stride,
                                  const void *k, int64_t k_stride, const void *v, int64_t v_stride, int kv_heads,
                                  const float *q_weight, const float *k_weight, float eps, const float *inv_freq,
                                  int rotary_dim, const int32_t *positions, void *k_cache, void *v_cache,
                                  int64_t num_pages, const int32_t *block_table, int64_t bt_stride,
                                  const int32_t *seq_lens, const int32_t *cu_seqlens_q, int q_len)
{
    AppendParams p;
    std::memset(&p, 0, sizeof p);
    p.q = static_cast<const uint16_t *>(q);
    p.q_stride = q_stride;
    p.q_heads = q_heads;
    p.out_q = static_cast<uint16_t *>(out_q);
    p.out_q_stride = out_q_stride;
    p.k = static_cast<const uint16_t *>(k);
    p.k_stride = k_stride;
    p.v = static_cast<const uint16_t *>(v);
    p.v_stride = v_stride;
    p.kv_heads = kv_heads;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.eps = eps;
    p.inv_freq = inv_freq;
    p.rot = rotary_dim;
    p.positions = positions;
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.num_pages = num_pages;
    p.block_table = block_table;
    p.bt_stride = bt_stride;
    p.seq_lens = seq_lens;
    p.cu = cu_seqlens_q;
    p.q_len = q_len;
    return p;
}

}  // namespace msa

using namespace msa;

extern "C" msa_status msa_cache_append(const void *q, int64_t q_stride, int q_heads, void *out_q, int64_t out_q_stride,
                                       const void *k, int64_t k_stride, const void *v, int64_t v_stride, int kv_heads,
                                       const float *q_weight, const float *k_weight, float eps, const float *inv_freq,
                                       int rotary_dim, int interleaved, const int32_t *positions, void *k_cache,
                                       const int64_t *k_strides, void *v_cache, const int64_t *v_strides,
                                       int64_t num_pages, const int32_t *block_table, int64_t bt_stride,
                                       const int32_t *seq_lens, const int32_t *cu_seqlens_q, int64_t total_rows,
                                       int batch, int q_len, int max_model_len, void *workspace,
                                       size_t workspace_bytes, void *stream)
{
    AppendParams p = append_params(q, q_stride, q_heads, out_q, out_q_stride, k, k_stride, v, v_stride, kv_heads, q_weight,
                                   k_weight, eps, inv_freq, rotary_dim, positions, k_cache, v_cache, num_pages,
                                   block_table, bt_stride, seq_lens, cu_seqlens_q, q_len);
    return append_entry(p, k_strides, v_strides, interleaved, total_rows, batch, max_model_len, workspace,
                        workspace_bytes, stream, false);
}

extern "C" msa_status msa_cache_append_fp8(const void *q, int64_t q_stride, int q_heads, void *out_q,
                                           int64_t out_q_stride, const void *k, int64_t k_stride, const void *v,
                                           int64_t v_stride, int kv_heads, const float *q_weight,
                                           const float *k_weight, float eps, const float *inv_freq, int rotary_dim,
                                           int interleaved, const int32_t *positions, void *k_cache,
                                           const int64_t *k_strides, float *k_scale, void *v_cache,
                                           const int64_t *v_strides, float *v_scale, int64_t num_pages,
                                           const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                                           const int32_t *cu_seqlens_q, int64_t total_rows, int batch, int q_len,
                                           int max_model_len, void *workspace, size_t workspace_bytes, void *stream)
{
    AppendParams p = append_params(q, q_stride, q_heads, out_q, out_q_stride, k, k_stride, v, v_stride, kv_heads, q_weight,
                                   k_weight, eps, inv_freq, rotary_dim, positions, k_cache, v_cache, num_pages,
                                   block_table, bt_stride, seq_lens, cu_seqlens_q, q_len);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    return append_entry(p, k_strides, v_strides, interleaved, total_rows, batch, max_model_len, workspace,
                        workspace_bytes, stream, true);
}

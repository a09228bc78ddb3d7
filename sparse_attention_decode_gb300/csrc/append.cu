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
// That is exact but for F's own rounding (position * 2^-64 turns); an fp32 product
// would be off by 0.06 rad at a position of 10^6, and 64-bit floating-point products run
// at a 64th of the rate.  (Integer work of one thread a pair: nothing beside the heads.)
#include <algorithm>
#include <cmath>

#include "attn_ptx.cuh"
#include "host_util.cuh"
#include "layout.cuh"

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

constexpr int kAppendThreads = 256;
constexpr int kAppendHeads = kAppendThreads / 16;  // heads at a time: 16 lanes a head, 8 values a lane
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
        r = 0;  // whole turns
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

// A row a block (or a share of its heads, blockIdx.y of gridDim.y): query heads, then key heads, then value heads, 16
// at a time.
template <bool FP8, bool INTER>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p)
{
    __shared__ float s_cos[kDim / 2], s_sin[kDim / 2];
    const int tid = threadIdx.x, lane = tid & 31, sub = tid & 15;
    const int64_t row = blockIdx.x;
    // the row's request and token (every warp for itself)
    int b, n, i;
    bool bad = false, live = true;
    if (p.cu) {
        int before = 0;  // requests that end at or before the row
        for (int at = lane; at < p.batch; at += 32)
            before += p.cu[at + 1] <= row;
        b = __reduce_add_sync(0xffffffffu, before);
        live = b < p.batch;
        const int lo = live ? p.cu[b] : 0, hi = live ? p.cu[b + 1] : 0;
        n = hi - lo;
        i = static_cast<int>(row) - lo;
        bad = live && (lo < 0 || lo > row || hi <= row || hi > p.rows);
    } else {
        b = static_cast<int>(row / p.q_len);
        n = p.q_len;
        i = static_cast<int>(row - static_cast<int64_t>(b) * n);
    }
    const int len = live ? p.seq_lens[b] : 0;
    bad |= live && (len < 0 || len > p.seq_limit || (p.cu && n > len));
    const int token = len - n + i;
    if (bad && tid == 0)
        atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
    if (!live || bad || token < 0)
        return;
    const int position = p.positions ? p.positions[row] : token;
    int page = p.block_table[b * p.bt_stride + token / kPage];
    if (page < 0 || page >= p.num_pages) {
        if (tid == 0)
            atomicOr(p.fault, MSA_FAULT_PAGE_ID);
        page = -1;
    }
    const int slot = token % kPage;
    const int pairs = p.rot / 2;
    if (tid < pairs)
        turn(turns_of(p.inv_freq[tid]), position, s_cos[tid], s_sin[tid]);
    __syncthreads();

    // kinds one after the other: a lane's coefficients are a kind's
    const int half = p.rot / 16;  // lanes of a head that hold a first half of the rotated dims (pairs apart)
    const int partner = INTER ? sub : sub < half ? sub + half : sub < 2 * half ? sub - half : sub;
    for (int kind = 0; kind < 3; ++kind) {
        const int heads = kind == 0 ? (p.q ? p.q_heads : 0) : kind == 1 ? p.kv_heads : (p.v ? p.kv_heads : 0);
        if (!heads || (kind > 0 && page < 0))
            continue;
        const uint16_t *src = (kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                              row * (kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride) + sub * 8;
        const float *weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
        float A[8], B[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            A[j] = weight ? weight[sub * 8 + j] : 1.0f;
            B[j] = 0.0f;
        }
        if (kind < 2 && sub < 2 * half) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = INTER ? sub * 4 + j / 2 : (sub % half) * 8 + j;
                const float wp = weight ? weight[INTER ? sub * 8 + (j ^ 1) : partner * 8 + j] : 1.0f;
                const bool first = INTER ? j % 2 == 0 : sub < half;
                A[j] *= s_cos[at];
                B[j] = first ? -wp * s_sin[at] : wp * s_sin[at];
            }
        }
        for (int h0 = blockIdx.y * kAppendHeads; h0 < heads; h0 += gridDim.y * kAppendHeads) {
            const int h = h0 + tid / 16;
            const bool have = h < heads;
            const uint4 raw = have ? *reinterpret_cast<const uint4 *>(src + h * kDim) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            float y[8];
            if (kind < 2) {
                float x[8], xp[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[2 * j] = __uint_as_float(w[j] << 16);
                    x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                    const uint32_t o = INTER ? (w[j] << 16) | (w[j] >> 16)
                                             : __shfl_sync(0xffffffffu, w[j], (lane & 16) | partner);
                    xp[2 * j] = __uint_as_float(o << 16);
                    xp[2 * j + 1] = __uint_as_float(o & 0xffff0000u);
                }
                float inv = 1.0f;
                if (weight) {
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sum = fmaf(x[j], x[j], sum);
                    inv = rsqrtf(half_warp_sum(sum) * (1.0f / kDim) + p.eps);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = fmaf(x[j], A[j], xp[j] * B[j]) * inv;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    y[2 * j] = __uint_as_float(w[j] << 16);
                    y[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                }
            }
            if (kind == 0 || !FP8) {
                if (!have)
                    continue;
                uint16_t *dst = kind == 0 ? p.out_q + row * p.out_q_stride + h * kDim
                                          : reinterpret_cast<uint16_t *>(kind == 1 ? p.k_cache : p.v_cache) +
                                                page * (kind == 1 ? p.kc_stride : p.vc_stride)[0] +
                                                slot * (kind == 1 ? p.kc_stride : p.vc_stride)[1] +
                                                h * (kind == 1 ? p.kc_stride : p.vc_stride)[2];
                *reinterpret_cast<uint4 *>(dst + sub * 8) =
                    make_uint4(f32x2_to_bf16x2(y[0], y[1]), f32x2_to_bf16x2(y[2], y[3]), f32x2_to_bf16x2(y[4], y[5]),
                               f32x2_to_bf16x2(y[6], y[7]));
            } else {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    top = fmaxf(top, fabsf(y[j]));
                top = half_warp_max(top);
                const float unit = top < 6.018531076210112e-36f ? 0.0f : top / 448.0f;  // 2^-117: the quotient is normal
                const float inv = unit > 0.0f ? 1.0f / unit : 0.0f;
                if (!have)
                    continue;
                const int64_t *st = kind == 1 ? p.kc_stride : p.vc_stride;
                uint8_t *dst = (kind == 1 ? p.k_cache : p.v_cache) + page * st[0] + slot * st[1] + h * st[2];
                uint32_t c[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    c[j] = e4m3_pair(y[4 * j] * inv, y[4 * j + 1] * inv) |
                           static_cast<uint32_t>(e4m3_pair(y[4 * j + 2] * inv, y[4 * j + 3] * inv)) << 16;
                *reinterpret_cast<uint2 *>(dst + sub * 8) = unit > 0.0f ? make_uint2(c[0], c[1]) : make_uint2(0u, 0u);
                if (sub == 0)
                    (kind == 1 ? p.k_scale : p.v_scale)[(static_cast<int64_t>(page) * p.kv_heads + h) * kPage + slot] = unit;
            }
        }
    }
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
        (p.q && (p.q_stride % 8 || p.q_stride < qd || p.out_q_stride % 8 || p.out_q_stride < qd)))
        return MSA_ERR_INVALID_ARG;
    if (fp8 && (!p.k_scale || (values && !p.v_scale) || unaligned(p.k_scale, 16) || unaligned(p.v_scale, 16)))
        return MSA_ERR_INVALID_ARG;
    if (workspace_bytes < kHeaderBytes)
        return MSA_ERR_WORKSPACE_TOO_SMALL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return MSA_ERR_CUDA;
    const int sms = device_sms(dev);
    if (sms <= 0)
        return MSA_ERR_CUDA;
    for (int i = 0; i < 3; ++i) {
        p.kc_stride[i] = k_strides[i];
        p.vc_stride[i] = values ? v_strides[i] : 0;
    }
    p.fault = &static_cast<WorkspaceHeader *>(workspace)->fault;
    p.rows = total_rows;
    p.batch = batch;
    p.seq_limit = static_cast<int>(std::min<int64_t>(max_model_len, kPage * p.bt_stride));
    const int heads = std::max(p.q ? p.q_heads : 0, p.kv_heads);
    const int shares = (heads + kAppendHeads - 1) / kAppendHeads;
    const dim3 grid(static_cast<unsigned>(total_rows), static_cast<unsigned>(total_rows * 2 <= sms ? std::min(shares, 64) : 1));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (fp8)
        interleaved ? append_kernel<true, true><<<grid, kAppendThreads, 0, st>>>(p)
                    : append_kernel<true, false><<<grid, kAppendThreads, 0, st>>>(p);
    else
        interleaved ? append_kernel<false, true><<<grid, kAppendThreads, 0, st>>>(p)
                    : append_kernel<false, false><<<grid, kAppendThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
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

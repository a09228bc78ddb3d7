// Attention of all requests' query rows over the prefix they share: a dense
// product on the 5th-generation tensor cores.
//
// The rows of one KV head (batch * q_len * group of them) read the same keys, so
// they stand side by side as the M rows of S = Q K^T and O = P V.  A unit is
// (KV head, tile of 256 rows); the prefix's pages of all units, one after the
// other, are cut into one equal range a CTA, and a range's part of a unit goes
// to the workspace as (O / L, M + log2 L) in fp32; the kernel that walks each
// request's own pages joins the parts (block_attn.cuh), always in page order.
//
// Per page and 128-row tile: S (128 x 128, fp32) in tensor memory; a warpgroup
// with one thread a row takes the row's maximum, 2^(c s - m) and the sum, and
// writes the weights as bf16 over S; the second product reads them from there
// (A in tensor memory, V's page from shared memory with the dims contiguous:
// the B operand's transposed form).  Two tiles alternate, so that one is in the
// tensor cores while the other is in its softmax.  The reference m of a row is
// only moved (and O, L rescaled) when the maximum outgrows it by more than 2^8:
// weights then stay at most 2^8, which costs no precision in fp32 sums and bf16
// operands, and the rescaling of O in tensor memory becomes rare.
#pragma once

#include "block_attn.cuh"

namespace msa {

constexpr int kPrefixStages = 4;  // K and V tiles of two pages
constexpr int kPrefixThreads = 320;  // two softmax warpgroups, a TMA warp, an MMA warp
constexpr int kPrefixMaxGrid = 256;
constexpr float kPrefixLag = 8.0f;

struct PrefixAttnParams {
    CUtensorMap kmap, vmap;
    const uint16_t *q;
    const int32_t *prefix_table;
    const int32_t *prefix_len;
    PrefixParts parts;
    uint32_t *fault;
    int64_t q_stride, num_pages;
    float scale_log2;
};

struct PrefixSmem {
    uint64_t kv_full[kPrefixStages], kv_empty[kPrefixStages];
    uint64_t q_full[2], s_full[2], p_full[2], o_done[2];
    uint64_t drained;
    uint32_t tmem;
    int abort_flag;
};

constexpr size_t kPrefixSmemBytes = 1024 + 2 * kPageBytes + kPrefixStages * kPageBytes + sizeof(PrefixSmem);

// D[tmem] (+)= A[tmem] * B[smem] (kind::f16, cta_group::1): A's 128 rows lie in the lanes, two bf16 of K a column.
template <bool ACC>
__device__ __forceinline__ void umma_ts_f16(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc)
{
    asm volatile(
        "{\n"
        "  .reg .b64 bd;\n"
        "  mov.b64 bd, {%2, %5};\n"
        "  tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %3, %4;\n"
        "}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "n"(ACC ? 1 : 0), "r"(b_hi)
        : "memory");
}

// 32 consecutive 32-bit columns of one TMEM lane per thread (shape 32x32b).
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// V as B operand: N (the dims) contiguous in the 128-byte swizzle.  64 dims x 8 tokens make an atom of 1024 bytes;
// the next 64 dims are one half tile (16 KiB) on, the next 8 tokens one atom on.
__device__ __forceinline__ uint32_t umma_desc_v_lo(uint32_t saddr)
{
    return ((saddr >> 4) & 0x3FFFu) | (static_cast<uint32_t>(kHalfPageBytes >> 4) << 16);
}

__global__ void __launch_bounds__(kPrefixThreads, 1) prefix_attn_kernel(const __grid_constant__ PrefixAttnParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *kv = smem + 2 * kPageBytes;  // after the two Q tiles
    auto *ctl = reinterpret_cast<PrefixSmem *>(kv + kPrefixStages * kPageBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    griddep_launch_dependents();
    const int prefix = prefix_tokens(p.parts, p.prefix_len);
    const PrefixSplit split(p.parts, prefix, static_cast<int>(gridDim.x));
    if (prefix == 0 && *p.prefix_len != 0 && blockIdx.x == 0 && tid == 0)
        atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
    const int cta = blockIdx.x;
    if (cta >= split.ctas)
        return;
    const int P = split.pages;
    const int64_t lo = split.start(cta), hi = split.start(cta + 1);
    const int tiles = p.parts.tile_rows / 128;  // 128-row tiles of a unit: 1 or 2

    if (tid == 0) {
        for (int s = 0; s < kPrefixStages; ++s) {
            mbar_init(smem_addr(&ctl->kv_full[s]), 1);
            mbar_init(smem_addr(&ctl->kv_empty[s]), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_addr(&ctl->q_full[t]), 128);
            mbar_init(smem_addr(&ctl->s_full[t]), 1);
            mbar_init(smem_addr(&ctl->p_full[t]), 128);
            mbar_init(smem_addr(&ctl->o_done[t]), 1);
        }
        mbar_init(smem_addr(&ctl->drained), 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_addr(&ctl->tmem), 512);
        tmem_relinquish_alloc_permit();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem;  // columns 0, 128: S (and the weights); 256, 384: O

    if (warp == 8) {
        // ---- K and V tiles, page after page ----
        bool alive = true;
        uint32_t it = 0;
        int pages = -1;
        for (int64_t x = lo; x < hi && alive; ++x) {
            const int i = static_cast<int>(x - lo);
            if ((i & 31) == 0) {
                pages = -1;
                if (x + lane < hi) {
                    pages = p.prefix_table[(x + lane) % P];
                    if (pages < 0 || pages >= p.num_pages) {
                        pages = -1;
                        atomicOr(p.fault, MSA_FAULT_PAGE_ID);
                    }
                }
            }
            const int page = __shfl_sync(0xffffffffu, pages, i & 31);
            const int h = static_cast<int>(x / P) / p.parts.head_tiles;
            for (int kvi = 0; kvi < 2; ++kvi, ++it) {
                const int s = static_cast<int>(it % kPrefixStages);
                if (it >= kPrefixStages)
                    alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->kv_empty[s]),
                                      (it / kPrefixStages + 1) & 1);
                if (!alive)
                    break;
                if (lane == 0) {
                    const uint32_t bar = smem_addr(&ctl->kv_full[s]), dst = smem_addr(kv) + s * kPageBytes;
                    if (page < 0) {
                        mbar_arrive(bar);
                    } else {
                        const CUtensorMap *map = kvi ? &p.vmap : &p.kmap;
                        mbar_arrive_expect_tx(bar, kPageBytes);
                        tma_load_4d(dst, map, 0, 0, h, page, bar);
                        tma_load_4d(dst + kHalfPageBytes, map, 64, 0, h, page, bar);
                    }
                }
            }
        }
        // the copies in flight land before the CTA may end, also where another role gave up
        for (uint32_t j = it >= kPrefixStages ? it - kPrefixStages : 0; j < it; ++j)
            mbar_wait(smem_addr(&ctl->kv_full[j % kPrefixStages]), (j / kPrefixStages) & 1);
    } else if (warp == 9) {
        // ---- one thread issues both products of both tiles ----
        if (lane == 0) {
            constexpr uint32_t idesc_s = umma_idesc_bf16_f32(128, 128);
            constexpr uint32_t idesc_o = umma_idesc_bf16_f32(128, 128) | (1u << 16);  // B with N contiguous
            volatile int *abort_flag = &ctl->abort_flag;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (*abort_flag || !mbar_wait(smem_addr(bar), parity)) {
                    if (!*abort_flag)
                        atomicOr(p.fault, MSA_FAULT_TIMEOUT);
                    *abort_flag = 1;
                    return false;
                }
                return true;
            };
            auto scores = [&](int t, int s) {
                const uint32_t a = umma_desc_lo(smem_addr(smem) + t * kPageBytes);
                const uint32_t b = umma_desc_lo(smem_addr(kv) + s * kPageBytes);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t off = ((ks >> 2) * kHalfPageBytes + (ks & 3) * 32) >> 4;
                    if (ks == 0)
                        umma_f16<false>(tmem + t * 128, a + off, b + off, idesc_s);
                    else
                        umma_f16<true>(tmem + t * 128, a + off, b + off, idesc_s);
                }
                umma_commit(smem_addr(&ctl->s_full[t]));
            };
            bool alive = true;
            uint32_t it = 0, seg = 0;
            for (int64_t x = lo; x < hi && alive; ++seg) {
                const int n = static_cast<int>(min(hi, (x / P + 1) * P) - x);
                x += n;
                for (int t = 0; t < tiles && alive; ++t)
                    alive = wait(&ctl->q_full[t], seg & 1);
                if (alive)
                    alive = wait(&ctl->kv_full[(2 * it) % kPrefixStages], (2 * it / kPrefixStages) & 1);
                if (!alive)
                    break;
                tc_fence_after_sync();
                for (int t = 0; t < tiles; ++t)
                    scores(t, (2 * it) % kPrefixStages);
                umma_commit(smem_addr(&ctl->kv_empty[(2 * it) % kPrefixStages]));
                for (int j = 0; j < n && alive; ++j, ++it) {
                    const int sv = (2 * it + 1) % kPrefixStages, next = (2 * it + 2) % kPrefixStages;
                    for (int t = 0; t < tiles && alive; ++t) {
                        alive = wait(&ctl->p_full[t], it & 1);
                        if (alive && t == 0)
                            alive = wait(&ctl->kv_full[sv], ((2 * it + 1) / kPrefixStages) & 1);
                        if (!alive)
                            break;
                        tc_fence_after_sync();
                        const uint32_t b = umma_desc_v_lo(smem_addr(kv) + sv * kPageBytes);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {  // 16 tokens each: 8 columns of weights, two atoms of V
                            const uint32_t bk = b + ((ks * 2048) >> 4);
                            if (ks == 0 && j == 0)
                                umma_ts_f16<false>(tmem + 256 + t * 128, tmem + t * 128, bk, kUmmaDescHi, idesc_o);
                            else
                                umma_ts_f16<true>(tmem + 256 + t * 128, tmem + t * 128 + ks * 8, bk, kUmmaDescHi, idesc_o);
                        }
                        umma_commit(smem_addr(&ctl->o_done[t]));
                        if (t == tiles - 1)
                            umma_commit(smem_addr(&ctl->kv_empty[sv]));
                        // the next page's scores overwrite the weights that this product reads: MMAs of one
                        // thread run in the order of their issue
                        if (j + 1 < n) {
                            if (t == 0)
                                alive = wait(&ctl->kv_full[next], ((2 * it + 2) / kPrefixStages) & 1);
                            if (!alive)
                                break;
                            scores(t, next);
                            if (t == tiles - 1)
                                umma_commit(smem_addr(&ctl->kv_empty[next]));
                        }
                    }
                }
            }
            umma_commit(smem_addr(&ctl->drained));  // nothing in flight when the tensor memory is freed
            mbar_wait(smem_addr(&ctl->drained), 0);
        }
        __syncwarp();
    } else if (warp / 4 < tiles) {
        // ---- softmax: one thread a row ----
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // (32 * (warp % 4)) << 16
        const uint32_t ts = tmem + t * 128 + lanes, to = tmem + 256 + t * 128 + lanes;
        const float c = p.scale_log2;
        bool alive = true;
        uint32_t it = 0;
        for (int64_t x = lo; x < hi; ) {
            const int u = static_cast<int>(x / P), j0 = static_cast<int>(x % P);
            const int n = static_cast<int>(min(hi - x, static_cast<int64_t>(P - j0)));
            x += n;
            const int h = u / p.parts.head_tiles;
            const int nrow = (u % p.parts.head_tiles) * p.parts.tile_rows + t * 128 + row;
            const bool have = nrow < p.parts.rows;
            {
                const uint16_t *src = p.q + static_cast<int64_t>(nrow / p.parts.group) * p.q_stride +
                                      (h * p.parts.group + nrow % p.parts.group) * kDim;
                uint4 v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[i] = have ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0u, 0u, 0u, 0u);
                uint8_t *dst = smem + t * kPageBytes + row * 128;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    *reinterpret_cast<uint4 *>(dst + (i >> 3) * kHalfPageBytes + (((i & 7) ^ (row & 7)) << 4)) = v[i];
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            mbar_arrive(smem_addr(&ctl->q_full[t]));
            float m = -INFINITY, l = 0.0f;
            int page = p.prefix_table[j0];
            for (int j = 0; j < n && alive; ++j, ++it) {
                // tokens of the page that count
                const int valid = page < 0 || page >= p.num_pages ? 0 : min(kPage, prefix - (j0 + j) * kPage);
                if (j + 1 < n)
                    page = p.prefix_table[j0 + j + 1];
                alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->s_full[t]), it & 1);
                if (!alive)
                    break;
                tc_fence_after_sync();
                uint32_t s[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    tmem_ld32(ts + q * 32, s[q]);
                tmem_wait_ld(s[0]);
                tmem_regs_ready(s[1]);
                tmem_regs_ready(s[2]);
                tmem_regs_ready(s[3]);
                if (valid < kPage) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (q * 32 + i >= valid)
                                s[q][i] = 0xff800000u;
                    if (t == 0) {
                        // what lies in V past the tokens is no data: zero it (0 x NaN is NaN)
                        const int sv = (2 * it + 1) % kPrefixStages;
                        alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->kv_full[sv]),
                                          ((2 * it + 1) / kPrefixStages) & 1);
                        if (!alive)
                            break;
                        if (row >= valid) {
                            uint8_t *at = kv + sv * kPageBytes + row * 128;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                *reinterpret_cast<uint4 *>(at + (i >> 3) * kHalfPageBytes + (i & 7) * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                }
                float mx[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mx[q] = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        mx[q] = fmaxf(mx[q], __uint_as_float(s[q][i]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                if (j == 0) {
                    m = top;
                } else if (__any_sync(0xffffffffu, top > m + kPrefixLag)) {
                    const float to_m = fmaxf(m, top), f = rescale(m, to_m);
                    m = to_m;
                    l *= f;
                    alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->o_done[t]), (it - 1) & 1);
                    if (!alive)
                        break;
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t o[32];
                        tmem_ld32(to + q * 32, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st32(to + q * 32, o);
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                uint32_t w[2][32];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float a = exp2_approx(fmaf(__uint_as_float(s[q][i]), c, -ref));
                        const float b = exp2_approx(fmaf(__uint_as_float(s[q][i + 1]), c, -ref));
                        sum[q] += a + b;
                        w[q >> 1][(q & 1) * 16 + i / 2] = f32x2_to_bf16x2(a, b);
                    }
                tmem_st32(ts, w[0]);
                tmem_st32(ts + 32, w[1]);
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive(smem_addr(&ctl->p_full[t]));
            }
            // ---- the range's part of the unit ----
            if (alive)
                alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->o_done[t]), (it - 1) & 1);
            tc_fence_after_sync();
            const int64_t slot = static_cast<int64_t>(cta) + u;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            if (alive) {
                // through the tile's Q (every product with it is done), 64 dims at a time, each warp its 32 rows:
                // a thread holds a row, a store of a warp should cover whole lines
                float *part = p.parts.o + (slot * p.parts.tile_rows + t * 128 + (row & ~31)) * kDim;
                uint8_t *turn = smem + t * kPageBytes + (row & ~31) * 256;
                const int left = p.parts.rows - (nrow & ~31);  // rows of the warp that exist
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t o[32];
                        tmem_ld32(to + half * 64 + q * 32, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(turn + lane * 256 + (((q * 8 + i / 4) ^ (lane & 7)) << 4)) =
                                make_float4(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv,
                                            __uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int r = lane >> 4; r < 32; r += 2)
                        if (r < left)
                            *reinterpret_cast<float4 *>(part + r * kDim + half * 64 + (lane & 15) * 4) =
                                *reinterpret_cast<const float4 *>(turn + r * 256 + (((lane & 15) ^ (r & 7)) << 4));
                }
                __syncwarp();
            }
            // +inf marks a part that is not whole
            p.parts.lse[slot * p.parts.tile_rows + t * 128 + row] =
                !alive ? INFINITY : l == 0.0f ? -INFINITY : m + log2f(l);
        }
        tc_fence_before_sync();
    }
    __syncthreads();
    if (warp == 9)
        tmem_dealloc(tmem, 512);
}

}  // namespace msa

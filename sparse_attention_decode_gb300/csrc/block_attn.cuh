// Attention of a few query rows over a list of 128-token cache pages: the blocks
// selected for them, or (OWN) all pages of their request, whose result is then one
// part of the attention with a shared prefix.
//
// Mathematics.  For a row n with query q_n and the valid tokens T_n,
//     s = scale * q_n . K[t],   out_n = sum_T 2^(c s - M) V[t] / L,
//     M = max_T c s,  L = sum_T 2^(c s - M),  c = log2 e,  lse_n = (M + log2 L) ln 2,
// taken page by page with the running maximum and sum of a softmax: a part
// (M1, L1, O1) joins another by O = 2^(M1-M) O1 + 2^(M2-M) O2 (L alike), with
// M = max(M1, M2).  (E4M3: as (M1, L1, O1 / L1), whose share is 2^(M1-M) L1 / L: no
// larger than V itself, whatever the scales.)  M, L and O stay in fp32; the weights
// 2^(c s - M) are rounded once, to the operand type of the second product (bf16 beside a bf16 cache,
// f16 beside an E4M3 one), after L has taken them in full.
//
// What bounds it: every K and V byte is used by the 1..64 rows of one KV head
// only, so the cache stream does (64 KiB a page in bf16).  Hence TMA into a ring
// of tiles with two CTAs an SM (192 KiB in flight an SM), mma.sync on 16-row
// tiles read by ldmatrix (the tensor work of 16 rows is a third of the stream
// time; the 128-row tiles of tcgen05 would be filled to an eighth), and a
// cluster of up to 8 CTAs that splits one list when there are few: the parts
// join through distributed shared memory, in cluster-rank order, so there is one
// launch, no scratch, and the same result each time.  256 requests x 4 heads x 16
// blocks (1.05 GB): 166-168 us, 0.93 of the copy rate.  Few requests are bound by
// latency: of one request's 8 us, 1.3 are the length, ids and table, 1.3 the first
// tile, 2 two pages (a page alone on an SM takes a CTA 1 us, two CTAs 1.28 each), 2.5
// the parts' way to the output.
//
// Draft positions walk a list each: 32 requests x 4 positions x 4 x 16 heads read 537
// MB of which 160 are distinct, 56 us (E4M3 66).  E4M3, 32 requests: 22.4 us for 69 MB;
// neither the stream (0.36 of DRAM's cycles), the MMAs (0.14) nor the issue slots
// (0.27) are full: 256 CTAs stand in 304 places, so that 104 SMs walk 16 pages and 48
// walk 8, and the chain of one request is around them.  256 requests: 120 us, 0.67 of
// the copy rate.  Groups of 17 to 64 rows keep more than their registers (spills of 20
// to 52 bytes, E4M3 76 to 104): 64 requests x 4 x 32 heads 55 us (E4M3 67) for 266 MB
// (139), x 4 x 64 heads 91 (115).
#pragma once

#include <algorithm>
#include <cmath>

#include "attn_common.cuh"
#include "attn_ptx.cuh"
#include "host_util.cuh"
#include "keys.cuh"
#include "layout.cuh"
#include "tcgen05.cuh"

#include "msa_attention.h"

namespace msa {

// Tiles of the cache: bf16 as two 16 KiB halves of 64 dims, E4M3 as one 16 KiB
// tile and its 128 per-token scales; 128-byte rows in the TMA 128-byte swizzle.
struct AttnBf16 {
    static constexpr bool kFp8 = false;
    static constexpr int kTileBytes = kPageBytes;
    static constexpr int kScaleBytes = 0;
    static constexpr int kStages = 3;
};
struct AttnFp8 {
    static constexpr bool kFp8 = true;
    static constexpr int kTileBytes = kPage * kDim;
    static constexpr int kScaleBytes = kPage * 4;
    static constexpr int kStages = 6;
};

constexpr int kAttnWarps = 4;  // consumer warps; one producer warp after them
constexpr int kAttnThreads = 32 * (kAttnWarps + 1);
constexpr int kAttnMaxRows = 64;  // rows of one unit (query heads of a KV head): 1, 2 or 4 tiles of 16
constexpr int kAttnOStride = kDim + 4;  // fp32 row stride of a partial O in shared memory (bank spread)

struct BlockAttnParams {
    CUtensorMap kmap, vmap;  // [page][head][token][dim], box 1 x 1 x 128 x (64 bf16 | 128 E4M3)
    const uint16_t *q;
    const float *kscale, *vscale;  // E4M3: [page, head, 128]
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *ids;  // selected blocks [rows, sel_heads, k]
    uint16_t *out;
    float *part;  // OWN: in place of out, fp32 [rows, heads, 128]
    float *lse;   // optional; OWN: required, in log2 units
    float *mass;  // optional: [rows, kv heads, k]
    uint32_t *fault;
    int64_t q_stride;  // elements between query rows
    int64_t bt_stride;
    int64_t num_pages;
    int batch, q_len, kv_heads, sel_heads, group, k, seq_limit;
    int row_tiles;  // OWN: tiles of kAttnMaxRows rows that a request's q_len * group are cut into
    float scale_log2;
    int withhold;  // test of the bounded waits: the producer loads and signals no page
};

template <class F>
struct BlockAttnSmem {
    uint64_t full[F::kStages], empty[F::kStages];
    int own_base[F::kStages];     // OWN: first token of the tile's page, or -1: a page that is skipped
    int list_page[MSA_MAX_TOPK];  // this CTA's valid selected blocks in slot order
    int list_base[MSA_MAX_TOPK];
    int list_slot[MSA_MAX_TOPK];
    int count;                    // pages this CTA walks
    int abort_flag;
    float wm[kAttnWarps][16], wl[kAttnWarps][16];  // each warp's rows: running maximum (log2 units) and sum
    float cm[kAttnMaxRows], cl[kAttnMaxRows];      // the CTA's rows, read by the whole cluster
    float rm[kAttnMaxRows], rinv[kAttnMaxRows];    // final maximum and 1 / sum (0: nothing)
    float fac[8][kAttnMaxRows];                    // what each rank's part of a row is multiplied by
};

// Mass scratch: [page of this CTA][slice * rows] of (sum, maximum at that time); 64 entries a page.  Two CTAs fit on
// an SM with 24 pages of it (E4M3: 18): an unsplit list of 32 blocks has one (160 requests x 4 heads: 241 us, without
// the mass 208; E4M3 218 and 142).
__host__ __device__ constexpr size_t block_attn_mass_bytes(int pages) { return static_cast<size_t>(pages) * 64 * 8; }

template <class F>
__host__ __device__ constexpr size_t block_attn_smem(int mass_pages)
{
    return 1024 + static_cast<size_t>(F::kStages) * (F::kTileBytes + F::kScaleBytes) + sizeof(BlockAttnSmem<F>) +
           block_attn_mass_bytes(mass_pages);
}

__device__ __forceinline__ void consumer_barrier()
{
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kAttnWarps) : "memory");
}

// E4M3: the unit of a row's (weight x V scale) products, the largest power of two <= v, and its inverse; v within
// [2^-112, 2^126] keeps both, and the inverse times kVTop, normal.  In f16 such a product is below 4 kVTop.
constexpr float kVTop = 8192.0f;                   // 2^13
constexpr float kVLeast = 1.925929944387236e-34f;  // 2^-112
constexpr float kVMost = 8.507059173023462e37f;    // 2^126
__device__ __forceinline__ float v_unit(float v) { return __uint_as_float(__float_as_uint(v) & 0x7f800000u); }
__device__ __forceinline__ float v_unit_inverse(float v) { return __uint_as_float(0x7f000000u - (__float_as_uint(v) & 0x7f800000u)); }

// MT: 16-row tiles of a unit (the four warps are MT tiles x 4 / MT slices of a
// page's tokens).  A unit is (query row, KV head) with its group's rows, or, OWN,
// (request, row tile, KV head) with the rows of all positions.
template <class F, int MT, bool OWN>
__global__ void __launch_bounds__(kAttnThreads, 2) block_attn_kernel(const __grid_constant__ BlockAttnParams p)
{
    constexpr int KS = kAttnWarps / MT;      // slices of a page
    constexpr int kSlice = kPage / KS;       // tokens of a slice
    constexpr int kChunks = kSlice / 32;     // 32 tokens at a time
    constexpr uint32_t kStageBytes = F::kTileBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *scales = reinterpret_cast<float *>(smem + F::kStages * F::kTileBytes);
    auto *ctl = reinterpret_cast<BlockAttnSmem<F> *>(smem + F::kStages * (F::kTileBytes + F::kScaleBytes));
    float2 *mass_part = reinterpret_cast<float2 *>(ctl + 1);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (OWN)
        griddep_launch_dependents();  // the join may take its place; it waits for this grid's end
    const int S = static_cast<int>(cluster_nctarank()), crank = static_cast<int>(cluster_ctarank());
    const int unit = static_cast<int>(blockIdx.x) / S;
    const int h = unit % p.kv_heads, owner = unit / p.kv_heads;  // KV head; query row, or request and row tile
    const int b = owner / (OWN ? p.row_tiles : p.q_len);
    const int row0 = OWN ? owner % p.row_tiles * kAttnMaxRows : 0;
    const int rows = OWN ? min(p.q_len * p.group - row0, kAttnMaxRows) : p.group;
    // row n of the unit: its position in the request, and its place among [query rows, query heads]
    auto position = [&](int n) { return OWN ? (row0 + n) / p.group : owner % p.q_len; };
    auto place = [&](int n) {
        const int64_t q = OWN ? static_cast<int64_t>(b) * p.q_len + (row0 + n) / p.group : owner;
        return (q * p.kv_heads + h) * p.group + (OWN ? (row0 + n) % p.group : n);
    };

    const int L = p.seq_lens[b];
    // a lane's selected block, asked for together with the length
    const int sel_id = !OWN && warp == kAttnWarps && lane < p.k
                           ? p.ids[(static_cast<int64_t>(owner) * p.sel_heads + h / (p.kv_heads / p.sel_heads)) * p.k + lane]
                           : -1;
    const bool bad_len = L < 0 || L > p.seq_limit;
    if (tid == 0 && bad_len)
        atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
    const int len = bad_len ? 0 : L;  // the request's tokens: what lies past them is no data
    auto visible = [&](int i) { return max(0, len - (p.q_len - 1 - i)); };  // tokens position i sees

    if (tid == 0) {
        for (int s = 0; s < F::kStages; ++s) {
            mbar_init(smem_addr(&ctl->full[s]), 1);
            mbar_init(smem_addr(&ctl->empty[s]), kAttnWarps);
        }
        ctl->abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kAttnWarps) {
        if (lane < 2)
            prefetch_tensormap(lane ? &p.vmap : &p.kmap);
        if (OWN) {
            const int nb = pages_of(len);
            if (lane == 0)
                ctl->count = nb > crank ? (nb - crank + S - 1) / S : 0;
        } else {
            const int nb = pages_of(visible(position(0)));
            const int id = sel_id;
            int page = -1;
            bool ok = id >= 0;
            if (ok && id >= nb) {
                ok = false;
                if (!bad_len)
                    atomicOr(p.fault, MSA_FAULT_BLOCK_ID);
            }
            if (ok) {
                page = p.block_table[static_cast<int64_t>(b) * p.bt_stride + id];
                if (page < 0 || page >= p.num_pages) {
                    ok = false;
                    atomicOr(p.fault, MSA_FAULT_PAGE_ID);
                }
            }
            const uint32_t got = __ballot_sync(0xffffffffu, ok);
            const int at = __popc(got & ((1u << lane) - 1u));
            if (ok && at % S == crank) {
                ctl->list_page[at / S] = page;
                ctl->list_base[at / S] = id * kPage;
                ctl->list_slot[at / S] = lane;
            }
            const int n = __popc(got);
            if (lane == 0)
                ctl->count = n > crank ? (n - crank + S - 1) / S : 0;
            if (p.mass && lane < p.k && !ok && crank == 0)
                p.mass[(static_cast<int64_t>(owner) * p.kv_heads + h) * p.k + lane] = 0.0f;
        }
    }
    __syncthreads();
    const int count = ctl->count;

    if (warp == kAttnWarps) {
        // ---- producer: K and V tile of each page, one stage each ----
        bool alive = true;
        uint32_t it = 0;
        int pages = -1;
        for (int i = 0; i < count && alive; ++i) {
            int page;
            if (OWN) {
                if ((i & 31) == 0) {  // a lane's share of the next 32 pages
                    pages = -1;
                    if (i + lane < count)
                        pages = p.block_table[static_cast<int64_t>(b) * p.bt_stride + crank + (i + lane) * S];
                    if (i + lane < count && (pages < 0 || pages >= p.num_pages)) {
                        pages = -1;
                        atomicOr(p.fault, MSA_FAULT_PAGE_ID);
                    }
                }
                page = __shfl_sync(0xffffffffu, pages, i & 31);
            } else {
                page = ctl->list_page[i];
            }
            for (int kv = 0; kv < 2; ++kv, ++it) {
                const int s = static_cast<int>(it % F::kStages);
                const uint32_t bar = smem_addr(&ctl->full[s]);
                if (it >= F::kStages)
                    alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->empty[s]), (it / F::kStages + 1) & 1, p.withhold);
                if (!alive)
                    break;
                if (lane == 0 && !p.withhold) {
                    if (OWN) {
                        ctl->own_base[s] = page < 0 ? -1 : (crank + i * S) * kPage;
                        if (page < 0) {
                            mbar_arrive(bar);
                            continue;
                        }
                    }
                    const CUtensorMap *map = kv ? &p.vmap : &p.kmap;
                    const uint32_t dst = smem_addr(smem) + s * kStageBytes;
                    mbar_arrive_expect_tx(bar, F::kTileBytes + F::kScaleBytes);
                    tma_load_4d(dst, map, 0, 0, h, page, bar);
                    if (F::kFp8)
                        bulk_load(smem_addr(scales + s * kPage),
                                  (kv ? p.vscale : p.kscale) + (static_cast<int64_t>(page) * p.kv_heads + h) * kPage,
                                  F::kScaleBytes, bar);
                    else
                        tma_load_4d(dst + kHalfPageBytes, map, 64, 0, h, page, bar);
                }
            }
        }
        // the copies in flight land before the CTA may end, also where a consumer gave up
        for (uint32_t j = it >= F::kStages ? it - F::kStages : 0; j < it && !p.withhold; ++j)
            mbar_wait(smem_addr(&ctl->full[j % F::kStages]), (j / F::kStages) & 1);
    } else {
        // ---- consumers ----
        const int mt = warp % MT, slice = warp / MT;
        const int g = lane >> 2, t = lane & 3;
        // query fragments of rows g and g + 8, zero past the unit's rows
        uint32_t qa[8][4];
        float undo0 = 1.0f, undo1 = 1.0f;
        int sees0, sees1;  // tokens the two rows see
        {
            float am0 = 0.0f, am1 = 0.0f;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int n = mt * 16 + g + 8 * r;
                const bool have = n < rows;
                (r ? sees1 : sees0) = have ? visible(position(n)) : 0;
                const int64_t qr = OWN ? static_cast<int64_t>(b) * p.q_len + position(n) : owner;
                const uint16_t *src = p.q + qr * p.q_stride + (h * p.group + (OWN ? (row0 + n) % p.group : n)) * kDim;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    // bf16: columns 2t, 2t+1 and 2t+8, 2t+9 of each 16; E4M3: 4t .. 4t+3, as the codes' bytes lie
                    const int c0 = 16 * ks + (F::kFp8 ? 4 * t : 2 * t), c1 = 16 * ks + (F::kFp8 ? 4 * t + 2 : 2 * t + 8);
                    qa[ks][r] = have ? *reinterpret_cast<const uint32_t *>(src + c0) : 0u;
                    qa[ks][2 + r] = have ? *reinterpret_cast<const uint32_t *>(src + c1) : 0u;
                    if (F::kFp8) {
                        const float a = fmaxf(fmaxf(fabsf(bf16_lo(qa[ks][r])), fabsf(bf16_hi(qa[ks][r]))),
                                              fmaxf(fabsf(bf16_lo(qa[ks][2 + r])), fabsf(bf16_hi(qa[ks][2 + r]))));
                        (r ? am1 : am0) = fmaxf(r ? am1 : am0, a);
                    }
                }
            }
            if (F::kFp8) {
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    am0 = fmaxf(am0, __shfl_xor_sync(0xffffffffu, am0, o));
                    am1 = fmaxf(am1, __shfl_xor_sync(0xffffffffu, am1, o));
                }
                const float f0 = q_row_factor(am0, &undo0), f1 = q_row_factor(am1, &undo1);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float f = (r & 1) ? f1 : f0;
                        qa[ks][r] = f32x2_to_f16x2(bf16_lo(qa[ks][r]) * f, bf16_hi(qa[ks][r]) * f);
                    }
            }
        }
        float o[16][4];
#pragma unroll
        for (int d = 0; d < 16; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[d][e] = 0.0f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
        // E4M3: a row's o is held in units of a power of two next to the largest (weight x V scale) met so far, at the
        // running maximum; v0, v1 follow that product and the units their exponents
        float v0 = kVLeast, v1 = kVLeast;

        bool alive = true;
        uint32_t it = 0;
        for (int i = 0; i < count && alive; ++i, it += 2) {
            const int s_k = static_cast<int>(it % F::kStages), s_v = static_cast<int>((it + 1) % F::kStages);
            alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->full[s_k]), (it / F::kStages) & 1, p.withhold);
            if (!alive)
                break;
            const int base = OWN ? ctl->own_base[s_k] : ctl->list_base[i];
            float ps0 = 0.0f, ps1 = 0.0f;  // this page's weight, at the running maximum
            const uint32_t kt = smem_addr(smem) + s_k * kStageBytes, vt = smem_addr(smem) + s_v * kStageBytes;
            bool v_waited = false, k_held = true;
#pragma unroll 1
            for (int ch = 0; ch < kChunks; ++ch) {
                const int tok = slice * kSlice + ch * 32;  // first token of the chunk in the page
                if (OWN && base < 0)
                    break;
                // S = Q K^T: 16 rows x 32 tokens
                float s[4][4];
#pragma unroll
                for (int f = 0; f < 4; ++f)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[f][e] = 0.0f;
                if (!F::kFp8) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                        for (int f = 0; f < 4; f += 2) {
                            const int row = tok + f * 8 + (lane & 7) + ((lane >> 4) << 3);
                            const int chunk = (ks & 3) * 2 + ((lane >> 3) & 1);
                            uint32_t r[4];
                            ldsm_x4(r, kt + (ks >> 2) * kHalfPageBytes + row * 128 + ((chunk ^ (row & 7)) << 4));
                            mma_bf16_16816(s[f], qa[ks], r[0], r[1]);
                            mma_bf16_16816(s[f + 1], qa[ks], r[2], r[3]);
                        }
                } else {
#pragma unroll
                    for (int f = 0; f < 4; ++f)
#pragma unroll
                        for (int ks = 0; ks < 8; ks += 4) {
                            const int row = tok + f * 8 + (lane & 7);
                            const int chunk = ks + (lane >> 3);
                            uint32_t r[4];
                            ldsm_x4(r, kt + row * 128 + ((chunk ^ (row & 7)) << 4));
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                mma_f16_16816(s[f], qa[ks + u], e4m3x2_to_f16x2(static_cast<uint16_t>(r[u] & 0xffffu)),
                                              e4m3x2_to_f16x2(static_cast<uint16_t>(r[u] >> 16)));
                        }
                    const float *ksc = scales + s_k * kPage;
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const float2 sc = *reinterpret_cast<const float2 *>(ksc + tok + f * 8 + 2 * t);
                        s[f][0] *= sc.x * undo0;
                        s[f][1] *= sc.y * undo0;
                        s[f][2] *= sc.x * undo1;
                        s[f][3] *= sc.y * undo1;
                    }
                }
                if (ch == kChunks - 1) {  // K's tile is free for the next page while this one's weights are worked on
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&ctl->empty[s_k]));
                    k_held = false;
                }
                const int left0 = sees0 - base - tok, left1 = sees1 - base - tok;  // visible tokens of the chunk
                if (min(left0, left1) < 32) {
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const int c = f * 8 + 2 * t;
                        s[f][0] = c < left0 ? s[f][0] : -INFINITY;
                        s[f][1] = c + 1 < left0 ? s[f][1] : -INFINITY;
                        s[f][2] = c < left1 ? s[f][2] : -INFINITY;
                        s[f][3] = c + 1 < left1 ? s[f][3] : -INFINITY;
                    }
                }
                float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    x0 = fmaxf(x0, fmaxf(s[f][0], s[f][1]));
                    x1 = fmaxf(x1, fmaxf(s[f][2], s[f][3]));
                }
#pragma unroll
                for (int q = 1; q < 4; q <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, q));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, q));
                }
                const float n0 = fmaxf(m0, x0 * p.scale_log2), n1 = fmaxf(m1, x1 * p.scale_log2);
                float a0 = rescale(m0, n0), a1 = rescale(m1, n1);
                m0 = n0;
                m1 = n1;
                l0 *= a0;
                l1 *= a1;
                ps0 *= a0;
                ps1 *= a1;
                const float z0 = n0 == -INFINITY ? 0.0f : n0, z1 = n1 == -INFINITY ? 0.0f : n1;
                float r0 = 0.0f, r1 = 0.0f;
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    s[f][0] = exp2_approx(fmaf(s[f][0], p.scale_log2, -z0));
                    s[f][1] = exp2_approx(fmaf(s[f][1], p.scale_log2, -z0));
                    s[f][2] = exp2_approx(fmaf(s[f][2], p.scale_log2, -z1));
                    s[f][3] = exp2_approx(fmaf(s[f][3], p.scale_log2, -z1));
                    r0 += s[f][0] + s[f][1];
                    r1 += s[f][2] + s[f][3];
                }
                ps0 += r0;
                ps1 += r1;
                l0 += r0;
                l1 += r1;
                if (!v_waited) {
                    alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->full[s_v]), ((it + 1) / F::kStages) & 1, p.withhold);
                    v_waited = true;
                    if (!alive)
                        break;
                }
                const int vleft = len - base - tok;  // tokens of the chunk that are data
                uint32_t pa[2][4];
                if (!F::kFp8) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        pa[j][0] = f32x2_to_bf16x2(s[2 * j][0], s[2 * j][1]);
                        pa[j][1] = f32x2_to_bf16x2(s[2 * j][2], s[2 * j][3]);
                        pa[j][2] = f32x2_to_bf16x2(s[2 * j + 1][0], s[2 * j + 1][1]);
                        pa[j][3] = f32x2_to_bf16x2(s[2 * j + 1][2], s[2 * j + 1][3]);
                    }
                } else {
                    // Weights times V's per-token scales in f16, relative to the largest such product of the row: in
                    // [2^13, 2^14) at most, so that products down to 2^-28 of it keep f16's 11 bits (down to 2^-38 some).
                    // Relative to the largest scale alone, a token with a large scale and no weight would take the bits
                    // of all others.
                    const float *vsc = scales + s_v * kPage;
                    float2 sc[4];
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        sc[f] = *reinterpret_cast<const float2 *>(vsc + tok + f * 8 + 2 * t);
                    if (vleft < 32) {
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            const int c = f * 8 + 2 * t;
                            sc[f].x = c < vleft ? sc[f].x : 0.0f;
                            sc[f].y = c + 1 < vleft ? sc[f].y : 0.0f;
                        }
                    }
                    float x0 = 0.0f, x1 = 0.0f;
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        s[f][0] *= sc[f].x;
                        s[f][1] *= sc[f].y;
                        s[f][2] *= sc[f].x;
                        s[f][3] *= sc[f].y;
                        x0 = fmaxf(x0, fmaxf(fabsf(s[f][0]), fabsf(s[f][1])));
                        x1 = fmaxf(x1, fmaxf(fabsf(s[f][2]), fabsf(s[f][3])));
                    }
#pragma unroll
                    for (int q = 1; q < 4; q <<= 1) {
                        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, q));
                        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, q));
                    }
                    const float y0 = v_unit(v0), y1 = v_unit(v1);
                    v0 = fminf(fmaxf(fmaxf(v0 * a0, x0), kVLeast), kVMost);
                    v1 = fminf(fmaxf(fmaxf(v1 * a1, x1), kVLeast), kVMost);
                    const float i0 = v_unit_inverse(v0), i1 = v_unit_inverse(v1);
                    a0 = a0 * y0 * i0;  // o from the units so far to the new ones
                    a1 = a1 * y1 * i1;
                    const float w0 = i0 * kVTop, w1 = i1 * kVTop;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        pa[j][0] = f32x2_to_f16x2(s[2 * j][0] * w0, s[2 * j][1] * w0);
                        pa[j][1] = f32x2_to_f16x2(s[2 * j][2] * w1, s[2 * j][3] * w1);
                        pa[j][2] = f32x2_to_f16x2(s[2 * j + 1][0] * w0, s[2 * j + 1][1] * w0);
                        pa[j][3] = f32x2_to_f16x2(s[2 * j + 1][2] * w1, s[2 * j + 1][3] * w1);
                    }
                }
                if (__any_sync(0xffffffffu, a0 != 1.0f || a1 != 1.0f)) {
#pragma unroll
                    for (int d = 0; d < 16; ++d) {
                        o[d][0] *= a0;
                        o[d][1] *= a0;
                        o[d][2] *= a1;
                        o[d][3] *= a1;
                    }
                }
                // O += P V; tokens that are not data are zeroed in V's fragments (0 x NaN is NaN)
                const bool cut = vleft < 32;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = tok + j * 16 + (lane & 15);
                    const int tk = j * 16 + 2 * t;  // tokens of b0: tk, tk + 1; of b1: tk + 8, tk + 9
                    const uint32_t k0 = (tk < vleft ? 0xffffu : 0u) | (tk + 1 < vleft ? 0xffff0000u : 0u);
                    const uint32_t k1 = (tk + 8 < vleft ? 0xffffu : 0u) | (tk + 9 < vleft ? 0xffff0000u : 0u);
                    if (!F::kFp8) {
#pragma unroll
                        for (int d = 0; d < 16; d += 2) {
                            const int chunk = (d & 7) + (lane >> 4);
                            uint32_t r[4];
                            ldsm_x4_t(r, vt + (d >> 3) * kHalfPageBytes + row * 128 + ((chunk ^ (row & 7)) << 4));
                            if (cut) {
                                r[0] &= k0;
                                r[1] &= k1;
                                r[2] &= k0;
                                r[3] &= k1;
                            }
                            mma_bf16_16816(o[d], pa[j], r[0], r[1]);
                            mma_bf16_16816(o[d + 1], pa[j], r[2], r[3]);
                        }
                    } else {
                        // a 16-bit element holds dims 2g, 2g + 1 of one token: the halves of the converted pair go
                        // to two output tiles, of the even and of the odd dims of the 16-dim chunk
#pragma unroll
                        for (int c = 0; c < 8; c += 2) {
                            const int chunk = c + (lane >> 4);
                            uint32_t r[4];
                            ldsm_x4_t(r, vt + row * 128 + ((chunk ^ (row & 7)) << 4));
                            if (cut) {
                                r[0] &= k0;
                                r[1] &= k1;
                                r[2] &= k0;
                                r[3] &= k1;
                            }
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const uint32_t x0 = e4m3x2_to_f16x2(static_cast<uint16_t>(r[2 * u] & 0xffffu));
                                const uint32_t x1 = e4m3x2_to_f16x2(static_cast<uint16_t>(r[2 * u] >> 16));
                                const uint32_t y0 = e4m3x2_to_f16x2(static_cast<uint16_t>(r[2 * u + 1] & 0xffffu));
                                const uint32_t y1 = e4m3x2_to_f16x2(static_cast<uint16_t>(r[2 * u + 1] >> 16));
                                mma_f16_16816(o[2 * (c + u)], pa[j], __byte_perm(x0, x1, 0x5410),
                                              __byte_perm(y0, y1, 0x5410));
                                mma_f16_16816(o[2 * (c + u) + 1], pa[j], __byte_perm(x0, x1, 0x7632),
                                              __byte_perm(y0, y1, 0x7632));
                            }
                        }
                    }
                }
            }
            if (alive && !v_waited)
                alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->full[s_v]), ((it + 1) / F::kStages) & 1, p.withhold);
            __syncwarp();
            if (lane == 0) {
                if (k_held)
                    mbar_arrive(smem_addr(&ctl->empty[s_k]));
                mbar_arrive(smem_addr(&ctl->empty[s_v]));
            }
            if (!OWN && p.mass) {
#pragma unroll
                for (int q = 1; q < 4; q <<= 1) {
                    ps0 += __shfl_xor_sync(0xffffffffu, ps0, q);
                    ps1 += __shfl_xor_sync(0xffffffffu, ps1, q);
                }
                if (t == 0) {
                    mass_part[i * 64 + warp * 16 + g] = make_float2(ps0, m0);
                    mass_part[i * 64 + warp * 16 + g + 8] = make_float2(ps1, m1);
                }
            }
        }
        // ---- the warps' parts join in shared memory (the ring is done with) ----
#pragma unroll
        for (int q = 1; q < 4; q <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, q);
            l1 += __shfl_xor_sync(0xffffffffu, l1, q);
        }
        if (t == 0) {
            ctl->wm[warp][g] = m0;
            ctl->wm[warp][g + 8] = m1;
            ctl->wl[warp][g] = l0;
            ctl->wl[warp][g + 8] = l1;
        }
        consumer_barrier();  // every warp has read its last tile
        float *wo = reinterpret_cast<float *>(smem);  // [warp][16][kAttnOStride]
        if (!ctl->abort_flag) {
            const float u0 = v_unit(v0) * (1.0f / kVTop), u1 = v_unit(v1) * (1.0f / kVTop);  // E4M3
            if (F::kFp8) {
                const float i0 = l0 == 0.0f ? 0.0f : 1.0f / l0, i1 = l1 == 0.0f ? 0.0f : 1.0f / l1;
#pragma unroll
                for (int d = 0; d < 16; ++d) {
                    o[d][0] *= i0;
                    o[d][1] *= i0;
                    o[d][2] *= i1;
                    o[d][3] *= i1;
                }
            }
            float *at = wo + warp * 16 * kAttnOStride;
#pragma unroll
            for (int d = 0; d < 16; d += 2) {
                // bf16: tile d holds dims 8d + 2t, +1; E4M3: tiles d, d + 1 hold dims 8d + 4t (+2) and (+1, +3)
                if (!F::kFp8) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int col = (d + u) * 8 + 2 * t;
                        *reinterpret_cast<float2 *>(at + g * kAttnOStride + col) = make_float2(o[d + u][0], o[d + u][1]);
                        *reinterpret_cast<float2 *>(at + (g + 8) * kAttnOStride + col) =
                            make_float2(o[d + u][2], o[d + u][3]);
                    }
                } else {
                    const int col = d * 8 + 4 * t;
                    *reinterpret_cast<float4 *>(at + g * kAttnOStride + col) =
                        make_float4(o[d][0] * u0, o[d + 1][0] * u0, o[d][1] * u0, o[d + 1][1] * u0);
                    *reinterpret_cast<float4 *>(at + (g + 8) * kAttnOStride + col) =
                        make_float4(o[d][2] * u1, o[d + 1][2] * u1, o[d][3] * u1, o[d + 1][3] * u1);
                }
            }
        }
        consumer_barrier();
        float *co = wo + kAttnWarps * 16 * kAttnOStride;  // [rows][kAttnOStride]: the CTA's part
        for (int n = warp; n < rows; n += kAttnWarps) {
            const int col = lane * 4, w0 = n / 16, r = n % 16;
            float M = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
                M = fmaxf(M, ctl->wm[w0 + k * MT][r]);
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float share[KS];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const float f = rescale(ctl->wm[w0 + k * MT][r], M), fl = f * ctl->wl[w0 + k * MT][r];
                sum += fl;
                share[k] = F::kFp8 ? fl : f;
            }
            const float inv = !F::kFp8 ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int w = w0 + k * MT;
                const float f = share[k] * inv;
                const float4 v = *reinterpret_cast<const float4 *>(wo + (w * 16 + r) * kAttnOStride + col);
                acc.x += f * v.x;
                acc.y += f * v.y;
                acc.z += f * v.z;
                acc.w += f * v.w;
            }
            if (ctl->abort_flag) {  // a part that is not whole
                acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                M = -INFINITY;
                sum = 0.0f;
            }
            *reinterpret_cast<float4 *>(co + n * kAttnOStride + col) = acc;
            if (lane == 0) {
                ctl->cm[n] = M;
                ctl->cl[n] = sum;
            }
        }
    }
    // ---- the cluster's parts join in rank order ----
    __syncwarp();
    if (S > 1)
        cluster_sync_all();
    else
        __syncthreads();
    if (warp < kAttnWarps) {
        const float *co = reinterpret_cast<const float *>(smem) + kAttnWarps * 16 * kAttnOStride;
        const uint32_t a_co = smem_addr(co), a_cm = smem_addr(ctl->cm), a_cl = smem_addr(ctl->cl);
        // a thread a row: maximum, sum and factors, every rank's numbers under way at once
        if (tid < rows) {
            float m[8], l[8];
            int gave_up = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                m[c] = -INFINITY;
                l[c] = 0.0f;
                if (c < S) {
                    m[c] = dsmem_ld_f32(mapa_shared(a_cm + tid * 4, c));
                    l[c] = dsmem_ld_f32(mapa_shared(a_cl + tid * 4, c));
                    gave_up |= dsmem_ld_s32(mapa_shared(smem_addr(&ctl->abort_flag), c));
                }
            }
            float M = m[0], sum = 0.0f;
#pragma unroll
            for (int c = 1; c < 8; ++c)
                M = fmaxf(M, m[c]);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float f = rescale(m[c], M);
                l[c] *= f;
                sum += l[c];
                if (!F::kFp8)
                    ctl->fac[c][tid] = f;
            }
            if (gave_up)
                sum = 0.0f;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            if (F::kFp8) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    ctl->fac[c][tid] = l[c] * inv;
            }
            ctl->rm[tid] = M;
            ctl->rinv[tid] = inv;
            if ((OWN || p.lse) && crank == 0) {
                // OWN: +inf marks a part that is not whole
                const float e = sum == 0.0f ? -INFINITY : M + log2f(sum);
                p.lse[place(tid)] = OWN ? (gave_up ? INFINITY : e) : e * kLn2;
            }
        }
        consumer_barrier();
#pragma unroll 2
        for (int n = warp + kAttnWarps * crank; n < rows; n += kAttnWarps * S) {
            float4 v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < S)
                    v[c] = dsmem_ld_f32x4(mapa_shared(a_co + (n * kAttnOStride + lane * 4) * 4, c));
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < S) {
                    const float f = ctl->fac[c][n];
                    acc.x += f * v[c].x;
                    acc.y += f * v[c].y;
                    acc.z += f * v[c].z;
                    acc.w += f * v[c].w;
                }
            const bool none = ctl->rinv[n] == 0.0f;  // nothing visible: zeros
            const float inv = F::kFp8 ? 1.0f : ctl->rinv[n];
            if (OWN) {
                *reinterpret_cast<float4 *>(p.part + place(n) * kDim + lane * 4) =
                    make_float4(none ? 0.0f : acc.x * inv, none ? 0.0f : acc.y * inv, none ? 0.0f : acc.z * inv,
                                none ? 0.0f : acc.w * inv);
                continue;
            }
            uint2 w;
            w.x = none ? 0u : f32x2_to_bf16x2(acc.x * inv, acc.y * inv);
            w.y = none ? 0u : f32x2_to_bf16x2(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2 *>(p.out + place(n) * kDim + lane * 4) = w;
        }
        if (!OWN && p.mass) {
            // a block's mass: its 64 (slice, row) sums, moved to their rows' final maximum and sum
            for (int i = warp; i < count; i += kAttnWarps) {
                float v = 0.0f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int e = lane + 32 * u, n = (e / 16) % MT * 16 + e % 16;
                    const float2 x = mass_part[i * 64 + e];
                    if (n < rows && ctl->rinv[n] != 0.0f)
                        v += x.x * rescale(x.y, ctl->rm[n]) * ctl->rinv[n];
                }
#pragma unroll
                for (int q = 16; q >= 1; q >>= 1)
                    v += __shfl_xor_sync(0xffffffffu, v, q);
                if (lane == 0)
                    p.mass[(static_cast<int64_t>(owner) * p.kv_heads + h) * p.k + ctl->list_slot[i]] = v;
            }
        }
    }
    // This grid runs beside prefix_attn_kernel and needs nothing of it, but must not complete before it: who waits for
    // this grid reads the parts of both.
    if (OWN && blockIdx.x == 0)
        griddep_wait();
    __syncwarp();
    if (S > 1)
        cluster_sync_all();  // no CTA ends while another reads its shared memory
}

}  // namespace msa

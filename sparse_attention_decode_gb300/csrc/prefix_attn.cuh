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
//
// The time of a tile's page is its chain, scores (512 cycles) -> softmax (1360) ->
// product (512), with a barrier between each; two chains run side by side, each
// with an MMA thread of its own, so that one thread's waits pass while the other's
// MMAs run (one thread for both tiles: 5000 cycles a page, the tensor pipe a third
// busy).  Where a KV head has at most 128 rows, the two chains are the even and the
// odd pages of one tile, and a range leaves two parts.
#pragma once

#include "block_attn.cuh"

namespace msa {

constexpr int kPrefixStages = 4;  // K and V tiles of two pages
constexpr int kPrefixThreads = 352;  // two softmax warpgroups, a TMA warp, two MMA warps
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
    uint64_t q_full[2], s_full[2];
    uint64_t p_half[2], p_full[2];  // the first 64 weights of each row and the turn to issue; all weights
    uint64_t o_done[2];
    uint64_t drained[2];
    uint32_t tmem;
    int abort_flag;
};

constexpr size_t kPrefixSmemBytes = 1024 + 2 * kPageBytes + kPrefixStages * kPageBytes + sizeof(PrefixSmem);

// The MMA warps run their whole loop converged, with one elected lane behind a
// predicate: descriptors and addresses are then the warp's, not a thread's, and an
// instruction needs no moves from thread to uniform registers.  (Issued from inside
// `if (lane == 0)`, an instruction of 64 cycles took about 110.)
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  elect.sync _|p, 0xffffffff;\n"
        "  selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(one));
    return one;
}

// D[tmem] (+)= A[smem] * B[smem]^T, by the elected lane.
template <bool ACC>
__device__ __forceinline__ void umma_ss_one(uint32_t one, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc)
{
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  .reg .b64 ad, bd;\n"
        "  setp.ne.u32 p, %6, 0;\n"
        "  mov.b64 ad, {%1, %5};\n"
        "  mov.b64 bd, {%2, %5};\n"
        "  @p tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %3, %4;\n"
        "}\n" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(ACC ? 1 : 0), "r"(kUmmaDescHi), "r"(one)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], by the elected lane: A's 128 rows lie in the lanes, two bf16 of K a column.
template <bool ACC>
__device__ __forceinline__ void umma_ts_one(uint32_t one, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc)
{
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  .reg .b64 bd;\n"
        "  setp.ne.u32 p, %6, 0;\n"
        "  mov.b64 bd, {%2, %5};\n"
        "  @p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %3, %4;\n"
        "}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "n"(ACC ? 1 : 0), "r"(kUmmaDescHi), "r"(one)
        : "memory");
}

__device__ __forceinline__ void umma_commit_one(uint32_t one, uint32_t bar)
{
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  setp.ne.u32 p, %1, 0;\n"
        "  @p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
        "}\n" ::"r"(bar),
        "r"(one)
        : "memory");
}

// Two fp32 operations an instruction, and the maximum of three.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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

// Chain t's MMAs, by one warp: for each of its pages the product of the weights
// with V and the next page's scores.
template <int t>
__device__ __forceinline__ void issue_chain(const PrefixAttnParams &p, PrefixSmem *ctl, uint8_t *smem, uint8_t *kv,
                                            uint32_t tmem, int64_t lo, int64_t hi, int P)
{
    constexpr uint32_t idesc_s = umma_idesc_bf16_f32(128, 128);
    constexpr uint32_t idesc_o = umma_idesc_bf16_f32(128, 128) | (1u << 16);  // B with N contiguous
    const uint32_t one = elect_one();
    const int ways = p.parts.ways;
    const uint32_t d_s = tmem + t * 128, d_o = tmem + 256 + t * 128;
    const uint32_t q_desc = umma_desc_lo(smem_addr(smem) + t * kPageBytes), kv_addr = smem_addr(kv);
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(smem_addr(bar), parity)))
            return true;
        return attn_wait(&ctl->abort_flag, p.fault, smem_addr(bar), parity);
    };
    auto pass = [&](int chain) {
        if (one)
            mbar_arrive(smem_addr(&ctl->p_half[chain]));
    };
    // the scores of page number kp of the CTA, whose tile has landed; the turn goes to chain `next` (-1: it does not
    // pass) while the last ones are still to be issued, so that its product reaches the pipe before it runs dry
    auto scores = [&](uint32_t kp, int next) {
        const uint32_t s = (2 * kp) % kPrefixStages;
        const uint32_t b = umma_desc_lo(kv_addr + s * kPageBytes);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            const uint32_t off = ((ks >> 2) * kHalfPageBytes + (ks & 3) * 32) >> 4;
            if (ks == 0)
                umma_ss_one<false>(one, d_s, q_desc + off, b + off, idesc_s);
            else
                umma_ss_one<true>(one, d_s, q_desc + off, b + off, idesc_s);
            if (ks == 5 && next >= 0)
                pass(next);
        }
        umma_commit_one(one, smem_addr(&ctl->s_full[t]));
        umma_commit_one(one, smem_addr(&ctl->kv_empty[s]));
    };
    auto landed = [&](uint32_t tile) { return wait(&ctl->kv_full[tile % kPrefixStages], (tile / kPrefixStages) & 1); };
    // The chains take turns, product and next scores together: chain 0's softmax then runs beside chain 1's MMAs and
    // the other way round (left alone they fall into step and share the pipe).  The turn is one of p_half's arrivals,
    // so that one wait covers both; chain 0 begins.
    if (t == 0)
        pass(0);
    bool alive = true;
    uint32_t it = 0, kp0 = 0, seg = 0;
    int left = static_cast<int>(hi - lo), in_unit = P - static_cast<int>(lo % P);
    for (; left > 0 && alive; ++seg) {
        const int n = min(left, in_unit);
        left -= n;
        in_unit = P;
        alive = wait(&ctl->q_full[t], seg & 1);
        const int j0 = ways == 2 ? t : 0;
        if (alive && j0 < n) {
            alive = landed(2 * (kp0 + j0));
            if (!alive)
                break;
            tc_fence_after_sync();
            scores(kp0 + j0, -1);
        }
        for (int j = j0; j < n; j += ways, ++it) {
            const uint32_t kp = kp0 + j;
            const bool more = j + ways < n;
            // with one tile's pages in turn, the last page has no successor in the other chain: the turn stays
            const int next = t == 0 && ways == 2 && j + 1 >= n ? 0 : 1 - t;
            alive = landed(2 * kp + 1) && (!more || landed(2 * (kp + ways))) && wait(&ctl->p_half[t], it & 1);
            if (!alive)
                break;
            tc_fence_after_sync();
            // 16 tokens an instruction: 8 columns of weights, two atoms of V; the first half while the second half's
            // weights are on their way
            const uint32_t sv = (2 * kp + 1) % kPrefixStages;
            const uint32_t b = umma_desc_v_lo(kv_addr + sv * kPageBytes);
            if (j == j0)
                umma_ts_one<false>(one, d_o, d_s, b, idesc_o);
            else
                umma_ts_one<true>(one, d_o, d_s, b, idesc_o);
#pragma unroll
            for (int ks = 1; ks < 4; ++ks)
                umma_ts_one<true>(one, d_o, d_s + ks * 8, b + ((ks * 2048) >> 4), idesc_o);
            alive = wait(&ctl->p_full[t], it & 1);
            if (!alive)
                break;
            tc_fence_after_sync();
#pragma unroll
            for (int ks = 4; ks < 8; ++ks)
                umma_ts_one<true>(one, d_o, d_s + ks * 8, b + ((ks * 2048) >> 4), idesc_o);
            umma_commit_one(one, smem_addr(&ctl->o_done[t]));
            umma_commit_one(one, smem_addr(&ctl->kv_empty[sv]));
            // the next page's scores overwrite the weights that this product reads: MMAs of one thread run in the
            // order of their issue
            if (more)
                scores(kp + ways, next);
            else
                pass(next);
        }
        kp0 += n;
    }
    umma_commit_one(one, smem_addr(&ctl->drained[t]));  // nothing in flight when the tensor memory is freed
    mbar_wait(smem_addr(&ctl->drained[t]), 0);
    __syncwarp();
}

__global__ void __launch_bounds__(kPrefixThreads, 1) prefix_attn_kernel(const __grid_constant__ PrefixAttnParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *kv = smem + 2 * kPageBytes;  // after the two Q tiles
    auto *ctl = reinterpret_cast<PrefixSmem *>(kv + kPrefixStages * kPageBytes);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in all lanes, and known to be

    griddep_launch_dependents();
    const int prefix = __shfl_sync(0xffffffffu, prefix_tokens(p.parts, p.prefix_len), 0);
    const PrefixSplit split(p.parts, prefix, static_cast<int>(gridDim.x));
    if (prefix == 0 && *p.prefix_len != 0 && blockIdx.x == 0 && tid == 0)
        atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
    const int cta = blockIdx.x;
    if (cta >= split.ctas)
        return;
    const int P = split.pages;
    const int64_t lo = split.start(cta), hi = split.start(cta + 1);
    const int ways = p.parts.ways;  // 1: two tiles, every page in both; 2: one tile, its pages in turn

    if (tid == 0) {
        for (int s = 0; s < kPrefixStages; ++s) {
            mbar_init(smem_addr(&ctl->kv_full[s]), 1);
            mbar_init(smem_addr(&ctl->kv_empty[s]), 2 / ways);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_addr(&ctl->q_full[t]), 128);
            mbar_init(smem_addr(&ctl->s_full[t]), 1);
            mbar_init(smem_addr(&ctl->p_half[t]), 129);  // the rows, and the other chain's passing of the turn
            mbar_init(smem_addr(&ctl->p_full[t]), 128);
            mbar_init(smem_addr(&ctl->o_done[t]), 1);
            mbar_init(smem_addr(&ctl->drained[t]), 1);
        }
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
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);  // columns 0, 128: S (and the weights); 256, 384: O

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
        issue_chain<0>(p, ctl, smem, kv, tmem, lo, hi, P);
    } else if (warp == 10) {
        issue_chain<1>(p, ctl, smem, kv, tmem, lo, hi, P);
    } else {
        // ---- softmax: one thread a row ----
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // (32 * (warp % 4)) << 16
        const uint32_t ts = tmem + t * 128 + lanes, to = tmem + 256 + t * 128 + lanes;
        const float c = p.scale_log2;
        bool alive = true;
        uint32_t it = 0, kp0 = 0;  // pages of this chain, pages of the CTA before the unit's
        for (int64_t x = lo; x < hi; ) {
            const int u = static_cast<int>(x / P), j0 = static_cast<int>(x % P);
            const int n = static_cast<int>(min(hi - x, static_cast<int64_t>(P - j0)));
            x += n;
            const int h = u / p.parts.head_tiles;
            const int nrow = (u % p.parts.head_tiles) * p.parts.tile_rows + (ways == 1 ? t * 128 : 0) + row;
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
            const int first = ways == 2 ? t : 0;
            int page = first < n ? p.prefix_table[j0 + first] : 0;
            for (int j = first; j < n && alive; j += ways, ++it) {
                // tokens of the page that count
                const int valid = page < 0 || page >= p.num_pages ? 0 : min(kPage, prefix - (j0 + j) * kPage);
                if (j + ways < n)
                    page = p.prefix_table[j0 + j + ways];
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
                    // what lies in V past the tokens is no data: zero it (0 x NaN is NaN); both chains do, since
                    // neither product waits for the other's softmax
                    const uint32_t vt = 2 * (kp0 + j) + 1;
                    alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->kv_full[vt % kPrefixStages]),
                                      (vt / kPrefixStages) & 1);
                    if (!alive)
                        break;
                    if (row >= valid) {
                        uint8_t *at = kv + (vt % kPrefixStages) * kPageBytes + row * 128;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            *reinterpret_cast<uint4 *>(at + (i >> 3) * kHalfPageBytes + (i & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                float mx[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mx[q] = fmaxf(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]));
#pragma unroll
                    for (int i = 2; i < 32; i += 2)
                        mx[q] = max3(mx[q], __uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                if (j == first) {
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
                uint64_t sum[4] = {0, 0, 0, 0};  // two fp32 sums each
                const uint64_t c2 = pack2(c, c), r2 = pack2(-ref, -ref);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t w[32];
#pragma unroll
                    for (int q = 2 * half; q < 2 * half + 2; ++q)
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float a, b;
                            unpack2(fma2(pack2(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])), c2, r2), a, b);
                            a = exp2_approx(a);
                            b = exp2_approx(b);
                            sum[q] = add2(sum[q], pack2(a, b));
                            w[(q & 1) * 16 + i / 2] = f32x2_to_bf16x2(a, b);
                        }
                    tmem_st32(ts + half * 32, w);
                    tmem_wait_st();
                    tc_fence_before_sync();
                    mbar_arrive(smem_addr(half ? &ctl->p_full[t] : &ctl->p_half[t]));
                }
                float a, b;
                unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
                l += a + b;
            }
            // ---- the range's part of the unit ----
            const bool some = first < n;
            if (alive && some)
                alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->o_done[t]), (it - 1) & 1);
            tc_fence_after_sync();
            kp0 += n;
            // 128 rows in a row of slots: chain t of a unit with two tiles holds its rows t * 128 .., of one with one tile its part t
            const int64_t block = (static_cast<int64_t>(cta) + u) * 2 + t;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            if (alive && some) {
                // through the tile's Q (every product with it is done), 64 dims at a time, each warp its 32 rows:
                // a thread holds a row, a store of a warp should cover whole lines
                float *part = p.parts.o + (block * 128 + (row & ~31)) * kDim;
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
            p.parts.lse[block * 128 + row] =
                !alive ? INFINITY : l == 0.0f ? -INFINITY : m + log2f(l);
        }
        tc_fence_before_sync();
    }
    __syncthreads();
    if (warp == 9)
        tmem_dealloc(tmem, 512);
}

}  // namespace msa

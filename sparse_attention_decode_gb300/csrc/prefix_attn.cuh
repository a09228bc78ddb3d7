// Attention of all requests' query rows over the prefix they share: a dense
// product on the 5th-generation tensor cores.
//
// The rows of one KV head (batch * q_len * group of them) read the same keys, so
// they stand side by side as the M rows of S = Q K^T and O = P V.  A unit is
// (KV head, tile of 256 rows), or of 128 where there are not more; the prefix's
// pages of all units, one after the other, are cut into one equal range a CTA, and
// a range's part of a unit goes to the workspace as (O / L, M + log2 L) in fp32.
// block_attn_kernel makes one more part of each request's own pages, and
// join_kernel adds a row's parts up, always in page order.
//
// The prefix is bound by the tensor cores and the softmax, own pages by the cache
// stream.  So the two run side by side: this kernel takes as many SMs as its share
// of the work by the live lengths (its other CTAs end at once), and the own pages'
// CTAs, launched as its dependents, start on the rest and follow as its CTAs end.
// (Few own CTAs are launched first instead, and this kernel as their dependent.)
// (64 requests over 32768 + 147000 tokens: 88 us; one after the other 125; own pages
// as further units of this kernel 193, a few microseconds of latency for each of
// their short runs.)
//
// Per page and 128-row tile: S (128 x 128, fp32) in tensor memory; a warpgroup
// with one thread a row takes the row's maximum, 2^(c s - m) and the sum, and
// writes the weights as bf16 over S; the second product reads them from there
// (A in tensor memory, V's page from shared memory with the dims contiguous:
// the B operand's transposed form).  The reference m of a row is only moved (and
// O, L rescaled) when the maximum outgrows it by more than 2^8: weights then stay
// at most 2^8, which costs no precision in fp32 sums and bf16 operands, and the
// rescaling of O in tensor memory becomes rare.
//
// The time of a tile's page is its chain, scores (512 cycles) -> softmax (1000 to
// 1400) -> product (512), with a barrier between each.  Two chains run side by
// side, each with an MMA warp of its own, and take turns at the tensor cores: the
// two tiles of 256 rows, or the even and the odd pages of one tile, whose range
// then leaves two parts.  2700 to 3000 cycles a page of 256 rows (1.45-1.6 us), 0.7 to
// 3/4 of the MMA rate; one issuing thread for both took 5000, two without turns 5000
// as well.  What is left is the MMAs' own: a turn's 16 take 1350 cycles where the pipe
// alone would take 1024 (the scores read 8 KiB of shared memory each in 64 cycles, all
// there is).  Without any loads of tiles a page takes 2850, with two threads a row in
// the softmax, with three tiles of K and two of V, or with the turn passed earlier the
// same as now.  Around the pages: 1.5 us until the split is known, 3 to 3.5 until the
// first scores, 3 for the parts, 1.5 to 2 until the join knows that both kernels have
// ended, 2 to 4 for the join.
#pragma once

#include "block_attn.cuh"

namespace msa {

constexpr int kPrefixStages = 4;  // K and V tiles of two pages
constexpr int kPrefixThreads = 352;  // two softmax warpgroups, a TMA warp, two MMA warps
constexpr int kPrefixMaxGrid = 256;
constexpr float kPrefixLag = 8.0f;

// Where the parts lie.  Unit u = head * head_tiles + tile; the units' pages stand
// one after the other, u * pages + j, and CTA g of the `ctas` that take part covers
// [start(g), start(g + 1)); what it has of unit u is in slot g + u (unique: both
// grow along the sequence).  A slot holds two blocks of 128 rows: the halves of a
// tile of 256 rows (ways = 1), or two parts of a tile of 128 (ways = 2).
struct PrefixParts {
    float *o, *lse;          // [slot][2][128] rows, lse in log2 units; -inf: nothing (o is not written), +inf: not whole
    float *own_o, *own_lse;  // [query rows, heads]: the part of a row's own pages
    int batch, q_len, group, kv_heads;
    int rows;  // rows of a KV head: batch * q_len * group
    int tile_rows, ways, head_tiles, units;
    int own_cost;          // of an own page and KV head, in eighths of a 128-row tile's page of the prefix
    int own_most;          // pages of one request that count in that comparison: their sum stays below 2^31
    int limit, seq_limit;  // bounds on the prefix's and a request's tokens
    int grid;              // CTAs prefix_attn_kernel is launched with
    int spare;             // of them, so many take no part: their SMs are the own pages'
};

__device__ __forceinline__ int tokens_in(int n, int limit) { return n < 0 || n > limit ? 0 : n; }

// Pages a CTA's range should have at least: one for each chain of a small tile.  Fewer pages are more parts to join,
// more of them a longer range: 2 requests over 4133 tokens take 13.3 us (15.8 with 1, 14.6 with 3, 14.5 with 4), over
// 8192 15.9 (16.5, 15.0, 15.6: 64 parts a row cost more there than a third page), over 16384 18.3 with any, and larger
// batches have more pages a CTA anyway.
constexpr int kPrefixMinPages = 2;

// 32-bit numbers (the host refuses more): quotients of 64 bits would be half the start of every kernel.
struct PrefixSplit {
    int pages, ctas;
    int span, per;    // `per` CTAs share `span` pages: those of one unit, or of all
    int range, more;  // pages of a CTA's range; the first `more` of the `per` have one more
    // own: the batch's own pages, which run beside the prefix on the SMs that are left
    __device__ PrefixSplit(const PrefixParts &p, int prefix, int own)
    {
        pages = pages_of(prefix);
        const int total = pages * p.units;
        // shares of the GPU: an estimate, in the same steps wherever it is made
        const float mine = static_cast<float>(total) * (p.ways == 1 ? 2.0f : 1.0f);
        const float all = __fadd_rn(mine, __fmul_rn(static_cast<float>(own), static_cast<float>(p.own_cost * p.kv_heads) * 0.125f));
        const int most =
            min(p.grid - p.spare, max(1, __float2int_rn(__fmul_rn(static_cast<float>(p.grid), __fdividef(mine, all)))));
        const int per_unit = (pages + kPrefixMinPages - 1) / kPrefixMinPages;
        ctas = min(most, (total + kPrefixMinPages - 1) / kPrefixMinPages);
        // The same number of CTAs for every unit where that leaves few out: no range then ends in a second unit, and
        // the tiles of a head walk the same pages at the same time, from L2 but for the first.
        const int each = min(most / p.units, per_unit);
        if (each > 0 && each * p.units * 8 >= ctas * 7) {
            span = pages;
            per = each;
            ctas = per * p.units;
        } else {
            span = total;
            per = ctas;
        }
        range = per > 0 ? span / per : 0;
        more = span - range * per;
    }
    __device__ int start(int g) const
    {
        const int k = g / per, i = g - k * per;
        return k * span + i * range + min(i, more);
    }
    // the CTA whose range holds page x of the sequence
    __device__ int owner(int x) const
    {
        const int k = x / span, y = x - k * span, longer = more * (range + 1);
        return k * per + (y < longer ? y / (range + 1) : more + (y - longer) / range);
    }
};

struct PrefixAttnParams {
    CUtensorMap kmap, vmap;
    const uint16_t *q;
    const int32_t *prefix_table;
    const int32_t *prefix_len;
    const int32_t *seq_lens;
    PrefixParts parts;
    uint32_t *fault;
    int64_t q_stride, num_pages;
    float scale_log2;
    int withhold;  // test of the bounded waits: the producer loads and signals no page
};

// The batch's own pages, added up by a whole block (every thread gets the sum).
// `sums`: shared, one entry a warp.
template <int THREADS>
__device__ __forceinline__ int own_pages(const int32_t *seq_lens, const PrefixParts &p, int *sums)
{
    const int tid = threadIdx.x;
    int n = 0;
    for (int b = tid; b < p.batch; b += THREADS)
        n += min(pages_of(tokens_in(seq_lens[b], p.seq_limit)), p.own_most);
    n = __reduce_add_sync(0xffffffffu, n);
    if ((tid & 31) == 0)
        sums[tid >> 5] = n;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < THREADS / 32; ++w)
        all += sums[w];
    return all;
}

struct PrefixSmem {
    uint64_t kv_full[kPrefixStages], kv_empty[kPrefixStages];
    uint64_t q_full[2], s_full[2];
    uint64_t p_half[2], p_full[2];  // the first 64 weights of each row and the turn to issue; all weights
    uint64_t o_done[2];
    uint64_t drained[2];
    int warp_sums[12];
    uint32_t tmem;
    int abort_flag;
};

constexpr size_t kPrefixSmemBytes = 1024 + (2 + kPrefixStages) * kPageBytes + sizeof(PrefixSmem);

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

// The maximum of three.
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
                                            uint32_t tmem, int lo, int hi, int P)
{
    constexpr uint32_t idesc_s = umma_idesc_bf16_f32(128, 128);
    constexpr uint32_t idesc_o = umma_idesc_bf16_f32(128, 128) | (1u << 16);  // B with N contiguous
    const uint32_t one = elect_one();
    const int ways = p.parts.ways;
    const uint32_t d_s = tmem + t * 128, d_o = tmem + 256 + t * 128;
    const uint32_t q_desc = umma_desc_lo(smem_addr(smem) + t * kPageBytes), kv_addr = smem_addr(kv);
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return attn_wait(&ctl->abort_flag, p.fault, smem_addr(bar), parity, p.withhold);
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
    int left = hi - lo, in_unit = P - lo % P;
    while (left > 0 && alive) {
        const int n = min(left, in_unit);
        left -= n;
        in_unit = P;
        const int j0 = ways == 2 ? t : 0;
        if (j0 < n) {  // a chain without a page of the unit takes no part: its query tile is not loaded either
            alive = wait(&ctl->q_full[t], seg++ & 1) && landed(2 * (kp0 + j0));
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
    const int cta = blockIdx.x;
    // set up while the lengths are on their way; tensor memory too, by CTAs that may turn out to have no part in it
    // (an SM has no room for a second CTA that wants it)
    const int given = *p.prefix_len;  // under way together with the lengths
    if (tid == 8 * 32) {
        prefetch_tensormap(&p.kmap);
        prefetch_tensormap(&p.vmap);
        for (int s = 0; s < kPrefixStages; ++s) {
            mbar_init(smem_addr(&ctl->kv_full[s]), 1);
            mbar_init(smem_addr(&ctl->kv_empty[s]), 2 / p.parts.ways);
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
    const int own = own_pages<kPrefixThreads>(p.seq_lens, p.parts, ctl->warp_sums);
    const int prefix = __shfl_sync(0xffffffffu, tokens_in(given, p.parts.limit), 0);
    if (cta == 0 && tid == 0 && prefix != given)
        atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
    const PrefixSplit split(p.parts, prefix, own);
    tc_fence_after_sync();
    if (cta >= split.ctas) {
        if (warp == 9)
            tmem_dealloc(ctl->tmem, 512);
        if (cta == 0)
            griddep_wait();
        return;
    }
    const int P = split.pages, ways = p.parts.ways;
    const int lo = split.start(cta), hi = split.start(cta + 1);
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);  // columns 0, 128: S (and the weights); 256, 384: O

    if (warp == 8) {
        // ---- K and V tiles, page after page ----
        bool alive = true;
        uint32_t it = 0;
        int pages = -1;  // a lane's share of 32 entries of the table
        int u = lo / P, at = lo - u * P;
        const int n = hi - lo;
        for (int i = 0; i < n && alive; ++i) {
            if ((i & 31) == 0) {
                pages = -1;
                if (i + lane < n) {
                    pages = p.prefix_table[(at + lane) % P];
                    if (pages < 0 || pages >= p.num_pages) {
                        pages = -1;
                        atomicOr(p.fault, MSA_FAULT_PAGE_ID);
                    }
                }
            }
            const int page = __shfl_sync(0xffffffffu, pages, i & 31);
            const int h = u / p.parts.head_tiles;
            for (int kvi = 0; kvi < 2; ++kvi, ++it) {
                const int s = static_cast<int>(it % kPrefixStages);
                if (it >= kPrefixStages)
                    alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->kv_empty[s]),
                                      (it / kPrefixStages + 1) & 1, p.withhold);
                if (!alive)
                    break;
                if (lane == 0 && !p.withhold) {
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
            if (++at == P) {
                at = 0;
                ++u;
            }
        }
        // the copies in flight land before the CTA may end, also where another role gave up
        for (uint32_t j = it >= kPrefixStages ? it - kPrefixStages : 0; j < it && !p.withhold; ++j)
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
        for (int x = lo; x < hi; ) {
            const int u = x / P, page0 = x - u * P;
            const int n = min(hi - x, P - page0);
            x += n;
            const int h = u / p.parts.head_tiles;
            const int nrow = (u % p.parts.head_tiles) * p.parts.tile_rows + (ways == 1 ? t * 128 : 0) + row;
            const bool have = nrow < p.parts.rows;
            const bool some_row = __any_sync(0xffffffffu, have);  // a warp without rows only keeps the barriers going
            const int first = ways == 2 ? t : 0;
            const bool some = first < n;  // pages of the unit for this chain
            // Both chains are through with the units before (named barrier 2, the two softmax warpgroups): a wait tells a
            // phase by its parity, so a chain that begins with a stage must know that the stage's phase before, which may
            // have been the other chain's, is over, and a chain without a page of a unit must not run ahead.
            asm volatile("bar.sync 2, 256;" ::: "memory");
            if (some) {
                // the warp's 32 rows, two at a time: 16 lanes a row of 256 bytes
                const int64_t src = have ? static_cast<int64_t>(nrow / p.parts.group) * p.q_stride +
                                               (h * p.parts.group + nrow % p.parts.group) * kDim
                                         : -1;
                uint8_t *dst = smem + t * kPageBytes + ((lane >> 3) & 1) * kHalfPageBytes + (row & ~31) * 128;
#pragma unroll 1
                for (int r0 = lane >> 4; r0 < 32; r0 += 16) {
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t from = __shfl_sync(0xffffffffu, src, r0 + 2 * i);
                        v[i] = from >= 0 ? reinterpret_cast<const uint4 *>(p.q + from)[lane & 15] : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = r0 + 2 * i;
                        *reinterpret_cast<uint4 *>(dst + r * 128 + (((lane ^ r) & 7) << 4)) = v[i];
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                mbar_arrive(smem_addr(&ctl->q_full[t]));
            }
            float m = -INFINITY, l = 0.0f;
            int page = some ? p.prefix_table[page0 + first] : 0;
            for (int j = first; j < n && alive; j += ways, ++it) {
                // tokens of the page that count
                const int valid = page < 0 || page >= p.num_pages ? 0 : min(kPage, prefix - (page0 + j) * kPage);
                if (j + ways < n)
                    page = p.prefix_table[page0 + j + ways];
                alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->s_full[t]), it & 1, p.withhold);
                if (!alive)
                    break;
                tc_fence_after_sync();
                if (!some_row && valid == kPage) {
                    tc_fence_before_sync();
                    mbar_arrive(smem_addr(&ctl->p_half[t]));
                    mbar_arrive(smem_addr(&ctl->p_full[t]));
                    continue;
                }
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
                                      (vt / kPrefixStages) & 1, p.withhold);
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
                if (j == first)
                    m = top;
                // two quarters of the scores to weights (bf16 pairs) and their sums, at the reference m
                const uint64_t c2 = pack2(c, c);
                auto weigh = [&](const uint32_t (&x)[32], const uint32_t (&y)[32], uint32_t (&w)[32]) {
                    const float ref = m == -INFINITY ? 0.0f : m;
                    const uint64_t r2 = pack2(-ref, -ref);
                    uint64_t sx = 0, sy = 0;  // two fp32 sums each
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float a, b, d, e;
                        unpack2(fma2(pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c2, r2), a, b);
                        unpack2(fma2(pack2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), c2, r2), d, e);
                        a = exp2_approx(a);
                        b = exp2_approx(b);
                        d = exp2_approx(d);
                        e = exp2_approx(e);
                        sx = add2(sx, pack2(a, b));
                        sy = add2(sy, pack2(d, e));
                        w[i / 2] = f32x2_to_bf16x2(a, b);
                        w[16 + i / 2] = f32x2_to_bf16x2(d, e);
                    }
                    float a, b;
                    unpack2(add2(sx, sy), a, b);
                    return a + b;
                };
                uint32_t w[32];
                // The first half is weighed beside the search for the maximum, at the reference so far; where a row of
                // the warp has outgrown it, the reference moves and the half, still in tensor memory, is weighed again.
                float sum = weigh(s[0], s[1], w);
                if (j != first && __any_sync(0xffffffffu, top > m + kPrefixLag)) {
                    const float to_m = fmaxf(m, top), f = rescale(m, to_m);
                    m = to_m;
                    l *= f;
                    alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->o_done[t]), (it - 1) & 1, p.withhold);
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
                    tmem_ld32(ts, s[0]);
                    tmem_ld32(ts + 32, s[1]);
                    tmem_wait_ld(s[0]);
                    tmem_regs_ready(s[1]);
                    if (valid < kPage) {
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (q * 32 + i >= valid)
                                    s[q][i] = 0xff800000u;
                    }
                    sum = weigh(s[0], s[1], w);
                }
                tmem_st32(ts, w);
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive(smem_addr(&ctl->p_half[t]));
                l += sum;
                l += weigh(s[2], s[3], w);
                tmem_st32(ts + 32, w);
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive(smem_addr(&ctl->p_full[t]));
            }
            // ---- the range's part of the unit ----
            if (alive && some)
                alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->o_done[t]), (it - 1) & 1, p.withhold);
            tc_fence_after_sync();
            kp0 += n;
            // chain t's block of the slot: its rows of a tile of 256, or its part of the one tile
            const int64_t block = ((static_cast<int64_t>(cta) + u) * 2 + t) * 128;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            if (alive && some && some_row) {
                // through the warp's own rows of the tile's Q (every product with it is done; the other warps may be
                // loading theirs for the next run), 64 dims at a time: a thread holds a row, a store of a warp should
                // cover whole lines
                float *part = p.parts.o + (block + (row & ~31)) * kDim;
                uint8_t *turn = smem + t * kPageBytes + (row & ~31) * 128;
                auto chunk = [&](int r, int c) {  // 16 bytes c of 16 of row r of the warp
                    return reinterpret_cast<float4 *>(turn + (c >> 3) * kHalfPageBytes + r * 128 + (((c ^ r) & 7) << 4));
                };
                const int left = p.parts.rows - (nrow - lane);  // rows of the warp that exist
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
                            *chunk(lane, q * 8 + i / 4) =
                                make_float4(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv,
                                            __uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int r = lane >> 4; r < 32; r += 2)
                        if (r < left)
                            *reinterpret_cast<float4 *>(part + r * kDim + half * 64 + (lane & 15) * 4) =
                                *chunk(r, lane & 15);
                }
                __syncwarp();
            }
            // +inf marks a part that is not whole
            if (have)
                p.parts.lse[block + row] =
                    !alive ? INFINITY : l == 0.0f ? -INFINITY : m + log2f(l);
        }
        tc_fence_before_sync();
    }
    __syncthreads();
    if (warp == 9)
        tmem_dealloc(tmem, 512);
    if (cta == 0)
        griddep_wait();  // where the own pages' kernel was launched first: the join waits for this grid only
}

// ---------------------------------------------------------------------------
// out = sum 2^(e - M) o / sum 2^(e - M) over a row's parts (o, e), prefix first,
// then own.  WPR warps a row take the parts in turn; each has the numbers of 32
// parts in its lanes and asks for several vectors at once.  Bound by those reads
// (L2): 4096 rows with 7 parts, 15 MB, take 4 us, 1024 rows with 26 parts 3.
struct JoinParams {
    PrefixParts parts;
    const int32_t *prefix_len;
    const int32_t *seq_lens;
    uint16_t *out;
    float *lse;
};

template <int WPR, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WPR == 1 ? 2 : WPR == 2 ? 3 : 5) join_kernel(const __grid_constant__ JoinParams p)
{
    constexpr int kRows = WARPS / WPR;  // rows of a block
    __shared__ float4 s_acc[WARPS][32];
    __shared__ float s_m[WARPS], s_sum[WARPS];
    __shared__ int s_bad[WARPS];
    const PrefixParts &a = p.parts;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = warp % WPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + warp / WPR;  // (query row, KV head, head of the group)
    const bool exists = row < static_cast<int64_t>(a.rows) * a.kv_heads;
    const int g = static_cast<int>(row % a.group), h = static_cast<int>(row / a.group % a.kv_heads);
    const int query = static_cast<int>(row / a.group / a.kv_heads);
    const int n = query * a.group + g;
    const PrefixSplit split(a, tokens_in(*p.prefix_len, a.limit),
                            own_pages<32 * WARPS>(p.seq_lens, a, s_bad));
    __syncthreads();
    int64_t first = 0;  // row of the prefix's first part; its next one is `step` on
    const int step = 256 / a.ways;
    int count = 0;  // parts of the prefix; the request's own comes after them
    if (exists && split.pages > 0) {
        const int u = h * a.head_tiles + n / a.tile_rows;
        const int g0 = split.owner(u * split.pages), g1 = split.owner((u + 1) * split.pages - 1) + 1;
        count = (g1 - g0) * a.ways;
        first = static_cast<int64_t>(g0 + u) * 256 + n % a.tile_rows;
    }
    const int64_t own_row = exists ? (static_cast<int64_t>(query) * a.kv_heads + h) * a.group + g : 0;
    griddep_wait();  // both kernels have ended
    float M = -INFINITY, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    bool bad = false;
    const int all = exists ? count + 1 : 0, mine = all > sub ? (all - sub + WPR - 1) / WPR : 0;
    for (int i0 = 0; i0 < mine; i0 += 32) {
        const int end = min(32, mine - i0);
        const int at = sub + i0 * WPR;  // the part of lane 0
        const int l_at = at + lane * WPR;
        const float x = lane >= end     ? -INFINITY
                        : l_at == count ? __ldcg(a.own_lse + own_row)
                                        : __ldcg(a.lse + first + static_cast<int64_t>(l_at) * step);
        bad |= __any_sync(0xffffffffu, x == INFINITY);
        float to = fmaxf(M, x);
#pragma unroll
        for (int q = 16; q >= 1; q >>= 1)
            to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, q));
        const float old = rescale(M, to), f = x == -INFINITY ? 0.0f : rescale(x, to);
        M = to;
        sum *= old;
        acc.x *= old;
        acc.y *= old;
        acc.z *= old;
        acc.w *= old;
        constexpr int kBatch = WPR == 2 ? 8 : 4;
        for (int i = 0; i < end; i += kBatch) {
            float4 v[kBatch];  // under way together, also where fewer are left
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int part = at + (i + k) * WPR;
                const float *o = part == count ? a.own_o + own_row * kDim : a.o + (first + static_cast<int64_t>(part) * step) * kDim;
                v[k] = i + k < end ? __ldcg(reinterpret_cast<const float4 *>(o) + lane) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float fi = __shfl_sync(0xffffffffu, f, i + k);  // 0 past the end
                const bool some = fi != 0.0f;  // what a part that holds nothing has there may be anything
                sum += fi;
                acc.x += some ? fi * v[k].x : 0.0f;
                acc.y += some ? fi * v[k].y : 0.0f;
                acc.z += some ? fi * v[k].z : 0.0f;
                acc.w += some ? fi * v[k].w : 0.0f;
            }
        }
    }
    if (WPR > 1) {
        s_acc[warp][lane] = acc;
        if (lane == 0) {
            s_m[warp] = M;
            s_sum[warp] = sum;
            s_bad[warp] = bad;
        }
        __syncthreads();
        if (sub != 0)
            return;
#pragma unroll
        for (int w = 1; w < WPR; ++w) {
            const float m = s_m[warp + w], to = fmaxf(M, m), fa = rescale(M, to), fb = rescale(m, to);
            const float4 v = s_acc[warp + w][lane];
            sum = sum * fa + s_sum[warp + w] * fb;
            acc.x = acc.x * fa + v.x * fb;
            acc.y = acc.y * fa + v.y * fb;
            acc.z = acc.z * fa + v.z * fb;
            acc.w = acc.w * fa + v.w * fb;
            M = to;
            bad |= s_bad[warp + w] != 0;
        }
    }
    if (!exists)
        return;
    const bool none = bad || sum == 0.0f;  // nothing visible, or a part that is not whole
    const float inv = none ? 0.0f : 1.0f / sum;
    const int64_t to = (static_cast<int64_t>(query) * a.kv_heads + h) * a.group + g;
    uint2 w;
    w.x = none ? 0u : f32x2_to_bf16x2(acc.x * inv, acc.y * inv);
    w.y = none ? 0u : f32x2_to_bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2 *>(p.out + to * kDim + lane * 4) = w;
    if (p.lse && lane == 0)
        p.lse[to] = none ? -INFINITY : (M + log2f(sum)) * kLn2;
}

}  // namespace msa

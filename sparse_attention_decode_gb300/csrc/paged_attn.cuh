// Attention of a few query rows over all pages of their request, on the
// 5th-generation tensor cores with the tokens as the rows of both products.
//
// Mathematics: the softmax over a row's tokens and the join of its parts as in
// block_attn.cuh.  A unit is (request, tile of up to 64 of its query rows, KV head);
// the pages of all units, one after the other, are cut into one equal range a CTA,
// so a context of any length keeps every SM busy to the end.  A unit inside one range
// goes straight to the output; the parts of one that a range's end cuts go to the
// workspace in fp32 and are joined, always in page order, by paged_join_kernel.
//
// Why tokens as rows: a tcgen05 product has 128 rows, a request's query rows are 1 to
// 64, a page is 128 tokens.  S^T = K Q^T (128 tokens x rows) and O^T = V^T P^T
// (128 dims x rows) fill the 128 rows with what there is, read K and V where TMA put
// them, and cost one pass of the operand through shared memory each, however many query
// rows there are: one product for all of them.  A thread has one token: the scale of an
// E4M3 token is one number for all its weights.
//
// What bounds it: the stream of pages, where a unit has many and its rows are 16 to 32
// (256 requests of 8000 to 8704 tokens, 4.4 GB: 625 us, 7.0 TB/s; E4M3, 32 of 30000 to
// 32768: 162 us, 6.5 TB/s; 64 bf16 rows, 8 of 32768: 89.6 us, 6.0 TB/s).  On one E4M3
// request of 131072 (30.0 us for a floor of 20.5) and below, what a unit costs once: its
// rows, the first page's references, the epilogue, the join, one after the other.  With
// 64 E4M3 rows the weights' arithmetic: 1.5 us a page for 0.8 of the stream.
//
// A row's maximum would be a reduction over the lanes for every page.  The reference m
// of a row need not be the maximum: it is kept until a score passes it by more than
// 2^8 (weights then stay below 2^8, which costs fp32 sums and bf16 operands nothing), so
// that a page asks one vote of its 128 threads, and the reductions, and the rescaling of
// O in tensor memory, follow only where somebody has passed it: once a unit as a rule.
//
// E4M3: the codes go into the products as they are (kind::f8f6f4), so the other operand
// has to be E4M3 as well.  A query row, its largest brought to [2^7, 2^8) by a power of two, is
// the sum of two E4M3 numbers, the second 2^-5 on: exactly where it is within 2^-14 of the
// row's largest (4 bits each), and to 2^-22 of that largest below.  A weight times its
// token's V scale is the sum of three, after one rounding to f16 (11 bits), and held
// relative to the row's largest such product so far: down to 2^-26 of it.  (Two terms would
// hold a weight near the largest to bf16's 2^-8, but one 2^-10 of it to 2^-4, and a long
// request can consist of such.)  The terms stand side by side as further rows of the
// product, so K and V still pass once.
#pragma once

#include <type_traits>

#include "attn_common.cuh"
#include "host_util.cuh"
#include "paged_split.cuh"
#include "tcgen05.cuh"

#include "msa_serving.h"

namespace msa {

struct PagedBf16 {
    static constexpr bool kFp8 = false;
    static constexpr int kTileBytes = kPageBytes;
    static constexpr int kScaleBytes = 0;
    static constexpr int kQTerms = 1, kPTerms = 1;
};
struct PagedFp8 {
    static constexpr bool kFp8 = true;
    static constexpr int kTileBytes = kPage * kDim;
    static constexpr int kScaleBytes = kPage * 4;
    static constexpr int kQTerms = 2, kPTerms = 3;
};

constexpr int kPagedMaxGrid = 256;
constexpr int kPagedMaxRows = 64;   // of a unit
constexpr float kPagedLag = 8.0f;
constexpr float kPagedMost = 32768.0f;  // of an E4M3 weight, in units of 2^-11 (what its terms are taken from)
constexpr float kPagedWideScale = 1024.0f;  // of V: times a unit, 2^117 at most, one above this may pass fp32

struct PagedParams {
    CUtensorMap kmap, vmap;
    const uint16_t *q;
    const float *kscale, *vscale;
    const int32_t *block_table, *seq_lens;
    uint16_t *out;
    float *lse;
    float *part_o, *part_lse;  // [2 a CTA][tile_rows] rows, lse in log2 units; -inf: nothing, +inf: not whole
    uint32_t *fault;
    int64_t q_stride, bt_stride, num_pages;
    int batch, q_len, kv_heads, group, seq_limit;
    int tile_rows, row_tiles;  // rows of a unit at most; units of a request and KV head
    int grid;                  // CTAs of paged_attn_kernel
    int lead;                  // what a unit costs beside its pages, in pages
    float scale_log2;
    int withhold;  // test of the bounded waits: the producer loads and signals no page
};

struct PagedScan {
    int slots[32], requests[32], early[32];  // the warps' sums
    PagedAt at;
};

// The batch's work, the slots of requests before `request` (in `before`) and the place of slot `want(work)` of the sequence
// (request `batch`: there is none), by a whole block.
template <int THREADS, class Want>
__device__ __forceinline__ PagedWork paged_find(const PagedParams &p, PagedScan *sc, int request, int &before, Want want)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int units = p.row_tiles * p.kv_heads;
    const int each = (p.batch + THREADS - 1) / THREADS;
    const int b0 = min(p.batch, tid * each), b1 = min(p.batch, b0 + each);
    int mine = 0, some = 0, early = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = paged_slots(p, b, units);
        mine += n;
        some += n > 0;
        early += b < request ? n : 0;
    }
    int upto = mine;  // inclusive over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        upto += lane >= o ? x : 0;
    }
    some = __reduce_add_sync(0xffffffffu, some);
    early = __reduce_add_sync(0xffffffffu, early);
    if (lane == 31) {
        sc->slots[warp] = upto;
        sc->requests[warp] = some;
        sc->early[warp] = early;
    }
    if (tid == 0)
        sc->at = PagedAt{p.batch, 0, 0};
    __syncthreads();
    int prior = 0;
    PagedWork work{0, 0};
    before = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        prior += w < warp ? sc->slots[w] : 0;
        work.slots += sc->slots[w];
        work.units += sc->requests[w] * units;
        before += sc->early[w];
    }
    const int x = want(work);
    const int from = prior + upto - mine;
    if (x >= from && x < from + mine)
        sc->at = paged_at(p, b0, b1, from, x);
    __syncthreads();
    return work;
}

template <int N, int WAYS, int GROUPS, int STAGES>
struct PagedSmem {
    static constexpr int kChains = WAYS * GROUPS, kRows = N * GROUPS;
    uint64_t kv_full[STAGES], kv_empty[STAGES];
    uint64_t q_full, q_taken, s_full[WAYS], s_free[WAYS], p_full[WAYS], o_done[WAYS], drained[WAYS];
    int page_ok[STAGES];
    PagedScan scan;
    uint32_t tmem;
    int abort_flag;
    int64_t q_at[kRows];             // the unit's rows: where their queries lie, from the request's and head's on,
    int at[kRows], hidden[kRows];    // their places among [query rows, query heads], the last tokens they do not see
    int sees[kRows];                 // and those they do, of the request at hand
    alignas(16) float coef[kRows];   // E4M3: the score scale and the query row's power of two, undone
    alignas(16) float nref[kChains][N];    // a chain's rows: the reference (log2 units), negative
    alignas(16) float unit[kChains][N];    // E4M3: what weights x V scale are multiplied by
    alignas(16) float fac[kChains][N];     // what a moved reference multiplies a row's O by,
    alignas(16) float lfac[kChains][N];    // and its sum
    float vtop[kChains][N];                // E4M3: the row's largest weight x V scale at its reference
    int wmax[kChains][4][N], omax[kChains][4][N];  // the warps' largest scores and products, in an order of integers
    float wsum[kChains][4][N];
    float share[WAYS][kRows];        // what a way's part of a row is multiplied by at the end
};

// Shared memory: query rows, the chains' weights, as many tiles of K and V as there is room for, their scales.
template <class F, int N, int WAYS, int GROUPS>
struct PagedLayout {
    static constexpr int kChains = WAYS * GROUPS;
    static constexpr int kThreads = kChains * 128 + 32 + WAYS * 32;      // softmax warpgroups, a TMA warp, MMA warps
    static constexpr int kRows = N * GROUPS;                             // of a unit
    static constexpr int kQBytes = kRows * kDim * 2;                     // (E4M3: two terms of a byte)
    static constexpr int kPBytes = F::kPTerms * N * kPage * (F::kFp8 ? 1 : 2);  // of a chain
    static constexpr int kKv = kQBytes + kChains * kPBytes;                    // 1024-byte aligned
    static constexpr int kRoom = 232448 - 1024 - kKv - static_cast<int>(sizeof(PagedSmem<N, WAYS, GROUPS, 12>));
    static constexpr int kStages = kRoom / (F::kTileBytes + F::kScaleBytes);
    using Smem = PagedSmem<N, WAYS, GROUPS, kStages>;
    static constexpr int kScales = kKv + kStages * F::kTileBytes;
    static constexpr int kCtl = kScales + kStages * F::kScaleBytes;
    static constexpr size_t kBytes = 1024 + kCtl + sizeof(Smem);
    static constexpr int kSCols = F::kQTerms * N, kOCols = F::kPTerms * N;  // of a chain
    static constexpr int kWayCols = GROUPS * (kSCols + kOCols);
    static constexpr int kCols = WAYS * kWayCols;
    static constexpr uint32_t kTmem = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    // a ring for each way, so that a stage's phases, which a wait tells by their parity, are all one way's
    static constexpr int kDepth = kStages / WAYS;
    static __device__ __forceinline__ int stage(int way, uint32_t tile)
    {
        return static_cast<int>(tile % kDepth) + way * kDepth;
    }
    static __device__ __forceinline__ uint32_t phase(uint32_t tile) { return (tile / kDepth) & 1; }
    static_assert(kKv % 1024 == 0 && kDepth >= 3 && kStages <= 12 && kBytes <= 232448 && kCols <= 512,
                  "shared and tensor memory");
};

// D[tmem] (+)= A B, by the elected lane; both operands in shared memory, the high words of their descriptors given.
template <bool FP8>
__device__ __forceinline__ void umma_small(uint32_t one, uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                           uint32_t b_hi, uint32_t idesc, uint32_t acc)
{
    if (FP8)
        asm volatile(
            "{\n"
            "  .reg .pred p, q;\n"
            "  .reg .b64 ad, bd;\n"
            "  setp.ne.u32 p, %6, 0;\n"
            "  setp.ne.u32 q, %7, 0;\n"
            "  mov.b64 ad, {%1, %4};\n"
            "  mov.b64 bd, {%2, %5};\n"
            "  @p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %3, q;\n"
            "}\n" ::"r"(d_tmem),
            "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(a_hi), "r"(b_hi), "r"(one), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n"
            "  .reg .pred p, q;\n"
            "  .reg .b64 ad, bd;\n"
            "  setp.ne.u32 p, %6, 0;\n"
            "  setp.ne.u32 q, %7, 0;\n"
            "  mov.b64 ad, {%1, %4};\n"
            "  mov.b64 bd, {%2, %5};\n"
            "  @p tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %3, q;\n"
            "}\n" ::"r"(d_tmem),
            "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(a_hi), "r"(b_hi), "r"(one), "r"(acc)
            : "memory");
}

// 16 (or 8) consecutive 32-bit columns of one TMEM lane per thread; valid after a wait (tmem_wait_all).
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}

// A barrier of `threads` threads that tells all of them whether one of them says so.
__device__ __forceinline__ bool barrier_any(int id, int threads, bool say)
{
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n"
        "  .reg .pred p, q;\n"
        "  setp.ne.u32 p, %3, 0;\n"
        "  barrier.cta.red.or.pred.aligned q, %1, %2, p;\n"
        "  selp.u32 %0, 1, 0, q;\n"
        "}\n"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(say))
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void barrier_sync(int id, int threads)
{
    __syncwarp();
    asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// fp32 in an order of signed integers, and back.
__device__ __forceinline__ int float_int(float x)
{
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float int_float(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// E4M3 terms: an f16 value times down(0) is the first; what that leaves, exact in f16, times down(1) the second, and so on.
// back(i) takes term i out.
// A query row, its largest in [2^14, 2^15): t[0] 2^7 + t[1] 2^2.  The first term's last bit of 4 leaves half of it, which is
// 2^8 at most in the second.  Exact from 1 on, where the first term is normal; 2^-8 off below.
struct QueryTerms {
    static __device__ constexpr uint32_t down(int i)
    {
        constexpr uint32_t kDown[2] = {0x20002000u, 0x34003400u};  // 2^-7, 2^-2, two each
        return kDown[i];
    }
    static __device__ constexpr uint32_t back(int i)
    {
        constexpr uint32_t kBack[2] = {0xd800d800u, 0xc400c400u};  // -2^7, -2^2
        return kBack[i];
    }
    static constexpr float kStep = 1.0f / 32.0f;  // a term's unit over the one before
};
// A weight x V scale, its row's largest 2^9 to 2^10 when its unit was chosen: t[0] 2^11 + t[1] 2^2 + t[2] 2^-7.  The second is
// 256 at most; the third can be asked for up to 2^12 where the value passes 2^11, and ends at 448: 8 bits are left then, 11 below.
struct WeightTerms {
    static __device__ constexpr uint32_t down(int i)
    {
        constexpr uint32_t kDown[3] = {0x10001000u, 0x34003400u, 0x58005800u};  // 2^-11, 2^-2, 2^7
        return kDown[i];
    }
    static __device__ constexpr uint32_t back(int i)
    {
        constexpr uint32_t kBack[3] = {0xe800e800u, 0xc400c400u, 0xa000a000u};  // -2^11, -2^2, -2^-7
        return kBack[i];
    }
    static constexpr float kStep = 1.0f / 512.0f;
};

// x, y as sums of E4M3 terms, two codes each, after one rounding to f16.
template <class V, int TERMS>
__device__ __forceinline__ void e4m3_terms(float x, float y, uint32_t (&t)[TERMS])
{
    uint32_t left = f32x2_to_f16x2(x, y);
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        uint16_t code;
        asm("{\n  .reg .b32 a;\n  mul.f16x2 a, %1, %2;\n  cvt.rn.satfinite.e4m3x2.f16x2 %0, a;\n}\n" : "=h"(code) : "r"(left), "r"(V::down(i)));
        t[i] = code;
        if (i + 1 < TERMS)
            asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(left) : "r"(e4m3x2_to_f16x2(code)), "r"(V::back(i)));
    }
}

// The sums over a warp's lanes of N values a thread: lane r (modulo N) gets value r's.
template <int N>
__device__ __forceinline__ float lanes_sum(const float (&l)[N], int lane)
{
    float v[16];
    if (N == 32) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float keep = lane & 16 ? l[(i + 16) % N] : l[i], give = lane & 16 ? l[i] : l[(i + 16) % N];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = l[i] + __shfl_xor_sync(0xffffffffu, l[i], 16);
    }
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < o) {
                const float keep = lane & o ? v[i + o] : v[i], give = lane & o ? v[i] : v[i + o];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
    return v[0];
}

// A way is a line of pages: all of the unit's (WAYS 1), or every second (2).  One warp issues its products, for all rows of
// the unit at once; GROUPS chains, a warpgroup each, take N of the rows (16 or 32) through the softmax.
template <class F, int N, int WAYS, int GROUPS>
__global__ void __launch_bounds__(PagedLayout<F, N, WAYS, GROUPS>::kThreads, 1) paged_attn_kernel(const __grid_constant__ PagedParams p)
{
    using L = PagedLayout<F, N, WAYS, GROUPS>;
    constexpr int R = L::kRows, C = L::kChains, kSoft = C * 128;  // threads of the softmax
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *kv = smem + L::kKv;
    float *scales = reinterpret_cast<float *>(smem + L::kScales);
    auto *ctl = reinterpret_cast<typename L::Smem *>(smem + L::kCtl);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in all lanes, and known to be
    const int cta = blockIdx.x;

    griddep_launch_dependents();
    if (tid == kSoft) {
        prefetch_tensormap(&p.kmap);
        prefetch_tensormap(&p.vmap);
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(smem_addr(&ctl->kv_full[s]), 1);
            mbar_init(smem_addr(&ctl->kv_empty[s]), 1 + 4 * GROUPS);  // a product and the chains' warps
        }
        mbar_init(smem_addr(&ctl->q_full), 4 * C);
        mbar_init(smem_addr(&ctl->q_taken), WAYS);
        for (int t = 0; t < WAYS; ++t) {
            mbar_init(smem_addr(&ctl->s_full[t]), 1);
            mbar_init(smem_addr(&ctl->s_free[t]), 4 * GROUPS);
            mbar_init(smem_addr(&ctl->p_full[t]), 4 * GROUPS);
            mbar_init(smem_addr(&ctl->o_done[t]), 1);
            mbar_init(smem_addr(&ctl->drained[t]), 1);
        }
        ctl->abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 4 * C + 1) {
        tmem_alloc(smem_addr(&ctl->tmem), L::kTmem);
        tmem_relinquish_alloc_permit();
    }
    tc_fence_before_sync();
    if (cta == 0)
        for (int b = tid; b < p.batch; b += L::kThreads)
            if (p.seq_lens[b] != paged_len(p, b))
                atomicOr(p.fault, MSA_FAULT_SEQ_LEN);
    int unused;
    const PagedWork total = paged_find<L::kThreads>(p, &ctl->scan, 0, unused, [&](const PagedWork &work) {
        const PagedSplit s(work, p);
        return cta < s.ctas ? s.start(cta) : -1;
    });
    const PagedSplit split(total, p);
    const int count = cta < split.ctas ? split.start(cta + 1) - split.start(cta) : 0;
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
    const int heads = p.kv_heads * p.group, unit_rows = p.q_len * p.group;
    PagedWalk walk(p, ctl->scan.at, count);

    if (warp == 4 * C) {
        // ---- K and V tiles, page after page ----
        bool alive = true;
        uint32_t tiles[2] = {0, 0};  // of the ways' rings
        uint32_t done = 0;
        for (; walk.left > 0 && alive; walk.next(p)) {
            const int n = walk.run(), h = walk.u % p.kv_heads;
            const int32_t *table = p.block_table + walk.b * p.bt_stride + walk.j;
            int pages = -1;  // a lane's share of 32 entries of the table
            for (int i = 0; i < n && alive; ++i, ++done) {
                if ((i & 31) == 0) {
                    pages = -1;
                    if (i + lane < n) {
                        pages = table[i + lane];
                        if (pages < 0 || pages >= p.num_pages) {
                            pages = -1;
                            atomicOr(p.fault, MSA_FAULT_PAGE_ID);
                        }
                    }
                }
                const int page = __shfl_sync(0xffffffffu, pages, i & 31);
                const int way = WAYS == 2 ? done & 1 : 0;
                for (int kvi = 0; kvi < 2; ++kvi) {
                    const uint32_t tile = way ? tiles[1]++ : tiles[0]++;
                    const int s = L::stage(way, tile);
                    if (tile >= L::kDepth)
                        alive = attn_wait(&ctl->abort_flag, p.fault, smem_addr(&ctl->kv_empty[s]), L::phase(tile) ^ 1, p.withhold);
                    if (!alive) {
                        way ? --tiles[1] : --tiles[0];
                        break;
                    }
                    if (lane == 0 && !p.withhold) {
                        const uint32_t bar = smem_addr(&ctl->kv_full[s]), dst = smem_addr(kv) + s * F::kTileBytes;
                        ctl->page_ok[s] = page >= 0;
                        if (page < 0) {
                            mbar_arrive(bar);
                        } else {
                            const CUtensorMap *map = kvi ? &p.vmap : &p.kmap;
                            mbar_arrive_expect_tx(bar, F::kTileBytes + F::kScaleBytes);
                            tma_load_4d(dst, map, 0, 0, h, page, bar);
                            if (F::kFp8)
                                bulk_load(smem_addr(scales + s * kPage),
                                          (kvi ? p.vscale : p.kscale) + (static_cast<int64_t>(page) * p.kv_heads + h) * kPage,
                                          F::kScaleBytes, bar);
                            else
                                tma_load_4d(dst + kHalfPageBytes, map, 64, 0, h, page, bar);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        // the copies in flight land before the CTA may end, also where another role gave up
        for (int way = 0; way < WAYS && !p.withhold; ++way)
            for (uint32_t j = tiles[way] >= L::kDepth ? tiles[way] - L::kDepth : 0; j < tiles[way]; ++j)
                mbar_wait(smem_addr(&ctl->kv_full[L::stage(way, j)]), L::phase(j));
    } else if (warp > 4 * C) {
        // ---- a way's products ----
        const int way = warp - 4 * C - 1;
        const uint32_t one = elect_one();
        constexpr uint32_t kTypes = (1u << 4) | (F::kFp8 ? 0u : (1u << 7) | (1u << 10)) | ((128u >> 4) << 24);
        constexpr uint32_t idesc_s = kTypes | (static_cast<uint32_t>(GROUPS * L::kSCols >> 3) << 17);
        constexpr uint32_t idesc_o = kTypes | (static_cast<uint32_t>(GROUPS * L::kOCols >> 3) << 17) | (1u << 15) | (1u << 16);  // both with their rows contiguous
        constexpr int kSteps = F::kFp8 ? 4 : 8;
        constexpr uint32_t kPlainHi = (2048u >> 4) | (1u << 14);  // no swizzle: 16 bytes of rows x 128 tokens, 2 KiB to the next rows
        const uint32_t d_s = tmem + way * L::kWayCols, d_o = d_s + GROUPS * L::kSCols;
        // query rows: bf16 in two halves of 64 dims, E4M3 in one, a chain's terms one after the other
        const uint32_t q_desc = umma_desc_lo(smem_addr(smem));
        const uint32_t p_desc = ((smem_addr(smem + L::kQBytes + way * GROUPS * L::kPBytes) >> 4) & 0x3FFFu) | ((128u >> 4) << 16);
        const uint32_t kv_addr = smem_addr(kv);
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return attn_wait(&ctl->abort_flag, p.fault, smem_addr(bar), parity, p.withhold);
        };
        auto landed = [&](uint32_t tile) { return wait(&ctl->kv_full[L::stage(way, tile)], L::phase(tile)); };
        auto test = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test_wait(smem_addr(bar), parity)); };
        auto scores = [&](uint32_t tile) {
            const int sk = L::stage(way, tile);
            const uint32_t a = umma_desc_lo(kv_addr + sk * F::kTileBytes);
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                const uint32_t off = F::kFp8 ? ks * 32 : (ks >> 2) * kHalfPageBytes + (ks & 3) * 32;
                const uint32_t boff = F::kFp8 ? ks * 32 : (ks >> 2) * (R * 128) + (ks & 3) * 32;
                umma_small<F::kFp8>(one, d_s, a + (off >> 4), kUmmaDescHi, q_desc + (boff >> 4), kUmmaDescHi, idesc_s, ks > 0);
            }
            umma_commit_one(one, smem_addr(&ctl->s_full[way]));
            umma_commit_one(one, smem_addr(&ctl->kv_empty[sk]));
        };
        bool alive = true;
        uint32_t it = 0, done = 0, seg = 0;
        for (; walk.left > 0 && alive; walk.next(p)) {
            const int n = walk.run();
            alive = wait(&ctl->q_full, seg++ & 1);
            if (one)
                mbar_arrive(smem_addr(&ctl->q_taken));
            bool ahead = false;  // the page's scores have been asked for
            for (int j = WAYS == 2 ? (way ^ done) & 1 : 0; j < n && alive; j += WAYS, ++it) {
                if (!ahead) {
                    alive = landed(2 * it);
                    if (!alive)
                        break;
                    tc_fence_after_sync();
                    scores(2 * it);
                }
                ahead = false;
                // the next page's scores as soon as its keys are there and this page's have been read, so that they run
                // beside the softmax; its weights otherwise
                for (uint32_t i = 0; j + WAYS < n && !ahead && i < kSpinLimit && !test(&ctl->p_full[way], it & 1) &&
                                     !*reinterpret_cast<volatile int *>(&ctl->abort_flag);
                     ++i)
                    if (test(&ctl->s_free[way], it & 1) && test(&ctl->kv_full[L::stage(way, 2 * it + 2)], L::phase(2 * it + 2))) {
                        tc_fence_after_sync();
                        scores(2 * it + 2);
                        ahead = true;
                    }
                alive = landed(2 * it + 1) && wait(&ctl->p_full[way], it & 1);
                if (!alive)
                    break;
                tc_fence_after_sync();
                const int sv = L::stage(way, 2 * it + 1);
                const uint32_t v = umma_desc_v_lo(kv_addr + sv * F::kTileBytes);
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks)
                    umma_small<F::kFp8>(one, d_o, v + ((ks * 1024 * (F::kFp8 ? 4 : 2)) >> 4), kUmmaDescHi,
                                        p_desc + ((ks * (F::kFp8 ? 512 : 256)) >> 4), kPlainHi, idesc_o, ks > 0 || j >= WAYS);
                umma_commit_one(one, smem_addr(&ctl->o_done[way]));
                umma_commit_one(one, smem_addr(&ctl->kv_empty[sv]));
            }
            done += n;
        }
        umma_commit_one(one, smem_addr(&ctl->drained[way]));  // nothing in flight when the tensor memory is freed
        mbar_wait(smem_addr(&ctl->drained[way]), 0);
        __syncwarp();
    } else {
        // ---- softmax: a thread a token ----
        const int t = warp >> 2, tau = tid & 127, way = t / GROUPS, rows0 = t % GROUPS * N;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // (32 * (warp % 4)) << 16
        const uint32_t ts = tmem + way * L::kWayCols + t % GROUPS * L::kSCols + lanes;
        const uint32_t to = tmem + way * L::kWayCols + GROUPS * L::kSCols + t % GROUPS * L::kOCols + lanes;
        uint8_t *pbuf = smem + L::kQBytes + t * L::kPBytes + tau * 16;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return attn_wait(&ctl->abort_flag, p.fault, smem_addr(bar), parity, p.withhold);
        };
        // requests without tokens: their rows are empty
        for (int b = cta; b < p.batch; b += gridDim.x) {
            if (paged_len(p, b) > 0)
                continue;
            const int64_t row0 = static_cast<int64_t>(b) * p.q_len * heads;
            for (int i = tid; i < p.q_len * heads * (kDim / 8); i += kSoft)
                reinterpret_cast<uint4 *>(p.out + row0 * kDim)[i] = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse)
                for (int i = tid; i < p.q_len * heads; i += kSoft)
                    p.lse[row0 + i] = -INFINITY;
        }
        // the rows of tile `row0` on: the same for every request and head
        auto lay_rows = [&](int row0) {
            if (tid < R) {
                const int i = (row0 + tid) / p.group, g = row0 + tid - i * p.group;
                ctl->q_at[tid] = i * p.q_stride + g * kDim;
                ctl->at[tid] = i * heads + g;
                ctl->hidden[tid] = row0 + tid < unit_rows ? p.q_len - 1 - i : 0x3fffffff;
            }
            barrier_sync(2, kSoft);
        };
        if (p.row_tiles == 1)
            lay_rows(0);
        // The query rows of the unit at `w` on their way to registers, 16 lanes a row, and from there to shared memory; then the
        // chains' products may begin, beside what is left to do for the unit before.
        auto load_rows = [&](const PagedWalk &w, uint4 (&v)[R / (8 * C)]) {
            const int tile_at = w.u / p.kv_heads, h = w.u - tile_at * p.kv_heads;
            const int rows = min(p.tile_rows, unit_rows - tile_at * p.tile_rows);
            const uint16_t *q = p.q + static_cast<int64_t>(w.b) * p.q_len * p.q_stride + h * p.group * kDim;
#pragma unroll
            for (int i = 0; i < R / (8 * C); ++i) {
                const int r = (tid >> 4) + 8 * C * i;
                v[i] = w.left > 0 && r < rows ? reinterpret_cast<const uint4 *>(q + ctl->q_at[r])[tid & 15] : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        auto put_rows = [&](const PagedWalk &w, const uint4 (&v)[R / (8 * C)]) {
            const int c = tid & 15;
#pragma unroll
            for (int i = 0; i < R / (8 * C); ++i) {
                const int r = (tid >> 4) + 8 * C * i;
                if (!F::kFp8) {
                    *reinterpret_cast<uint4 *>(smem + (c >> 3) * (R * 128) + r * 128 + (((c ^ r) & 7) << 4)) = v[i];
                    continue;
                }
                const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    top = max3(top, fabsf(bf16_lo(x[k])), fabsf(bf16_hi(x[k])));
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                // the power of two that brings it to [2^14, 2^15)
                const int e = max(14, min(254, static_cast<int>(__float_as_uint(top) >> 23)));
                const float f = __int_as_float((268 - e) << 23);
                uint32_t term[4][F::kQTerms];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    e4m3_terms<QueryTerms>(bf16_lo(x[k]) * f, bf16_hi(x[k]) * f, term[k]);
#pragma unroll
                for (int k = 0; k < F::kQTerms; ++k) {
                    const int at = (r / N) * L::kSCols + k * N + r % N;
                    *reinterpret_cast<uint2 *>(smem + at * 128 + ((((c >> 1) ^ at) & 7) << 4) + (c & 1) * 8) =
                        make_uint2(term[0][k] | term[1][k] << 16, term[2][k] | term[3][k] << 16);
                }
                if (c == 0)
                    ctl->coef[r] = __int_as_float((e - 7) << 23) * p.scale_log2;  // (2^-7 is in the terms)
            }
            if (tid < R)
                ctl->sees[tid] = max(0, w.len - ctl->hidden[tid]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&ctl->q_full));
        };
        auto start_rows = [&] {
            if (tau < N) {
                ctl->nref[t][tau] = INFINITY;
                ctl->unit[t][tau] = 1.0f;
                ctl->vtop[t][tau] = 0.0f;
            }
        };
        bool dead = false;
        uint32_t it = 0, done = 0;
        int seg = 0;
        PagedWalk walk_next = walk;
        uint4 q_next[R / (8 * C)];
        if (walk.left > 0) {
            if (p.row_tiles > 1)
                lay_rows(walk.u / p.kv_heads * p.tile_rows);
            load_rows(walk, q_next);
            start_rows();
            put_rows(walk, q_next);
        }
        for (; walk.left > 0; walk = walk_next, ++seg) {
            const int n = walk.run(), tile_at = walk.u / p.kv_heads, h = walk.u - tile_at * p.kv_heads;
            const int rows = min(p.tile_rows, unit_rows - tile_at * p.tile_rows), len = walk.len, j0 = walk.j;
            const bool whole = n == walk.P;
            const int64_t slot = static_cast<int64_t>(paged_part(cta, seg)) * p.tile_rows;
            const int64_t place0 = static_cast<int64_t>(walk.b) * p.q_len * heads + h * p.group;  // the first row's, ctl->at from there
            const int begins = WAYS == 2 ? done & 1 : 0;  // the way that has the run's first page
            walk_next = walk;
            walk_next.next(p);
            if (!dead) {
                if (p.row_tiles == 1)
                    load_rows(walk_next, q_next);
                barrier_sync(2, kSoft);  // the rows' numbers are all there
            }
            uint64_t l2[N / 2];  // sums of the token's weights, two rows each
#pragma unroll
            for (int r = 0; r < N / 2; ++r)
                l2[r] = 0;
            bool bad = false, stop = false;
            const int *sees = ctl->sees + rows0;
            const float *coef = ctl->coef + rows0;
            const int open = len - (p.q_len - 1);  // tokens that every row sees
            const int first = WAYS == 2 ? way ^ begins : 0;
            for (int j = first; j < n && !dead; j += WAYS, ++it) {
                const uint32_t tile = 2 * it;
                const int sk = L::stage(way, tile), sv = L::stage(way, tile + 1);
                const int base = (j0 + j) * kPage;
                bad |= !wait(&ctl->kv_full[sk], L::phase(tile));
                const int valid = ctl->page_ok[sk] ? min(kPage, len - base) : 0;  // tokens of the page that are data
                const float ks = F::kFp8 ? scales[sk * kPage + tau] : 1.0f;
                bad |= !wait(&ctl->s_full[way], it & 1);
                tc_fence_after_sync();
                float s[N];  // the token's scores: E4M3 in log2 units, bf16 before the scale
                {
                    uint32_t raw[F::kQTerms * N / 16][16];
#pragma unroll
                    for (int i = 0; i < F::kQTerms * N / 16; ++i)
                        tmem_ld_cols(ts + i * 16, raw[i]);
                    tmem_wait_ld(raw[0]);
#pragma unroll
                    for (int i = 1; i < F::kQTerms * N / 16; ++i)
                        tmem_regs_ready(raw[i]);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&ctl->s_free[way]));
                    const uint64_t down = pack2(QueryTerms::kStep, QueryTerms::kStep), ks2 = pack2(ks, ks);
#pragma unroll
                    for (int r = 0; r < N; r += 4) {
                        float cf[4];
                        if (F::kFp8)
                            *reinterpret_cast<float4 *>(cf) = *reinterpret_cast<const float4 *>(coef + r);
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            s[r + e] = __uint_as_float(raw[r / 16][r % 16 + e]);
                            s[r + e + 1] = __uint_as_float(raw[r / 16][r % 16 + e + 1]);
                            if (F::kFp8) {
                                const uint32_t(&low)[16] = raw[(N + r) / 16 % (F::kQTerms * N / 16)];
                                const uint64_t x = fma2(pack2(__uint_as_float(low[r % 16 + e]), __uint_as_float(low[r % 16 + e + 1])),
                                                        down, pack2(s[r + e], s[r + e + 1]));
                                unpack2(mul2(x, mul2(ks2, pack2(cf[e], cf[e + 1]))), s[r + e], s[r + e + 1]);
                            }
                        }
                    }
                }
                const bool masks = base + kPage > open || valid < kPage;
                if (masks) {
#pragma unroll
                    for (int r = 0; r < N; ++r)
                        s[r] = tau < valid && base + tau < sees[r] ? s[r] : -INFINITY;
                }
                // V's page: its scales, and what lies past the tokens is no data: zero it (0 x NaN is NaN)
                float vs = 1.0f;
                if (F::kFp8 || valid < kPage) {
                    bad |= !wait(&ctl->kv_full[sv], L::phase(tile + 1));
                    if (F::kFp8)
                        vs = tau < valid ? scales[sv * kPage + tau] : 0.0f;
                    // neighbouring lanes neighbouring 16 bytes (a row a thread: 1.2 us a page)
                    for (int half = 0; half < F::kTileBytes / (kPage * 128); ++half)
                        for (int i = valid * 8 + tau; i < kPage * 8; i += 128)
                            *reinterpret_cast<uint4 *>(kv + sv * F::kTileBytes + half * kHalfPageBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                // weights at the references so far; passed by somebody: again at new ones
                const float to_log2 = F::kFp8 ? 1.0f : p.scale_log2;
                const uint64_t c2 = pack2(to_log2, to_log2), vs2 = pack2(vs, vs);
                float w[N];
                uint64_t ls2[N / 2];
                float top = 0.0f, most = F::kFp8 ? vs * (kPagedMost / kPagedWideScale) : 0.0f;
                // At new references (`wide`) the weight comes before the scale, since scale x unit may pass fp32, and 0 times that
                // is NaN: pages with a scale where it may, by what `most` starts from, always go there.  (In this order everywhere
                // 64 rows spill: 32 requests of 31000 tokens 323 us for 317.)
                auto weigh = [&](auto wide) {
#pragma unroll
                    for (int r = 0; r < N; r += 4) {
                        float nr[4], un[4];
                        *reinterpret_cast<float4 *>(nr) = *reinterpret_cast<const float4 *>(&ctl->nref[t][r]);
                        if (F::kFp8)
                            *reinterpret_cast<float4 *>(un) = *reinterpret_cast<const float4 *>(&ctl->unit[t][r]);
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const int k = r + e;
                            float x, y;
                            unpack2(F::kFp8 ? add2(pack2(s[k], s[k + 1]), pack2(nr[e], nr[e + 1]))
                                            : fma2(pack2(s[k], s[k + 1]), c2, pack2(nr[e], nr[e + 1])),
                                    x, y);
                            if (masks) {
                                x = s[k] == -INFINITY ? -INFINITY : x;
                                y = s[k + 1] == -INFINITY ? -INFINITY : y;
                            }
                            top = max3(top, x, y);
                            w[k] = exp2_approx(x);
                            w[k + 1] = exp2_approx(y);
                            ls2[k / 2] = pack2(w[k], w[k + 1]);
                            if (F::kFp8) {
                                const uint64_t un2 = pack2(un[e], un[e + 1]);
                                unpack2(decltype(wide)::value ? mul2(mul2(ls2[k / 2], un2), vs2) : mul2(ls2[k / 2], mul2(vs2, un2)), w[k], w[k + 1]);
                                most = max3(most, w[k], w[k + 1]);
                            }
                        }
                    }
                };
                bool moves = j < WAYS;  // a unit's first page: no references yet
                if (!moves) {
                    weigh(std::false_type());
                    moves = barrier_any(3 + t, 128, top > kPagedLag || most > kPagedMost || bad);
                }
                if (moves) {
                    // new references: the largest scores; E4M3: and the largest weight x V scale, in log2
                    const float vs_log2 = F::kFp8 ? log2f(vs) : 0.0f;
#pragma unroll
                    for (int r = 0; r < N; ++r) {
                        const float x = s[r] * to_log2;
                        const int m = __reduce_max_sync(0xffffffffu, float_int(x));
                        const int o = F::kFp8 ? __reduce_max_sync(0xffffffffu, float_int(x + vs_log2)) : 0;
                        if (lane == r) {
                            ctl->wmax[t][warp & 3][r] = m;
                            if (F::kFp8)
                                ctl->omax[t][warp & 3][r] = o;
                        }
                    }
                    stop = barrier_any(3 + t, 128, bad);  // (what one warp saw alone is no reason to leave the others)
                    if (stop)
                        break;
                    if (tau < N) {
                        const float old = -ctl->nref[t][tau];
                        const float m = fmaxf(old, int_float(max(max(ctl->wmax[t][0][tau], ctl->wmax[t][1][tau]),
                                                                 max(ctl->wmax[t][2][tau], ctl->wmax[t][3][tau]))));
                        const float lfac = rescale(old, m);
                        ctl->nref[t][tau] = -m;
                        ctl->lfac[t][tau] = ctl->fac[t][tau] = lfac;
                        if (F::kFp8) {
                            const float o = int_float(max(max(ctl->omax[t][0][tau], ctl->omax[t][1][tau]),
                                                          max(ctl->omax[t][2][tau], ctl->omax[t][3][tau])));
                            const float before = ctl->vtop[t][tau] * lfac, unit = ctl->unit[t][tau];
                            const float most_now = fmaxf(before, o == -INFINITY ? 0.0f : exp2_approx(o - m));
                            // the power of two that brings it to [2^9, 2^10): room for 2^5 of growth until the next time.  Where every
                            // product so far is 0 the largest there is: the first one that is not passes kPagedMost, or is held in it.
                            const int e = static_cast<int>(__float_as_uint(most_now) >> 23);
                            const float to_unit = __int_as_float(max(10, min(244, 263 - e)) << 23);
                            ctl->vtop[t][tau] = most_now;
                            ctl->unit[t][tau] = to_unit;
                            // (4 at most: to_unit x before is below 2^10, unit x vtop from 2^9 on or unit the largest there is)
                            ctl->fac[t][tau] = lfac * to_unit * (1.0f / unit);
                        }
                    }
                    barrier_sync(3 + t, 128);
#pragma unroll
                    for (int r = 0; r < N; r += 2) {
                        const float2 f = *reinterpret_cast<const float2 *>(&ctl->lfac[t][r]);
                        l2[r / 2] = mul2(l2[r / 2], pack2(f.x, f.y));
                    }
                    if (j >= WAYS) {  // what the pages before left in O
                        bad |= !wait(&ctl->o_done[way], (it - 1) & 1);
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int i = 0; i < L::kOCols; i += 16) {
                            uint32_t o[16];
                            tmem_ld_cols(to + i, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * ctl->fac[t][i % N + k]);
                            tmem_st_cols(to + i, o);
                        }
                        tmem_wait_st();
                    }
                    weigh(std::true_type());
                }
                if (stop)
                    break;
                // (the product with the weights before has to be over)
                if (it > 0)
                    bad |= !wait(&ctl->o_done[way], (it - 1) & 1);
                if (!F::kFp8) {
#pragma unroll
                    for (int r = 0; r < N; r += 8)
                        *reinterpret_cast<uint4 *>(pbuf + (r / 8) * 2048) =
                            make_uint4(f32x2_to_bf16x2(w[r], w[r + 1]), f32x2_to_bf16x2(w[r + 2], w[r + 3]),
                                       f32x2_to_bf16x2(w[r + 4], w[r + 5]), f32x2_to_bf16x2(w[r + 6], w[r + 7]));
                } else {
#pragma unroll
                    for (int r = 0; r < N; r += 16) {
                        uint32_t c[F::kPTerms][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t a[F::kPTerms], b[F::kPTerms];
                            e4m3_terms<WeightTerms>(w[r + 4 * i], w[r + 4 * i + 1], a);
                            e4m3_terms<WeightTerms>(w[r + 4 * i + 2], w[r + 4 * i + 3], b);
#pragma unroll
                            for (int k = 0; k < F::kPTerms; ++k)
                                c[k][i] = a[k] | b[k] << 16;
                        }
#pragma unroll
                        for (int k = 0; k < F::kPTerms; ++k)
                            *reinterpret_cast<uint4 *>(pbuf + ((k * N + r) / 16) * 2048) = make_uint4(c[k][0], c[k][1], c[k][2], c[k][3]);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_addr(&ctl->p_full[way]));
                    mbar_arrive(smem_addr(&ctl->kv_empty[sk]));
                    mbar_arrive(smem_addr(&ctl->kv_empty[sv]));
                }
#pragma unroll
                for (int r = 0; r < N / 2; ++r)
                    l2[r] = add2(l2[r], ls2[r]);
            }
            done += n;
            // ---- the run's part of the unit ----
            if (!dead) {
                float l[N];
#pragma unroll
                for (int r = 0; r < N; r += 2)
                    unpack2(l2[r / 2], l[r], l[r + 1]);
                const float sum = lanes_sum<N>(l, lane);
                if (lane < N)
                    ctl->wsum[t][warp & 3][lane] = sum;
                bad |= stop;
                if (first < n && !bad)
                    bad |= !wait(&ctl->o_done[way], (it - 1) & 1);
                bad |= !wait(&ctl->q_taken, seg & 1);  // (who issues the products has seen this unit's rows)
                dead = barrier_any(2, kSoft, bad);
            }
            if (dead) {
                for (int r = tid >> 5; r < rows; r += 4 * C) {
                    if (!whole) {
                        if (lane == 0)
                            p.part_lse[slot + r] = INFINITY;
                        continue;
                    }
                    const int i = (tile_at * p.tile_rows + r) / p.group, g = tile_at * p.tile_rows + r - i * p.group;
                    const int64_t at = place0 + i * heads + g;
                    reinterpret_cast<uint2 *>(p.out + at * kDim)[lane] = make_uint2(0u, 0u);
                    if (p.lse && lane == 0)
                        p.lse[at] = -INFINITY;
                }
                continue;
            }
            // the scores of this unit have all been read: the next one's rows may take the place of its
            if (p.row_tiles == 1 && walk_next.left > 0)
                put_rows(walk_next, q_next);
            float top = 0.0f, all = 0.0f;
            if (tid < R) {
                float m[WAYS], sum[WAYS], M = -INFINITY;
#pragma unroll
                for (int c = 0; c < WAYS; ++c) {
                    const int chain = c * GROUPS + tid / N;
                    const float *x = &ctl->wsum[chain][0][tid % N];
                    m[c] = -ctl->nref[chain][tid % N];
                    sum[c] = (x[0] + x[N]) + (x[2 * N] + x[3 * N]);
                    M = fmaxf(M, m[c]);
                }
#pragma unroll
                for (int c = 0; c < WAYS; ++c) {
                    m[c] = sum[c] > 0.0f ? rescale(m[c], M) : 0.0f;
                    all += m[c] * sum[c];
                }
#pragma unroll
                for (int c = 0; c < WAYS; ++c)  // 0: nothing, and what stands in O may be anything
                    ctl->share[c][tid] =
                        sum[c] > 0.0f ? __fdividef(m[c], all) * (F::kFp8 ? 2048.0f / ctl->unit[c * GROUPS + tid / N][tid % N] : 1.0f) : 0.0f;
                top = M;
            }
            barrier_sync(2, kSoft);
            tc_fence_after_sync();
            if (p.row_tiles == 1)
                start_rows();
            if (tid < rows) {
                const float e = all > 0.0f ? top + log2f(all) : -INFINITY;
                if (!whole)
                    p.part_lse[slot + tid] = e;
                else if (p.lse)
                    p.lse[place0 + ctl->at[tid]] = e * kLn2;
            }
            // a thread a dim: the warpgroups take 8 rows at a time in turn, with all ways' shares of them
            for (int r0 = t * 8; r0 < rows; r0 += C * 8) {
                float acc[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    acc[k] = 0.0f;
#pragma unroll
                for (int c = 0; c < WAYS; ++c) {
                    if (WAYS == 2 && (c ^ begins) >= n)  // a way without a page
                        continue;
                    const uint32_t from = tmem + c * L::kWayCols + GROUPS * L::kSCols + r0 / N * L::kOCols + lanes + r0 % N;
                    uint32_t o[F::kPTerms][8];
#pragma unroll
                    for (int k = 0; k < F::kPTerms; ++k)
                        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                                     : "=r"(o[k][0]), "=r"(o[k][1]), "=r"(o[k][2]), "=r"(o[k][3]), "=r"(o[k][4]),
                                       "=r"(o[k][5]), "=r"(o[k][6]), "=r"(o[k][7])
                                     : "r"(from + k * N));
#pragma unroll
                    for (int k = 0; k < F::kPTerms; ++k)
                        asm volatile("tcgen05.wait::ld.sync.aligned;"
                                     : "+r"(o[k][0]), "+r"(o[k][1]), "+r"(o[k][2]), "+r"(o[k][3]), "+r"(o[k][4]),
                                       "+r"(o[k][5]), "+r"(o[k][6]), "+r"(o[k][7])::"memory");
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float x = __uint_as_float(o[0][k]);
                        if (F::kFp8)
                            x += WeightTerms::kStep * (__uint_as_float(o[F::kPTerms / 2][k]) +
                                                       WeightTerms::kStep * __uint_as_float(o[F::kPTerms - 1][k]));
                        const float share = ctl->share[c][r0 + k];
                        acc[k] += share != 0.0f ? share * x : 0.0f;
                    }
                }
                if (whole) {
                    uint16_t *out = p.out + place0 * kDim + tau;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (r0 + k < rows)
                            out[static_cast<int64_t>(ctl->at[r0 + k]) * kDim] = static_cast<uint16_t>(f32x2_to_bf16x2(acc[k], 0.0f));
                } else {
                    float *out = p.part_o + (slot + r0) * kDim + tau;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (r0 + k < rows)
                            out[k * kDim] = acc[k];
                }
            }
            tc_fence_before_sync();
            if (p.row_tiles > 1 && walk_next.left > 0) {  // tiles of rows: where they lie changes with the unit
                barrier_sync(2, kSoft);
                lay_rows(walk_next.u / p.kv_heads * p.tile_rows);
                load_rows(walk_next, q_next);
                start_rows();
                put_rows(walk_next, q_next);
            }
        }
        tc_fence_before_sync();
    }
    __syncthreads();
    if (warp == 4 * C + 1)
        tmem_dealloc(tmem, L::kTmem);
}

// ---------------------------------------------------------------------------
// The units that a range's end cuts, 8 / WPR of their rows a block, WPR warps a row that take its parts in turn.  UNITS:
// block x takes unit x, if it is cut; else the one that CTA x + 1 is the first to go on with.
template <int WPR, bool UNITS>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedParams p)
{
    constexpr int kRows = 8 / WPR;
    __shared__ PagedScan scan;
    __shared__ float4 s_acc[8][32];
    __shared__ float s_m[8], s_sum[8];
    __shared__ int s_bad[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = warp % WPR;
    const int units = p.row_tiles * p.kv_heads, x = blockIdx.x;
    int before;
    const PagedWork work = paged_find<256>(p, &scan, UNITS ? x / units : 0, before, [&](const PagedWork &all) {
        const PagedSplit s(all, p);
        return !UNITS && x + 1 < s.ctas ? s.start(x + 1) : -1;
    });
    const PagedSplit split(work, p);
    const PagedAt at = UNITS ? PagedAt{x / units, x % units, 0} : scan.at;
    const int P = at.b < p.batch ? pages_of(paged_len(p, at.b)) : 0;
    // the slots of the unit's pages [from, from + P), and the CTA that has the first
    const int from = UNITS ? before + at.u * (P + p.lead) + p.lead : (x + 1 < split.ctas ? split.start(x + 1) : 0) - at.j;
    const PagedParts where(split, from, P, p.lead);
    const int parts = where.n;
    griddep_wait();  // also where there is nothing to do: who waits for this grid reads what both have written
    if (parts < 2 || (!UNITS && (at.j <= 0 || where.first != x)))
        return;  // no unit goes on there, or another block has it
    const int h = at.u % p.kv_heads, row0 = at.u / p.kv_heads * p.tile_rows;
    const int rows = min(p.tile_rows, p.q_len * p.group - row0);
    const int r = blockIdx.y * kRows + warp / WPR;
    auto slot = [&](int i) { return static_cast<int64_t>(where.part(i)) * p.tile_rows + r; };
    float M = -INFINITY, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    bool bad = false;
    const bool exists = r < rows;
    const int mine = exists && parts > sub ? (parts - sub + WPR - 1) / WPR : 0;
    for (int i0 = 0; i0 < mine; i0 += 32) {
        const int end = min(32, mine - i0);
        const float x = lane < end ? __ldcg(p.part_lse + slot(sub + (i0 + lane) * WPR)) : -INFINITY;
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
        for (int i = 0; i < end; i += 8) {
            float4 v[8];  // under way together
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = i + k < end ? __ldcg(reinterpret_cast<const float4 *>(p.part_o + slot(sub + (i0 + i + k) * WPR) * kDim) + lane)
                                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float fi = __shfl_sync(0xffffffffu, f, i + k);
                const bool some = fi != 0.0f;
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
    const bool none = bad || sum == 0.0f;
    const float inv = none ? 0.0f : 1.0f / sum;
    const int64_t to = (static_cast<int64_t>(at.b) * p.q_len + (row0 + r) / p.group) * p.kv_heads * p.group + h * p.group +
                       (row0 + r) % p.group;
    uint2 w;
    w.x = none ? 0u : f32x2_to_bf16x2(acc.x * inv, acc.y * inv);
    w.y = none ? 0u : f32x2_to_bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2 *>(p.out + to * kDim + lane * 4) = w;
    if (p.lse && lane == 0)
        p.lse[to] = none ? -INFINITY : (M + log2f(sum)) * kLn2;
}

}  // namespace msa

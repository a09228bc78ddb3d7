// Attention over the blocks the indexer selected (block_attn.cuh) and of a batch
// that shares a prefix (prefix_attn.cuh): argument checks and launches.
#include "block_attn.cuh"
#include "prefix_attn.cuh"

namespace msa {

bool test_withhold_pages();  // msa_indexer_test_withhold_pages

// Tensor map of a paged cache as [page][head][token][dim]; strides in elements
// (page, token, head).  The stride of an axis of length 1 is never used.
bool make_cache_map(CUtensorMap *map, const void *base, const int64_t *strides, int64_t pages, int heads, bool fp8)
{
    const cuuint64_t size = fp8 ? 1 : 2;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kDim), static_cast<cuuint64_t>(kPage),
                                static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(pages)};
    const cuuint64_t bytes[3] = {static_cast<cuuint64_t>(strides[1]) * size,
                                 static_cast<cuuint64_t>(heads > 1 ? strides[2] : kDim) * size,
                                 static_cast<cuuint64_t>(pages > 1 ? strides[0] : kDim) * size};
    const cuuint32_t box[4] = {fp8 ? 128u : 64u, 128u, 1u, 1u};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    // What L2 fetches at a time: 256 bytes, but no more than an E4M3 token's 128 where the next token's do not follow them
    // (All pages of 32 requests of 31000 tokens, four heads a token: 236 us with 256, 170 with 128; heads apart, 165 either way.
    // 16 blocks each of 32 requests: 25.6 and 22.9; of 128: 75.1 and 68.3; of 32 with eight heads 40.9 and 35.6; of 1: 9.0 and 9.0.)
    const bool pieces = fp8 && strides[1] != kDim;
    return encode_map(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                      const_cast<void *>(base), dims, bytes, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, pieces ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// A cache's address and strides: 16-byte multiples, positive, within a tensor map's 2^40-byte strides.
bool cache_ok(const void *base, const int64_t *strides, int64_t pages, int heads, bool fp8)
{
    if (!base || !strides || (reinterpret_cast<uintptr_t>(base) & 15))
        return false;
    const int64_t unit = fp8 ? 16 : 8;
    for (int i = 0; i < 3; ++i) {
        if ((i == 0 && pages == 1) || (i == 2 && heads == 1))
            continue;
        if (strides[i] < kDim || strides[i] % unit || strides[i] >= (int64_t{1} << 38))
            return false;
    }
    return true;
}

bool unaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

template <class F, int MT, bool OWN>
bool block_attn_allowed(int dev)
{
    static std::atomic<bool> done[kMaxDevices];
    return allow_smem(block_attn_kernel<F, MT, OWN>, block_attn_smem<F>(MSA_MAX_TOPK), dev, done);
}

// Clusters of `size` CTAs (two an SM) that the device runs at the same time: those of 4 or 8 do not fill it, as a
// cluster stays within one of its parts.  0 where the query fails.  Asked of one kernel without the mass scratch: every
// form of it gives the same counts for 2 to 8 CTAs, with any scratch (152, 97, 74, 58, 46, 38, 36 on a GB300).
int resident_clusters(int dev, int size)
{
    static std::atomic<int> cache[kMaxDevices][9];
    int v = dev >= 0 && dev < kMaxDevices ? cache[dev][size].load(std::memory_order_relaxed) : 0;
    if (v > 0)
        return v;
    auto *kernel = block_attn_kernel<AttnBf16, 1, false>;
    const size_t smem = block_attn_smem<AttnBf16>(0);
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = smem;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!block_attn_allowed<AttnBf16, 1, false>(dev) ||
        cudaOccupancyMaxActiveClusters(&v, kernel, &cfg) != cudaSuccess)
        return 0;
    if (dev >= 0 && dev < kMaxDevices)
        cache[dev][size].store(v, std::memory_order_relaxed);
    return v;
}

// CTAs of the cluster that walks one list of at most `pages` pages: the most that still run all at once, and no more
// than it takes to make the longest share as short.  16 blocks, 4 KV heads: 19 requests in clusters of 3 21.1 us (E4M3
// 17.7), in clusters of 4 that do not all fit 27.4 (23.7); 24 requests 18.6 (E4M3) against 21.7 in clusters of 2.
int block_attn_split(int64_t units, int pages, int dev)
{
    int s = 8;
    while (s > 1 && (s > pages || units > resident_clusters(dev, s)))
        --s;
    const int longest = (pages + s - 1) / s;
    return (pages + longest - 1) / longest;
}

template <class F, int MT, bool OWN>
msa_status launch_block_attn(const BlockAttnParams &p, int64_t units, int split, int dev, cudaStream_t st,
                             bool dependent = false)
{
    const size_t smem = block_attn_smem<F>(p.mass ? (p.k + split - 1) / split : 0);
    auto *kernel = block_attn_kernel<F, MT, OWN>;
    if (!block_attn_allowed<F, MT, OWN>(dev))
        return MSA_ERR_CUDA;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(units * split));
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    // dependent: beside prefix_attn_kernel, CTAs start where it leaves room
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

static msa_status sparse_entry(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                               const float *k_scale, const void *v, const int64_t *v_strides, const float *v_scale,
                               int64_t num_pages, const int32_t *block_table, int64_t bt_stride,
                               const int32_t *seq_lens, int batch, int q_len, int kv_heads, int group,
                               int max_model_len, const int32_t *ids, int sel_heads, int topk, float scale, void *out,
                               float *out_lse, float *out_mass, void *workspace, size_t workspace_bytes, void *stream,
                               bool fp8)
{
    if (batch < 0 || q_len < 1 || kv_heads < 1 || group < 1 || sel_heads < 1 || topk < 1 || num_pages < 1 ||
        bt_stride < 1 || max_model_len < 1 || kv_heads % sel_heads || !(scale > 0.0f) || !(scale < INFINITY))
        return MSA_ERR_INVALID_ARG;
    if (batch > MSA_MAX_BATCH || num_pages > (int64_t{1} << 24) || topk > MSA_MAX_TOPK || group > MSA_MAX_GROUP ||
        kv_heads > 1024 || q_len > 64 || static_cast<int64_t>(batch) * q_len * kv_heads > (int64_t{1} << 27))
        return MSA_ERR_UNSUPPORTED;
    if (batch == 0)  // (an empty tensor has no address)
        return MSA_OK;
    if (!q || !block_table || !seq_lens || !ids || !out || !workspace || !cache_ok(k, k_strides, num_pages, kv_heads, fp8) ||
        !cache_ok(v, v_strides, num_pages, kv_heads, fp8) || unaligned(q, 16) || q_stride % 8 ||
        q_stride < static_cast<int64_t>(kv_heads) * group * kDim || unaligned(out, 16) || unaligned(workspace, 256))
        return MSA_ERR_INVALID_ARG;
    if (fp8 && (!k_scale || !v_scale || unaligned(k_scale, 16) || unaligned(v_scale, 16)))
        return MSA_ERR_INVALID_ARG;
    if (workspace_bytes < kHeaderBytes)
        return MSA_ERR_WORKSPACE_TOO_SMALL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return MSA_ERR_CUDA;
    const int sms = device_sms(dev);
    if (sms <= 0)
        return MSA_ERR_CUDA;
    BlockAttnParams p;
    std::memset(&p, 0, sizeof p);
    if (!make_cache_map(&p.kmap, k, k_strides, num_pages, kv_heads, fp8) ||
        !make_cache_map(&p.vmap, v, v_strides, num_pages, kv_heads, fp8))
        return MSA_ERR_CUDA;
    p.q = static_cast<const uint16_t *>(q);
    p.kscale = k_scale;
    p.vscale = v_scale;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.ids = ids;
    p.out = static_cast<uint16_t *>(out);
    p.lse = out_lse;
    p.mass = out_mass;
    p.fault = &static_cast<WorkspaceHeader *>(workspace)->fault;
    p.q_stride = q_stride;
    p.bt_stride = bt_stride;
    p.num_pages = num_pages;
    p.batch = batch;
    p.q_len = q_len;
    p.kv_heads = kv_heads;
    p.sel_heads = sel_heads;
    p.group = group;
    p.k = topk;
    p.seq_limit = static_cast<int>(std::min<int64_t>(max_model_len, kPage * bt_stride));
    p.scale_log2 = scale * kLog2e;
    p.withhold = test_withhold_pages();
    const int64_t units = static_cast<int64_t>(batch) * q_len * kv_heads;
    const int split = block_attn_split(units, topk, dev);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (fp8)
        return group <= 16   ? launch_block_attn<AttnFp8, 1, false>(p, units, split, dev, st)
               : group <= 32 ? launch_block_attn<AttnFp8, 2, false>(p, units, split, dev, st)
                             : launch_block_attn<AttnFp8, 4, false>(p, units, split, dev, st);
    return group <= 16   ? launch_block_attn<AttnBf16, 1, false>(p, units, split, dev, st)
           : group <= 32 ? launch_block_attn<AttnBf16, 2, false>(p, units, split, dev, st)
                         : launch_block_attn<AttnBf16, 4, false>(p, units, split, dev, st);
}

// The units of a batch's rows (a tile of 128 rows of a KV head where they do not fill more).
static void prefix_units(PrefixParts &a, int64_t rows, int kv_heads)
{
    a.tile_rows = rows <= 128 ? 128 : 256;
    a.ways = 256 / a.tile_rows;
    a.head_tiles = static_cast<int>((rows + a.tile_rows - 1) / a.tile_rows);
    a.units = a.head_tiles * kv_heads;
}

// Bytes: rows of the prefix's slots and one own part a row and head, 516 each.  The slots (34 MB) do not shrink with the
// batch or the prefix: how many CTAs share it is worked out on the device, from the live lengths.
static size_t prefix_workspace(int max_rows, int group, int kv_heads)
{
    PrefixParts a;
    const int64_t rows = static_cast<int64_t>(max_rows) * group;
    prefix_units(a, rows, kv_heads);
    const size_t prefix = (static_cast<size_t>(kPrefixMaxGrid) + a.units) * 256;
    return kHeaderBytes + (prefix + static_cast<size_t>(rows) * kv_heads) * (kDim + 1) * sizeof(float) + 4 * 256;
}

static void prefix_parts(PrefixParts &a, int batch, int q_len, int group, int kv_heads, int max_prefix_len,
                         uint8_t *workspace)
{
    std::memset(&a, 0, sizeof a);
    a.batch = batch;
    a.q_len = q_len;
    a.group = group;
    a.kv_heads = kv_heads;
    a.rows = batch * q_len * group;
    prefix_units(a, a.rows, kv_heads);
    // An own page takes an SM about as long as a 128-row tile's page of the prefix (1350 cycles) where the stream
    // bounds it (16 rows), and its share of the mma.sync rate where that does.  Measured on 11 batches: for 16 rows
    // 6/8 and 7/8 are the fastest (64 requests over 32768: 96 us, 99 at 8/8, 113 at 5/8), for 32 and 64 rows 12/8 a
    // tile of 16 (8 x 4 x 8 over 16384 + 8000 tokens: 26 us, 27 at 10/8, 31 at 8/8; 16 x 4 x 16 over 8192 + 37000: 60,
    // 62 and 66, 72 at 14/8).
    const int tiles = (q_len * group + 15) / 16;
    a.own_cost = tiles == 1 ? 7 : 12 * tiles;
    a.own_most = batch > 0 ? INT32_MAX / batch : 0;
    a.limit = max_prefix_len;
    uint8_t *at = workspace + kHeaderBytes;
    auto take = [&](size_t bytes) {
        uint8_t *here = at;
        at += round_up(bytes, 256);
        return here;
    };
    const size_t rows = (static_cast<size_t>(kPrefixMaxGrid) + a.units) * 256;
    const size_t own_rows = static_cast<size_t>(a.rows) * kv_heads;
    a.lse = reinterpret_cast<float *>(take(rows * sizeof(float)));
    a.own_lse = reinterpret_cast<float *>(take(own_rows * sizeof(float)));
    a.o = reinterpret_cast<float *>(take(rows * kDim * sizeof(float)));
    a.own_o = reinterpret_cast<float *>(take(own_rows * kDim * sizeof(float)));
}

template <int WPR, int WARPS>
static msa_status launch_join(const JoinParams &p, int64_t rows, cudaStream_t st)
{
    constexpr int kRows = WARPS / WPR;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg =
        pdl_config(dim3(static_cast<unsigned>((rows + kRows - 1) / kRows)), dim3(32 * WARPS), 0, st, attr);
    return cudaLaunchKernelEx(&cfg, join_kernel<WPR, WARPS>, p) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

static msa_status prefix_entry(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides, const void *v,
                               const int64_t *v_strides, int64_t num_pages, const int32_t *prefix_table,
                               const int32_t *prefix_len, int max_prefix_len, const int32_t *block_table,
                               int64_t bt_stride, const int32_t *seq_lens, int batch, int q_len, int kv_heads,
                               int group, int max_model_len, float scale, void *out, float *out_lse, void *workspace,
                               size_t workspace_bytes, void *stream)
{
    if (batch < 0 || q_len < 1 || kv_heads < 1 || group < 1 || num_pages < 1 || bt_stride < 1 || max_model_len < 1 ||
        max_prefix_len < 0 || !(scale > 0.0f) || !(scale < INFINITY))
        return MSA_ERR_INVALID_ARG;
    if (batch > MSA_MAX_BATCH || num_pages > (int64_t{1} << 24) || group > MSA_MAX_GROUP || kv_heads > 1024 ||
        q_len > 64 || static_cast<int64_t>(batch) * q_len * kv_heads * group > (int64_t{1} << 27))
        return MSA_ERR_UNSUPPORTED;
    if (batch == 0)  // (an empty tensor has no address)
        return MSA_OK;
    if (!q || !block_table || !seq_lens || (!prefix_table && max_prefix_len > 0) || !prefix_len || !out || !workspace ||
        !cache_ok(k, k_strides, num_pages, kv_heads, false) || !cache_ok(v, v_strides, num_pages, kv_heads, false) ||
        unaligned(q, 16) || q_stride % 8 || q_stride < static_cast<int64_t>(kv_heads) * group * kDim ||
        unaligned(out, 16) || unaligned(workspace, 256))
        return MSA_ERR_INVALID_ARG;
    PrefixAttnParams p;
    std::memset(&p, 0, sizeof p);
    if (workspace_bytes < prefix_workspace(batch * q_len, group, kv_heads))
        return MSA_ERR_WORKSPACE_TOO_SMALL;
    prefix_parts(p.parts, batch, q_len, group, kv_heads, max_prefix_len, static_cast<uint8_t *>(workspace));
    if ((static_cast<int64_t>(max_prefix_len) + kPage - 1) / kPage * p.parts.units > (1 << 30))
        return MSA_ERR_UNSUPPORTED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return MSA_ERR_CUDA;
    const int sms = device_sms(dev);
    if (sms <= 0)
        return MSA_ERR_CUDA;
    if (!make_cache_map(&p.kmap, k, k_strides, num_pages, kv_heads, false) ||
        !make_cache_map(&p.vmap, v, v_strides, num_pages, kv_heads, false))
        return MSA_ERR_CUDA;
    p.q = static_cast<const uint16_t *>(q);
    p.prefix_table = prefix_table;
    p.prefix_len = prefix_len;
    p.seq_lens = seq_lens;
    p.fault = &static_cast<WorkspaceHeader *>(workspace)->fault;
    p.q_stride = q_stride;
    p.num_pages = num_pages;
    p.scale_log2 = scale * kLog2e;
    p.withhold = test_withhold_pages();
    p.parts.seq_limit = static_cast<int>(std::min<int64_t>(max_model_len, kPage * bt_stride));
    p.parts.grid = std::min(sms, kPrefixMaxGrid);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    static std::atomic<bool> allowed[kMaxDevices];
    if (!allow_smem(prefix_attn_kernel, kPrefixSmemBytes, dev, allowed))
        return MSA_ERR_CUDA;
    BlockAttnParams o;
    std::memset(&o, 0, sizeof o);
    o.kmap = p.kmap;
    o.vmap = p.vmap;
    o.q = p.q;
    o.block_table = block_table;
    o.seq_lens = seq_lens;
    o.part = p.parts.own_o;
    o.lse = p.parts.own_lse;
    o.fault = p.fault;
    o.q_stride = q_stride;
    o.bt_stride = bt_stride;
    o.num_pages = num_pages;
    o.batch = batch;
    o.q_len = q_len;
    o.kv_heads = kv_heads;
    o.sel_heads = 1;
    o.group = group;
    o.seq_limit = p.parts.seq_limit;
    o.row_tiles = (p.parts.q_len * group + kAttnMaxRows - 1) / kAttnMaxRows;
    o.scale_log2 = p.scale_log2;
    o.withhold = p.withhold;
    // Clusters of up to 4 (16 requests x 4 positions x 16 heads over 8192 + 37000 tokens, at that time: 155 us
    // unsplit, 88 with 2, 65 with 4, 68 with 8; 8 x 4 x 8 over 16384 + 8000: 46, 32, 30.5, 36), of fewer where a request
    // cannot have as many pages (16 x 16 rows over 2048 + 300 tokens a request: 15.3 us, 17.3 with 4).
    const int64_t units = static_cast<int64_t>(batch) * kv_heads * o.row_tiles;
    const int own_pages = p.parts.seq_limit / kPage + (p.parts.seq_limit % kPage != 0);  // at most
    const int split = block_attn_split(units, own_pages >= 4 ? 4 : own_pages >= 2 ? 2 : 1, dev);
    const int unit_rows = std::min(q_len * group, kAttnMaxRows);
    auto launch_own = [&](bool dependent) {
        return unit_rows <= 16   ? launch_block_attn<AttnBf16, 1, true>(o, units, split, dev, st, dependent)
               : unit_rows <= 32 ? launch_block_attn<AttnBf16, 2, true>(o, units, split, dev, st, dependent)
                                 : launch_block_attn<AttnBf16, 4, true>(o, units, split, dev, st, dependent);
    };
    // Few own CTAs start first, on SMs kept free for them (a CTA may take one by itself), and the prefix as their
    // dependent: it ends last, and the join waits for one grid's end instead of two in a row (2 requests over 1000
    // tokens: 11.7 us against 11.95, over 4133: 13.3 and 13.6, over 16384: 18.5 and 20.7; 1 over 30000: 26.5 and 28.2).
    // Many would hold the prefix's CTAs up (4 requests over 8192, already no gain: 18.8 both ways).
    const bool own_first = units * split <= sms / 8;
    if (own_first) {
        p.parts.spare = static_cast<int>(units * split);
        const msa_status own = launch_own(false);
        if (own != MSA_OK)
            return own;
    }
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3(p.parts.grid), dim3(kPrefixThreads), kPrefixSmemBytes, st, attr);
    cfg.numAttrs = own_first ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, prefix_attn_kernel, p) != cudaSuccess)
        return MSA_ERR_CUDA;
    if (!own_first) {
        const msa_status own = launch_own(true);
        if (own != MSA_OK)
            return own;
    }
    JoinParams j;
    std::memset(&j, 0, sizeof j);
    j.parts = p.parts;
    j.prefix_len = prefix_len;
    j.seq_lens = seq_lens;
    j.out = static_cast<uint16_t *>(out);
    j.lse = out_lse;
    const int64_t rows = static_cast<int64_t>(p.parts.rows) * kv_heads;
    // Few rows have many parts each: more warps to a row.  Many rows: large blocks, since each works out the split and
    // not all are resident when the parts are done (64 x 32768: 87.4 us with 16 warps a block, 88.7 with 8).
    return rows <= 4 * sms ? launch_join<8, 8>(j, rows, st) : rows <= 16 * sms ? launch_join<2, 8>(j, rows, st)
                                                                               : launch_join<1, 16>(j, rows, st);
}

}  // namespace msa

using namespace msa;

extern "C" size_t msa_attention_prefix_workspace_bytes(int max_rows, int heads, int kv_heads, int max_prefix_len)
{
    if (max_rows < 0 || kv_heads < 1 || heads < kv_heads || heads % kv_heads || max_prefix_len < 0)
        return 0;
    return prefix_workspace(max_rows, heads / kv_heads, kv_heads);
}

extern "C" msa_status msa_attention_prefix(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                                           const void *v, const int64_t *v_strides, int64_t num_pages,
                                           const int32_t *prefix_table, const int32_t *prefix_len, int max_prefix_len,
                                           const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                                           int batch, int q_len, int kv_heads, int group, int max_model_len,
                                           float scale, void *out, float *out_lse, void *workspace,
                                           size_t workspace_bytes, void *stream)
{
    return prefix_entry(q, q_stride, k, k_strides, v, v_strides, num_pages, prefix_table, prefix_len, max_prefix_len,
                        block_table, bt_stride, seq_lens, batch, q_len, kv_heads, group, max_model_len, scale, out,
                        out_lse, workspace, workspace_bytes, stream);
}

extern "C" msa_status msa_attention_sparse(const void *q, int64_t q_stride, const void *k, const int64_t *k_strides,
                                           const void *v, const int64_t *v_strides, int64_t num_pages,
                                           const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                                           int batch, int q_len, int kv_heads, int group, int max_model_len,
                                           const int32_t *ids, int sel_heads, int topk, float scale, void *out,
                                           float *out_lse, float *out_mass, void *workspace, size_t workspace_bytes,
                                           void *stream)
{
    return sparse_entry(q, q_stride, k, k_strides, nullptr, v, v_strides, nullptr, num_pages, block_table, bt_stride,
                        seq_lens, batch, q_len, kv_heads, group, max_model_len, ids, sel_heads, topk, scale, out,
                        out_lse, out_mass, workspace, workspace_bytes, stream, false);
}

extern "C" msa_status msa_attention_sparse_fp8(const void *q, int64_t q_stride, const void *k,
                                               const int64_t *k_strides, const float *k_scale, const void *v,
                                               const int64_t *v_strides, const float *v_scale, int64_t num_pages,
                                               const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens,
                                               int batch, int q_len, int kv_heads, int group, int max_model_len,
                                               const int32_t *ids, int sel_heads, int topk, float scale, void *out,
                                               float *out_lse, float *out_mass, void *workspace,
                                               size_t workspace_bytes, void *stream)
{
    return sparse_entry(q, q_stride, k, k_strides, k_scale, v, v_strides, v_scale, num_pages, block_table, bt_stride,
                        seq_lens, batch, q_len, kv_heads, group, max_model_len, ids, sel_heads, topk, scale, out,
                        out_lse, out_mass, workspace, workspace_bytes, stream, true);
}

// csrc/paged_split.cuh compiled for the host: what each CTA of the attention over all pages takes of a batch, and where the
// join looks for the parts, by the functions that the kernels call.
#define __host__
#define __device__
#define __forceinline__ inline
#include "paged_split.cuh"

using namespace msa;

namespace {
struct Batch {
    const int32_t *seq_lens;
    int seq_limit, batch, row_tiles, kv_heads, lead, grid;
};

PagedWork work_of(const Batch &p)
{
    PagedWork w{0, 0};
    for (int b = 0; b < p.batch; ++b) {
        const int n = paged_slots(p, b, p.row_tiles * p.kv_heads);
        w.slots += n;
        w.units += n > 0 ? p.row_tiles * p.kv_heads : 0;
    }
    return w;
}

// Slot x as paged_find has it: the requests in shares, one a thread, and the share that holds the slot looks for it.
PagedAt place(const Batch &p, int threads, int x)
{
    PagedAt at{p.batch, 0, 0};
    const int each = (p.batch + threads - 1) / threads;
    int from = 0;
    for (int t = 0; t < threads; ++t) {
        const int b0 = p.batch < t * each ? p.batch : t * each, b1 = p.batch < b0 + each ? p.batch : b0 + each;
        int mine = 0;
        for (int b = b0; b < b1; ++b)
            mine += paged_slots(p, b, p.row_tiles * p.kv_heads);
        if (x >= from && x < from + mine)
            at = paged_at(p, b0, b1, from, x);
        from += mine;
    }
    return at;
}
}  // namespace

// Rows of 7: CTA, part, request, unit, first page, pages, tokens of the request.  Returns their number, -1 where there are more.
extern "C" int taken(const int32_t *lens, int limit, int batch, int row_tiles, int kv_heads, int lead, int grid, int threads,
                     int32_t *out, int most)
{
    const Batch p{lens, limit, batch, row_tiles, kv_heads, lead, grid};
    const PagedSplit split(work_of(p), p);
    int n = 0;
    for (int cta = 0; cta < split.ctas; ++cta) {
        int seg = 0;
        PagedWalk walk(p, place(p, threads, split.start(cta)), split.start(cta + 1) - split.start(cta));
        for (; walk.left > 0; walk.next(p), ++seg) {
            if (n == most)
                return -1;
            const int32_t row[7] = {cta, paged_part(cta, seg), walk.b, walk.u, walk.j, walk.run(), walk.len};
            for (int i = 0; i < 7; ++i)
                out[n * 7 + i] = row[i];
            ++n;
        }
    }
    return n;
}

// The parts of a unit as a block of the join that takes units finds them: their number (0: no work) and their places.
extern "C" int parts_of_unit(const int32_t *lens, int limit, int batch, int row_tiles, int kv_heads, int lead, int grid, int b, int u,
                             int32_t *out, int most)
{
    const Batch p{lens, limit, batch, row_tiles, kv_heads, lead, grid};
    const PagedSplit split(work_of(p), p);
    const int pages = pages_of(paged_len(p, b));
    int before = 0;
    for (int i = 0; i < b; ++i)
        before += paged_slots(p, i, row_tiles * kv_heads);
    const PagedParts where(split, before + u * (pages + lead) + lead, pages, lead);
    for (int i = 0; i < where.n && i < most; ++i)
        out[i] = where.part(i);
    return where.n;
}

// The same as block x of the join that takes ranges' ends finds them; its request and unit in out[0], out[1].
extern "C" int parts_at_end(const int32_t *lens, int limit, int batch, int row_tiles, int kv_heads, int lead, int grid, int threads,
                            int x, int32_t *out, int most)
{
    const Batch p{lens, limit, batch, row_tiles, kv_heads, lead, grid};
    const PagedSplit split(work_of(p), p);
    if (x + 1 >= split.ctas)
        return 0;
    const PagedAt at = place(p, threads, split.start(x + 1));
    const int pages = at.b < batch ? pages_of(paged_len(p, at.b)) : 0;
    const PagedParts where(split, split.start(x + 1) - at.j, pages, lead);
    if (where.n < 2 || at.j <= 0 || where.first != x)
        return 0;
    out[0] = at.b;
    out[1] = at.u;
    for (int i = 0; i < where.n && i + 2 < most; ++i)
        out[i + 2] = where.part(i);
    return where.n;
}

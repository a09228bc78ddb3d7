// How attention over all pages cuts a batch into equal ranges, one a CTA, and where the parts of a cut unit lie: the
// arithmetic of paged_attn.cuh's kernels, in functions that run on the host as well.  P is their parameters, or a struct with
// the same names for the batch: seq_lens, seq_limit, batch, row_tiles, kv_heads, lead, grid.
#pragma once

#include <cstdint>

#include "layout.cuh"

namespace msa {

template <class P>
__host__ __device__ __forceinline__ int paged_len(const P &p, int b)
{
    const int n = p.seq_lens[b];
    return n < 0 || n > p.seq_limit ? 0 : n;
}

// The batch's work: slots of all units, and units that have some.  A unit of n pages has `lead` slots, in which there is
// nothing to do and which stand for its start and its end, and then a slot a page.
struct PagedWork {
    int slots, units;
};

// The slots of request b's units.
template <class P>
__host__ __device__ __forceinline__ int paged_slots(const P &p, int b, int units)
{
    const int n = pages_of(paged_len(p, b));
    return n > 0 ? (n + p.lead) * units : 0;
}

// The ranges: CTA g has [start(g), start(g + 1)) of the units' slots, two pages at least, but no fewer ranges than units (at
// least 1, 2, 4 pages: one request of 300 tokens, 4 heads, 8.9, 9.4, 8.1 us; 2000: 9.6, 9.8, 11.1; 8700: 10.7, 10.5, 11.8).
struct PagedSplit {
    int ctas, range, more;
    template <class P>
    __host__ __device__ PagedSplit(const PagedWork &work, const P &p)
    {
        const int pairs = (work.slots - work.units * p.lead + 1) / 2, most = pairs > work.units ? pairs : work.units;
        ctas = p.grid < most ? p.grid : most;
        range = ctas > 0 ? work.slots / ctas : 0;
        more = work.slots - range * ctas;
    }
    __host__ __device__ int start(int g) const { return g * range + (g < more ? g : more); }
    // the CTA whose range holds slot x
    __host__ __device__ int owner(int x) const
    {
        const int longer = more * (range + 1);
        return x < longer ? x / (range + 1) : more + (x - longer) / range;
    }
};

// A place in the sequence of the units' slots.
struct PagedAt {
    int b, u, j;  // request, its unit, the unit's page (negative: its lead)
};

// Slot x, which is one of requests [b0, b1), whose first slot is `from`.
template <class P>
__host__ __device__ __forceinline__ PagedAt paged_at(const P &p, int b0, int b1, int from, int x)
{
    const int units = p.row_tiles * p.kv_heads;
    for (int b = b0; b < b1; ++b) {
        const int n = paged_slots(p, b, units);
        if (x < from + n) {
            const int each = pages_of(paged_len(p, b)) + p.lead, u = (x - from) / each;
            return PagedAt{b, u, x - from - u * each - p.lead};
        }
        from += n;
    }
    return PagedAt{p.batch, 0, 0};
}

// Runs through a range unit by unit.
struct PagedWalk {
    int b, u, j, left;  // the next page, and slots left from there on
    int len, P;         // of request b
    template <class Params>
    __host__ __device__ PagedWalk(const Params &p, const PagedAt &at, int n) : b(at.b), u(at.u), j(at.j), left(n), len(0), P(0)
    {
        left += j < 0 ? j : 0;
        j = j > 0 ? j : 0;
        if (left > 0) {
            len = paged_len(p, b);
            P = pages_of(len);
        }
    }
    __host__ __device__ int run() const { return left < P - j ? left : P - j; }
    template <class Params>
    __host__ __device__ void next(const Params &p)
    {
        left -= run() + p.lead;
        j = 0;
        if (++u == p.row_tiles * p.kv_heads && left > 0) {
            u = 0;
            do {
                if (++b >= p.batch) {  // not while the lengths stay as they are
                    left = 0;
                    return;
                }
                len = paged_len(p, b);
                P = pages_of(len);
            } while (P == 0);
        }
    }
};

// Which of a CTA's two parts its run of number `seg` writes, if the run is no whole unit: only its first and its last are cut.
__host__ __device__ __forceinline__ int paged_part(int cta, int seg) { return 2 * cta + (seg > 0); }

// The parts of a unit whose pages have the slots from `from` on; none of a unit without pages.
struct PagedParts {
    int first, n;  // the CTA that has the first page; CTAs that have some
    int part0;     // where the first part is: that CTA's first run, but where it has others before the unit
    __host__ __device__ PagedParts(const PagedSplit &split, int from, int pages, int lead)
    {
        first = pages > 0 ? split.owner(from) : 0;
        n = pages > 0 ? split.owner(from + pages - 1) - first + 1 : 0;
        part0 = paged_part(first, split.start(first) < from - lead);
    }
    __host__ __device__ int part(int i) const { return i == 0 ? part0 : paged_part(first + i, 0); }
};

}  // namespace msa

// Whether two tensors of strided rows share memory.
#pragma once

#include <algorithm>
#include <cstdint>
#include <numeric>

namespace msa {

// `n` rows of `width` bytes, `stride` >= width bytes from one to the next.
struct RowSpan {
    int64_t at, stride, width, n;
    RowSpan(const void *base, int64_t stride_, int64_t width_, int64_t n_)
        : at(static_cast<int64_t>(reinterpret_cast<uintptr_t>(base))), stride(stride_), width(width_), n(n_)
    {
        if (stride == width) {  // one piece
            width *= n;
            n = std::min<int64_t>(n, 1);
            stride = width;
        }
    }
    int64_t end() const { return at + (n - 1) * stride + width; }
    // a row that shares a byte with [from, to)
    bool meets(int64_t from, int64_t to) const
    {
        if (n == 0 || to <= at || from >= end())
            return false;
        // the first row that ends behind `from`
        const int64_t j = from < at + width ? 0 : n == 1 ? 1 : (from - at - width) / stride + 1;
        return j < n && at + j * stride < to;
    }
};

inline bool rows_overlap(const RowSpan &a, const RowSpan &b)
{
    if (a.n == 0 || b.n == 0 || a.end() <= b.at || b.end() <= a.at)
        return false;
    if (a.n == 1)
        return b.meets(a.at, a.end());
    // a's rows between b's ends.  One that crosses an end shares a byte, and is the first or the last of them; whether one
    // inside does goes by its distance from b's rows, which comes again after stride / gcd of the strides.
    const int64_t first = a.at + a.width > b.at ? 0 : (b.at - a.at - a.width) / a.stride + 1;
    const int64_t last = std::min(a.n - 1, (b.end() - 1 - a.at) / a.stride);
    const int64_t again = b.n == 1 ? 1 : b.stride / std::gcd(a.stride, b.stride);
    auto meets = [&](int64_t i) { return b.meets(a.at + i * a.stride, a.at + i * a.stride + a.width); };
    for (int64_t i = first; i <= last && i < first + again; ++i)
        if (meets(i))
            return true;
    return first <= last && meets(last);
}

}  // namespace msa

// Rows of logits read in 16-byte vectors, shared by the kernels that sum over a vocabulary.
#pragma once

#include <cmath>
#include <cstdint>

namespace msa {

// Logits in 16-byte vectors; NaN counts as -inf.
template <class T>
struct Logits;
template <>
struct Logits<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float one(const float *p) { return fmaxf(*p, -INFINITY); }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&x)[4])
    {
        x[0] = fmaxf(__uint_as_float(v.x), -INFINITY);
        x[1] = fmaxf(__uint_as_float(v.y), -INFINITY);
        x[2] = fmaxf(__uint_as_float(v.z), -INFINITY);
        x[3] = fmaxf(__uint_as_float(v.w), -INFINITY);
    }
};
template <>
struct Logits<uint16_t> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float one(const uint16_t *p)
    {
        return fmaxf(__uint_as_float(static_cast<uint32_t>(*p) << 16), -INFINITY);
    }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&x)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = fmaxf(__uint_as_float(w[i] << 16), -INFINITY);
            x[2 * i + 1] = fmaxf(__uint_as_float(w[i] & 0xffff0000u), -INFINITY);
        }
    }
};

// Vector v of a row (elements [v * N, v * N + N)) wherever the row starts, so that a
// row's sums are grouped by index alone, not by address: one 16-byte load where
// every row is aligned to it, else word by word (five words that hold the eight
// 2-byte elements, shifted into place when they are used; the outer two each hold a
// byte of the vector).
template <class T, bool ALIGNED>
struct RawVec {
    uint32_t w[ALIGNED || sizeof(T) == 4 ? 4 : 5];
    __device__ __forceinline__ void load(const T *row, int v)
    {
        const uint8_t *at = reinterpret_cast<const uint8_t *>(row) + static_cast<int64_t>(v) * 16;
        if (ALIGNED) {
            const uint4 x = *reinterpret_cast<const uint4 *>(at);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
            const uint32_t odd = sizeof(T) == 4 ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 2);
            const uint32_t *word = reinterpret_cast<const uint32_t *>(at - odd);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = word[i];
            if (sizeof(T) != 4)
                w[sizeof(w) / 4 - 1] = odd ? word[4] : 0u;
        }
    }
    __device__ __forceinline__ uint4 get(const T *row) const
    {
        if (ALIGNED || sizeof(T) == 4)
            return make_uint4(w[0], w[1], w[2], w[3]);
        const uint32_t bits = (reinterpret_cast<uintptr_t>(row) & 2) * 8;
        return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                          __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[sizeof(w) / 4 - 1], bits));
    }
};

constexpr int kBatch = 4;  // vectors a thread loads at a time

// A batch of a thread's share of a row: vectors v0 + u * ranks.
template <class T, bool ALIGNED>
__device__ __forceinline__ void load_batch(RawVec<T, ALIGNED> (&q)[kBatch], const T *row, int nv, int v0, int ranks)
{
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
        const int v = v0 + u * ranks;
        if (v < nv)
            q[u].load(row, v);
    }
}

}  // namespace msa

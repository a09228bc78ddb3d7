// What the attention kernels share: bounded waits of a warp, the softmax's rescaling,
// query rows brought into a narrow type's range.
#pragma once

#include <cmath>

#include "attn_ptx.cuh"
#include "layout.cuh"

#include "msa_attention.h"

namespace msa {

__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "  selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// Bounded wait of a whole warp; false, with the CTA's abort flag and the fault
// bit set, when it ran out or another warp gave up before.  A phase that is
// complete already, the common case in a page loop that the cache stream does not
// hold up, costs one test.  `withhold`: the test of the bounded waits, with far
// fewer polls.
constexpr uint32_t kWithheldPolls = 1u << 14;

__device__ __forceinline__ bool attn_wait(int *abort_flag, uint32_t *fault, uint32_t bar, uint32_t parity, int withhold)
{
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity)))
        return true;
    bool ok = false;
    if (!*reinterpret_cast<volatile int *>(abort_flag)) {
        const uint32_t polls = withhold ? kWithheldPolls : kSpinLimit;
        for (uint32_t i = 0; i < polls && !ok; ++i)
            ok = mbar_try_wait(bar, parity);
        if (!ok) {
            atomicOr(fault, MSA_FAULT_TIMEOUT);
            *reinterpret_cast<volatile int *>(abort_flag) = 1;
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// The factor 2^(a - b) that moves a part from maximum a to b >= a; 1 for an empty part (-inf both).
__device__ __forceinline__ float rescale(float a, float b) { return a == b ? 1.0f : exp2_approx(a - b); }

// A query row as f16: the power of two that puts its largest |q| in [2^13, 2^14)
// (exact for values within 2^-14 .. 2^14 of it), undone through *undo.
__device__ __forceinline__ float q_row_factor(float amax, float *undo)
{
    int e = 0;
    if (amax > 0.0f && amax < INFINITY) {
        frexpf(amax, &e);  // amax in [2^(e-1), 2^e)
        e = 14 - e;
        e = max(-100, min(100, e));
    }
    *undo = ldexpf(1.0f, -e);
    return ldexpf(1.0f, e);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

}  // namespace msa

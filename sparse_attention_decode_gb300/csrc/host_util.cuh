// Host-side helpers shared by the indexer's translation units: launch
// configuration with programmatic dependent launch, the driver's tensor-map
// encoder, and per-device attribute caches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "layout.cuh"

namespace msa {

// Launch configuration with programmatic dependent launch: the grid may be
// scheduled while the previous kernel on the stream is still running; it
// calls griddep_wait() before touching global memory, so it observes all of
// that kernel's writes (and the previous kernel cannot see any of its own).
static cudaLaunchConfig_t pdl_config(dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                     cudaLaunchAttribute (&attr)[1])
{
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_tiled()
{
    static EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// Encodes a tensor map (the arguments of cuTensorMapEncodeTiled).  The encoder
// wants a context that is current on the calling thread, and a thread whose first
// CUDA call this is has none yet: the runtime's is bound then and the map encoded.
template <class... Args>
static bool encode_map(Args... args)
{
    EncodeTiledFn enc = encode_tiled();
    if (!enc)
        return false;
    CUresult r = enc(args...);
    int dev = 0;
    if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess)
        r = enc(args...);
    return r == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

static int device_sms(int dev)
{
    static std::atomic<int> cache[kMaxDevices];
    int v = (dev >= 0 && dev < kMaxDevices) ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (v > 0)
        return v;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
        return 0;
    if (dev >= 0 && dev < kMaxDevices)
        cache[dev].store(v, std::memory_order_relaxed);
    return v;
}

// Lets `kernel` be launched with up to `most` bytes of dynamic shared memory on
// device `dev`, once (`done`: the kernel's own flags).  The setting belongs to the
// process: `most` is what the largest call asks for, whatever the call at hand
// does, so that no thread's launch meets a smaller one set by another.
template <class Kernel>
static bool allow_smem(Kernel *kernel, size_t most, int dev, std::atomic<bool> (&done)[kMaxDevices])
{
    const bool known = dev >= 0 && dev < kMaxDevices;
    if (known && done[dev].load(std::memory_order_acquire))
        return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most)) != cudaSuccess)
        return false;
    if (known)
        done[dev].store(true, std::memory_order_release);
    return true;
}

// L2 size of device `dev` in bytes (0 when the query fails).
static int64_t device_l2_bytes(int dev)
{
    static std::atomic<int> cache[kMaxDevices];
    int v = (dev >= 0 && dev < kMaxDevices) ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (v > 0)
        return v;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrL2CacheSize, dev) != cudaSuccess || v <= 0)
        return 0;
    if (dev >= 0 && dev < kMaxDevices)
        cache[dev].store(v, std::memory_order_relaxed);
    return v;
}

static int64_t blocks_for(int max_model_len) { return (static_cast<int64_t>(max_model_len) + kPage - 1) / kPage; }

}  // namespace msa

// launch.cuh -- kernel launch with programmatic dependent launch, and the
// argument checks shared by the C entries of the 8-bit cache and the prompt
// attention.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace treeattn {

template <typename Kernel, typename... Args>
inline cudaError_t launch_dependent(Kernel kernel, dim3 grid, dim3 block, size_t smem,
                                    cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// SMs of a device (asked for once), 0 if it cannot be told.
inline int sms_of(int dev) {
    static std::atomic<int> known[64];
    if (dev < 0) return 0;
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Lets a kernel have all of an SM's shared memory, and clusters of 16 CTAs where
// `wide` (asked for once per device; `configured` has a bit for each).
inline bool opt_in(const void* kernel, int dev, std::atomic<unsigned long long>& configured,
                   bool wide = false) {
    const unsigned long long bit = 1ull << (dev & 63);
    if ((configured.load(std::memory_order_relaxed) & bit) != 0) return true;
    int most = 0;
    cudaFuncAttributes fixed;
    if (cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
            cudaSuccess ||
        cudaFuncGetAttributes(&fixed, kernel) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             most - static_cast<int>(fixed.sharedSizeBytes)) != cudaSuccess)
        return false;
    if (wide && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                    cudaSuccess)
        return false;
    configured.fetch_or(bit);
    return true;
}

inline bool ptr_aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline bool page_size_ok(int P) { return P == 16 || P == 32 || P == 64 || P == 128; }

}  // namespace treeattn

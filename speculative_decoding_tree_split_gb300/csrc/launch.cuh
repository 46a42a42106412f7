// launch.cuh -- kernel launch with programmatic dependent launch, and the
// argument checks shared by the C entries of the 8-bit cache and the prompt
// attention.
#pragma once

#include <cuda_runtime.h>

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

inline bool ptr_aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline bool page_size_ok(int P) { return P == 16 || P == 32 || P == 64 || P == 128; }

}  // namespace treeattn

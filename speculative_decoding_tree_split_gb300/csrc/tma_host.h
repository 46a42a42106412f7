// tma_host.h -- tensor maps for TMA loads, encoded on the host.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

namespace treeattn {

using TiledEncoder = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline TiledEncoder tiled_encoder() {
    static TiledEncoder fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<TiledEncoder>(p);
    });
    return fn;
}

// A map of `rank` dimensions (innermost first; strides in bytes, without the
// innermost), boxes of box[], the given type and swizzle, zero fill outside.
inline bool encode_tiled(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base,
                         const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                         CUtensorMapSwizzle swizzle) {
    const TiledEncoder fn = tiled_encoder();
    if (fn == nullptr) return false;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return fn(map, type, rank, const_cast<void*>(base), dims, strides, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace treeattn

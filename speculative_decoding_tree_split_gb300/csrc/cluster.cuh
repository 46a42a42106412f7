// cluster.cuh -- thread-block clusters: launch, barrier, and another CTA's
// shared memory.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace treeattn {

// launch_dependent with `size` CTAs (along x) to a cluster.
template <typename Kernel, typename... Args>
inline cudaError_t launch_cluster(Kernel kernel, dim3 grid, dim3 block, size_t smem, int size,
                                  cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(size);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

namespace ptx {

// All threads of all CTAs of the cluster; orders their memory accesses.
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\t"
        "barrier.cluster.wait.acquire.aligned;" ::
            : "memory");
}

// The same in two halves, as far as all having begun is concerned: no memory is ordered
// by the first.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// Address in CTA `rank`'s shared memory of what lies at `addr` in one's own.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// The same for a pointer to shared memory, for plain loads and stores.
template <typename T>
__device__ __forceinline__ T* map_generic(T* p, uint32_t rank) {
    uint64_t r;
    asm("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<T*>(r);
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

}  // namespace ptx

// The sequence that is `rank`-th by length, longest first (equal ones in order): units
// that begin late should end soon.  For n <= blockDim.x sequences, by all threads;
// `scratch` holds n + 1 ints and is free again afterwards.
__device__ __forceinline__ int by_length(const int32_t* lens, int n, int rank, int* scratch) {
    const int tid = static_cast<int>(threadIdx.x);
    const int mine = tid < n ? lens[tid] : 0;
    if (tid < n) scratch[tid] = mine;
    __syncthreads();
    if (tid < n) {
        int before = 0;
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const int other = scratch[i];
            before += other > mine || (other == mine && i < tid);
        }
        if (before == rank) scratch[n] = tid;
    }
    __syncthreads();
    const int found = scratch[n];
    __syncthreads();
    return found;
}

}  // namespace treeattn

// Launches with attributes: kernels that may come up under the tail of the one before them (and wait
// for its results by griddepcontrol.wait), and kernels of clusters.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/ft_moe.h"
#include "ft_internal.h"

namespace ft {

__device__ __forceinline__ void wait_for_prior_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A word of shared memory of the cluster's CTA `rank`, at the place that p has in this one.
__device__ __forceinline__ float cluster_load(const void* p, uint32_t rank) {
    uint32_t at;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ float4 cluster_load4(const void* p, uint32_t rank) {      // p at a 16-byte word
    uint32_t at;
    float4 v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}

// cluster: CTAs per cluster along grid.x (1: none).
template <typename... P, typename... A>
int launch_with(void (*kernel)(P...), const char* name, dim3 grid, dim3 block, size_t smem, bool overlap, unsigned cluster,
                cudaStream_t s, A... args) {
    if (smem > 40 * 1024)      // 48 KB, with room for what a kernel has of fixed size
        if (int st = set_smem_limit(reinterpret_cast<const void*>(kernel), static_cast<int>(smem))) return st;
    cudaLaunchAttribute at[2];
    unsigned n = 0;
    if (overlap) {
        at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = cluster;
        at[n].val.clusterDim.y = 1;
        at[n++].val.clusterDim.z = 1;
    }
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = n;
    const cudaError_t e = cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(FT_ERR_LAUNCH, "launch of %s failed: %s", name, cudaGetErrorString(e));
    }
    return check_launch(name, grid, block, smem);
}

}  // namespace ft

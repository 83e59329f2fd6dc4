// Launches with attributes: kernels that may come up under the tail of the one before them (and wait
// for its results by griddepcontrol.wait), and kernels of clusters.
#pragma once

#include <cuda_runtime.h>

#include "../../include/ft_moe.h"
#include "ft_internal.h"

namespace ft {

__device__ __forceinline__ void wait_for_prior_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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

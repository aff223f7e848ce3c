// Launches that overlap the end of the kernel before them on the stream: the grid is set up while that
// kernel still runs, and waits for all of it (and its writes) before it touches memory.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace scope {

// The grid after this one may be set up.  Any thread may call it, at any time.
__device__ __forceinline__ void early_next()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Waits for the grid before this one; every thread of an early launch, before its first access.
__device__ __forceinline__ void early_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// cluster: blocks of a cluster (along x).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, unsigned cluster,
                         A &&...args)
{
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = attr;
    c.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&c, kernel, std::forward<A>(args)...);
}

}  // namespace scope

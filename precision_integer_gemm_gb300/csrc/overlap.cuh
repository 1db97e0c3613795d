// Launches that may be set up while the kernel before them in the stream ends.
#pragma once
#include <cuda_runtime.h>
#include "launch.cuh"

namespace igemm {

// First in a kernel launched by launch_overlapped: the kernel after it may be set
// up on SMs that this one has left, and nothing is read or written before the
// kernel before it has ended.
__device__ __forceinline__ void overlap_begin()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ... in clusters of `cluster` CTAs.
template <class... Params, class... Args>
int launch_overlapped_clusters(void (*kernel)(Params...), dim3 grid, int cluster, dim3 block, int smem,
                               cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) != cudaSuccess) return kCudaError;
    note_launch();
    return kOk;
}

template <class... Params, class... Args>
int launch_overlapped(void (*kernel)(Params...), dim3 grid, dim3 block, int smem, cudaStream_t stream, Args... args)
{
    return launch_overlapped_clusters(kernel, grid, 1, block, smem, stream, args...);
}

}  // namespace igemm

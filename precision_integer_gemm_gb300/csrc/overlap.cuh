// Launches that may be set up while the kernel before them in the stream ends.
#pragma once
#include <cuda_runtime.h>
#include "launch.cuh"

namespace igemm {

// First in a kernel launched by launch_overlapped: the kernel after it may be set
// up on SMs that this one has left, and nothing is read or written before the
// kernel before it has ended.  For kernels that leave most of the GPU free.
__device__ __forceinline__ void overlap_begin()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The two halves apart: a kernel that fills the SMs lets the next one in only towards
// its end, so that the next one's blocks spread over all SMs instead of settling where
// there happens to be room (back to back, us, from the start against at the end:
// routing of 8192 x 64 bfloat16 12.1 to 6.6, packing of 128 x 4096 float32 2.5 to 1.8,
// combining 256 x 8 rows of 4096 6.0 to 4.0).
__device__ __forceinline__ void overlap_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void overlap_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// What such a kernel reads may be written until the wait returns, and the kernel's
// life begins before that.  So it reads global memory with plain loads, or with the
// volatile ones of ptx.cuh, and its pointers are not restrict: a read-only (.nc) load
// promises memory that nobody writes during the kernel's life, and the compiler may
// move one above the wait.

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

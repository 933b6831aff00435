// dependent.cuh -- chains of small kernels: each is launched as a
// programmatic dependent of the one before it on the stream, so that its
// blocks are placed and set up while that one still runs, and waits on the
// device before it touches memory.
#pragma once

#include <cuda_runtime.h>

#include "../../include/sgemm.h"
#include "internal.h"

namespace sg {

// Every thread, before its first access to global memory: the kernels before
// this one have completed and their writes are visible.  (Every thread, also
// of blocks without work: a kernel that completed without waiting would let
// the one after it overtake the one before.)  What the kernels before write is
// read by ordinary loads: no __ldg, no const pointer declared __restrict__.
__device__ __forceinline__ void dependent_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
// The next kernel on the stream may be placed from here on, as far as this
// thread is concerned; it still waits for this one to complete.
__device__ __forceinline__ void dependent_release()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launches `kern` (which calls dependent_wait) as above, in clusters of
// `cluster` CTAs; counts the launch.
template <class... P, class... A>
int launch_dependent(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, unsigned cluster,
                     cudaStream_t st, const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    note_launch();
    return SGEMM_OK;
}

// What a C entry point returns: f()'s status; nothing that the host side may
// throw (allocation, locks) leaves it.
template <class F>
int c_entry(const F &f) noexcept
{
    try {
        return f();
    } catch (...) {
        return SGEMM_ERR_LAUNCH;
    }
}

}  // namespace sg

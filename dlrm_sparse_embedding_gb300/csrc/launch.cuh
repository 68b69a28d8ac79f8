// Launches that may begin while the stream's previous kernel ends (programmatic
// dependent launch): a block sets itself up, then waits for the earlier kernel's
// memory before it touches any.
#pragma once

#include <cuda_runtime.h>

#include "emb.h"

namespace emb {

// Every thread of every kernel launched with launch_next calls this before its
// first access to global memory: returns once all earlier work of the stream is
// done and visible.  (Where the kernel before lets the next one begin only after its own
// wait, what stood before that kernel may be read before this one's.)
__device__ __forceinline__ void wait_for_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The stream's next kernel may begin to set itself up.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... P, class... A>
int launch_next(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, unsigned cluster, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {cluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return EMB_ERR_CUDA;
    }
    return EMB_OK;
}

}  // namespace emb

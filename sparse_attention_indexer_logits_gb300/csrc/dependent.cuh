// Launches that may begin while the kernel before them in the stream ends:
// such a kernel calls grid_dependency_wait before it touches memory, and
// allow_dependent_launch when the next one's CTAs may come.
#pragma once

#include <cuda_runtime.h>

#include "ptx.cuh"

namespace pml {

template <class K, class... Args>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pml

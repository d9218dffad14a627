// One head dimension of the attention over caches held in 4 bits (a translation
// unit each, compiled side by side).
#pragma once

#include "nvfp4_attention.cuh"

namespace pml {

template <int D, bool FP16, bool SEL, int NT>
cudaError_t launch_nvfp4_one(const NvAttnArgs& a, const nvattn::Pieces& wp, const nvattn::Pieces& cp, int num_ctas,
                             cudaStream_t stream)
{
    using C = nvattn::Cfg<D, NT>;
    auto kernel = nvattn::nvfp4_attention_kernel<D, FP16, SEL, NT>;
    static int configured_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (configured_device != dev) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kTotal);
        if (e != cudaSuccess) return e;
        configured_device = dev;
    }
    return launch_dependent(kernel, dim3((unsigned)num_ctas), C::kThreads, C::kTotal, stream, a, wp, cp);
}

template <int D, bool FP16>
cudaError_t launch_nvfp4_type(int tiles, const NvAttnArgs& a, const nvattn::Pieces& wp, const nvattn::Pieces& cp,
                              int num_ctas, cudaStream_t stream)
{
    if (a.selected)
        return tiles == 1 ? launch_nvfp4_one<D, FP16, true, 1>(a, wp, cp, num_ctas, stream)
                          : launch_nvfp4_one<D, FP16, true, 2>(a, wp, cp, num_ctas, stream);
    return tiles == 1 ? launch_nvfp4_one<D, FP16, false, 1>(a, wp, cp, num_ctas, stream)
                      : launch_nvfp4_one<D, FP16, false, 2>(a, wp, cp, num_ctas, stream);
}

template <int D>
cudaError_t launch_nvfp4_attention_dim(bool fp16, int tiles, const NvAttnArgs& a, const nvattn::Pieces& wp,
                                       const nvattn::Pieces& cp, int num_ctas, cudaStream_t stream)
{
    return fp16 ? launch_nvfp4_type<D, true>(tiles, a, wp, cp, num_ctas, stream)
                : launch_nvfp4_type<D, false>(tiles, a, wp, cp, num_ctas, stream);
}

}  // namespace pml

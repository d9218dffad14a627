// One head dimension of the attention over caches held in 4 bits (a translation
// unit each, compiled side by side).
#pragma once

#include "cluster_counts.h"
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
    if (a.cluster > 1)
        return launch_dependent_clusters(kernel, dim3((unsigned)num_ctas), a.cluster, C::kThreads, C::kTotal, stream, a,
                                         wp, cp);
    return launch_dependent(kernel, dim3((unsigned)num_ctas), C::kThreads, C::kTotal, stream, a, wp, cp);
}

// Clusters of `size` CTAs that the device runs at a time, 0 if it cannot say.
template <int D, bool SEL, int NT>
int nvfp4_clusters(int size)
{
    using C = nvattn::Cfg<D, NT>;
    static ClusterCounts counts;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    return counts.get(dev, size, [](int s) {
        auto kernel = nvattn::nvfp4_attention_kernel<D, true, SEL, NT>;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)s);
        cfg.blockDim = dim3((unsigned)C::kThreads);
        cfg.dynamicSmemBytes = C::kTotal;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {(unsigned)s, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kTotal) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess)
            return n;
        cudaGetLastError();
        return 0;
    });
}

template <int D>
int nvfp4_clusters_dim(bool select, int tiles, int size)
{
    if (select) return tiles == 1 ? nvfp4_clusters<D, true, 1>(size) : nvfp4_clusters<D, true, 2>(size);
    return tiles == 1 ? nvfp4_clusters<D, false, 1>(size) : nvfp4_clusters<D, false, 2>(size);
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

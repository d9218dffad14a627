// Attention over caches held in 4 bits, heads of 128.
#include "nvfp4_attention_dim.cuh"

namespace pml {

template cudaError_t launch_nvfp4_attention_dim<128>(bool, int, const NvAttnArgs&, const nvattn::Pieces&,
                                                    const nvattn::Pieces&, int, cudaStream_t);
template int nvfp4_clusters_dim<128>(bool, int, int);

}  // namespace pml

// Attention over pages held in 4 bits by tiles, head dimension 64.
#include "paged_attention.cuh"

namespace pml {

cudaError_t launch_attention_nvfp4_d64(bool fp16, bool select, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                       const CUtensorMap& vmap, const AttnArgs& a, int num_ctas, cudaStream_t stream)
{
    if (fp16)
        return select ? attn::launch_kernel<64, true, true, true>(qmap, kmap, vmap, a, num_ctas, stream)
                      : attn::launch_kernel<64, true, false, true>(qmap, kmap, vmap, a, num_ctas, stream);
    return select ? attn::launch_kernel<64, true, true, true, false>(qmap, kmap, vmap, a, num_ctas, stream)
                  : attn::launch_kernel<64, true, false, true, false>(qmap, kmap, vmap, a, num_ctas, stream);
}

}  // namespace pml

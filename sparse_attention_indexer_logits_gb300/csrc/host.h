// Host-side helpers shared by the C ABI's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pml {

struct DeviceInfo {
    int device, sm_count, smem_optin;
    unsigned int* status;
};

// Properties of the current device and its status word's address, looked up
// once per device with that device current.
cudaError_t device_info(DeviceInfo& d);

// Records a CUDA error for pml_last_cuda_error and returns PML_ERR_CUDA.
int cuda_fail(cudaError_t e);

inline bool aligned(const void* p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Tiled map: dims/strides innermost first, strides in bytes for dimensions 1.. .
cudaError_t encode_tiled(CUtensorMap& map, CUtensorMapDataType dtype, int rank, const void* base,
                         const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                         CUtensorMapSwizzle swizzle);

}  // namespace pml

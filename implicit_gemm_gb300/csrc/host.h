// Host helpers shared by the library's translation units (defined in wgrad.cu,
// the status words of other units in those).  Internal: nothing here is exported.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <string>

namespace wg {

// Record the reason of a non-zero return (wg_last_error) and return the status.
int set_err(int status, const std::string& msg);
int cuda_fail(const char* what, cudaError_t e);

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled from the driver (null when it is not there).
EncodeTiledFn encode_fn();

// Raise a kernel's dynamic shared-memory limit when a launch needs more than
// any earlier one (per device).
int ensure_smem_ptr(const void* kernel, int bytes);
template <typename K>
int ensure_smem(K kernel, int bytes)
{
    return ensure_smem_ptr(reinterpret_cast<const void*>(kernel), bytes);
}

// SM count of the current device (a default when no device is visible).
int num_sms();

bool aligned16(const void* ptr);

// Programmatic stream serialization for a launch.
void pdl_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, unsigned* na, cudaStream_t stream);

// The device status words of update.cu and layer.cu.
cudaError_t read_update_status(unsigned int* v);
cudaError_t write_update_status(unsigned int v);
cudaError_t read_layer_status(unsigned int* v);
cudaError_t write_layer_status(unsigned int v);

}  // namespace wg

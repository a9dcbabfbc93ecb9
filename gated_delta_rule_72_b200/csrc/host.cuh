// host.cuh -- host-side helpers shared by the library's translation units
// (defined in gdn_api.cu).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace gdn {

// The driver's tensor-map encoder, or NULL.
PFN_cuTensorMapEncodeTiled_v12000 driver_tensor_map_encoder();
// Device word counting bounded waits that gave up on the current device, or NULL.
unsigned int *wait_timeout_counter();
// SMs of the current device.
int device_sm_count();

}  // namespace gdn

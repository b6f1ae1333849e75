// mx_host.hpp -- host helpers shared by the library's translation units
// (defined in mxgemm.hip).
#pragma once

#include <hip/hip_runtime.h>

namespace mxg {

// MXG_OK if the current device is gfx950, else MXG_ERR_DEVICE or MXG_ERR_HIP
// (looked up once per device).
__attribute__((visibility("hidden"))) int host_check_device();

// Keep a HIP error for mx_last_hip_error: MXG_OK for hipSuccess, else MXG_ERR_HIP.
__attribute__((visibility("hidden"))) int host_hip_status(hipError_t e);

}  // namespace mxg

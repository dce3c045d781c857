// Error reporting and device queries shared by the host sides of the C ABI
// (defined in moe_api.hip).
#pragma once

#include "moe.h"

#include <hip/hip_runtime.h>

namespace moe {

// Clears the calling thread's error text; every entry point starts with it.
void clear_error();
// Record the error text and return the status.
moe_status fail(moe_status st, const char* what);
moe_status hip_fail(hipError_t err, const char* where);
// Compute units of the current device (cached per device).
int device_cus();

}  // namespace moe

// Status and error-detail helpers of the C ABI's host files (defined in
// abi.cpp).  Plain C++.
#pragma once
#include <stddef.h>

#include "moe_qexpert.h"

namespace moe {

// Writes the calling thread's error detail and returns `s`.
moe_status fail(moe_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the detail; MOE_OK.
moe_status ok();
// MOE_OK for 0, else MOE_ERR_HIP with what failed.
moe_status hip_status(int e, const char* what);
bool aligned(const void* p, size_t a);
// gfx950 check, once per device and thread, on the first launching call;
// then any error left pending by the caller's earlier HIP calls is dropped.
moe_status check_device();

}  // namespace moe

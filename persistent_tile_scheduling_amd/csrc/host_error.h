// The error message behind gemm_last_error(), shared by the library's host
// files: one message per thread, set by the call that failed.
#pragma once

#include <hip/hip_runtime.h>

#include "pts_gemm.h"

namespace pts {

// Keep the message and return the status.
gemm_status fail(gemm_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3), visibility("hidden")));
gemm_status hip_fail(hipError_t e, const char *what) __attribute__((visibility("hidden")));

} // namespace pts

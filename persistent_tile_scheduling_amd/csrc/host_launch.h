// Launches of the library's host files.
#pragma once

#include <hip/hip_runtime.h>

#include <utility>

#include "host_error.h"

namespace pts {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void *p, size_t to) { return ((uintptr_t)p % to) == 0; }

// HIP limits a grid to 2^32 - 1 threads.
template <class... Args>
gemm_status launch_grid(void (*kernel)(Args...), int64_t x, int64_t y, int threads, void *stream, std::remove_const_t<Args> &...args)
{
    if (x * y * threads > (int64_t)UINT32_MAX || y > 65535)
        return fail(GEMM_ERR_UNSUPPORTED, "%lld x %lld workgroups: too large a problem for one launch", (long long)x, (long long)y);
    void *kargs[] = {&args...};
    const hipError_t e = hipLaunchKernel((const void *)kernel, dim3((uint32_t)x, (uint32_t)y), dim3(threads), kargs, 0, (hipStream_t)stream);
    return e == hipSuccess ? GEMM_OK : hip_fail(e, "hipLaunchKernel");
}

} // namespace pts

// Argument checks shared by the host files.
#pragma once

#include <climits>

#include "host_launch.h"
#include "linear/plan.h"
#include "pts_linear.h"

namespace pts {

constexpr int64_t MAX_PITCH = 1 << 22; // elements: 256 rows of them are within 2^31 bytes
inline bool extent(int64_t v) { return v >= 0 && v < MAX_EXTENT; }
inline bool operand_width(int64_t v) { return v <= MAX_PITCH - 8; } // some row stride passes check_operand
// Row stride of the library's own 16-bit matrices: rows start at whole cache lines, since a k tile of a row that starts
// inside one takes two (dx of 5000 x 7000 x 3000: 204 us, 178 with aligned rows of dz).
inline int64_t own_pitch(int64_t n) { return (n + 63) / 64 * 64; }

// A bf16 operand that the matrix unit reads: rows x width.
inline gemm_status check_operand(const char *name, const void *p, int64_t ld, int64_t rows, int64_t width)
{
    if (ld < width)
        return fail(GEMM_ERR_INVALID_VALUE, "%s: leading dimension %lld smaller than the packed extent %lld", name, (long long)ld,
                    (long long)width);
    if (ld % 8 != 0)
        return fail(GEMM_ERR_INVALID_VALUE, "%s: leading dimension %lld is not a multiple of 8 elements", name, (long long)ld);
    if (ld >= MAX_PITCH)
        return fail(GEMM_ERR_UNSUPPORTED, "%s: leading dimension %lld: a tile's offsets must fit in 32-bit", name, (long long)ld);
    if (rows > 0 && width > 0 && p == nullptr)
        return fail(GEMM_ERR_INVALID_VALUE, "%s: NULL pointer", name);
    if (!aligned(p, 16))
        return fail(GEMM_ERR_INVALID_VALUE, "%s must be 16-byte aligned", name);
    return GEMM_OK;
}

// A result or an addend of `size`-byte elements.
inline gemm_status check_rows(const char *name, const void *p, int64_t ld, int64_t rows, int64_t width, int size)
{
    if (ld < width || ld > INT64_MAX / 16 / (rows > 0 ? rows : 1))
        return fail(GEMM_ERR_INVALID_VALUE, "%s: leading dimension %lld for rows of %lld", name, (long long)ld, (long long)width);
    if (rows > 0 && width > 0 && p == nullptr)
        return fail(GEMM_ERR_INVALID_VALUE, "%s: NULL pointer", name);
    if (!aligned(p, size))
        return fail(GEMM_ERR_INVALID_VALUE, "%s must be element aligned", name);
    return GEMM_OK;
}
inline bool whole_rows(const void *p, int64_t ld, int size) { return aligned(p, 16) && ld * size % 16 == 0; }

inline gemm_status check_workspace(const void *workspace, size_t bytes, int64_t need)
{
    if (need > 0 && (workspace == nullptr || bytes < (size_t)need))
        return fail(GEMM_ERR_INVALID_VALUE, "workspace of %zu bytes; %lld needed", workspace == nullptr ? (size_t)0 : bytes, (long long)need);
    if (!aligned(workspace, 16))
        return fail(GEMM_ERR_INVALID_VALUE, "the workspace must be 16-byte aligned");
    return GEMM_OK;
}

} // namespace pts

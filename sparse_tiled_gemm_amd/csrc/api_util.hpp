// Host helpers shared by the C ABI layers (gemm_api.cpp, moe_api.cpp): status
// and message of the calling thread, the device check, size arithmetic and
// overlap tests.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.h"

namespace stg {

// Record a failure's message for gemm_last_error() and return its status.
gemm_status_t fail(gemm_status_t st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// Clear the message.
gemm_status_t ok();
gemm_status_t hip_fail(hipError_t e, const char *what);

struct DeviceInfo {
    int checked = 0;
    int is_gfx950 = 0;
    int num_cu = 0;
    char arch[64] = "";
};
// The current device, which has to be a gfx950.
gemm_status_t check_device(int *dev_out, DeviceInfo *info_out);

// a * b for a, b >= 0, saturating at INT64_MAX (size checks never overflow)
inline int64_t smul(int64_t a, int64_t b)
{
    return (a != 0 && b > INT64_MAX / a) ? INT64_MAX : a * b;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Byte range [lo, hi) of a matrix of `rows` rows of `cols` elements of
// `eb` bytes, `ld` elements apart.
struct Span {
    uintptr_t lo = 0, hi = 0;
};
inline Span span(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t eb)
{
    Span s;
    if (!p || rows <= 0 || cols <= 0)
        return s;
    s.lo = (uintptr_t)p;
    s.hi = s.lo + (uintptr_t)(((rows - 1) * ld + cols) * eb);
    return s;
}
inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

} // namespace stg

// Argument checks of the C ABI layers whose calls take matrices without a plan
// or with one of their own (moe_api.cpp, vocab_api.cpp).
#pragma once

#include <initializer_list>

#include "api_util.hpp"

namespace stg {

constexpr int64_t MAX_ELEMS = (int64_t)1 << 40;

inline bool is_16bit(int t) { return t == GEMM_F16 || t == GEMM_BF16; }

// A rows x cols matrix of leading dimension ld (0 = packed, filled in):
// negative sizes, a leading dimension below cols, more than 2^40 elements.
inline gemm_status_t check_matrix(const char *name, int64_t rows, int64_t cols, int64_t *ld)
{
    if (*ld == 0)
        *ld = cols > 0 ? cols : 1;
    if (rows < 0 || cols < 0 || *ld < cols)
        return fail(GEMM_ERR_INVALID_VALUE,
                    "%s: negative size or leading dimension smaller than the row", name);
    if (*ld > MAX_ELEMS || smul(rows, *ld) > MAX_ELEMS)
        return fail(GEMM_ERR_INVALID_VALUE, "%s spans more than 2^40 elements", name);
    return GEMM_OK;
}

// A buffer of a call: its bytes, its element alignment, and its part in it.
struct Buf {
    const char *name;
    const void *p;
    int64_t rows, cols, ld, eb;
    bool out;
    int align = 0; // bytes; 0 = eb
};

// Required pointers, alignment, and outputs apart from everything else.
// Buffers without elements may be NULL.
inline gemm_status_t check_buffers(std::initializer_list<Buf> bufs)
{
    for (const Buf &b : bufs) {
        if (b.rows <= 0 || b.cols <= 0)
            continue;
        if (!b.p)
            return fail(GEMM_ERR_NULL_POINTER, "%s is NULL", b.name);
        if (!aligned(b.p, (size_t)(b.align ? b.align : b.eb)))
            return fail(GEMM_ERR_MISALIGNED, "%s is not aligned to its element size", b.name);
    }
    for (const Buf *x = bufs.begin(); x != bufs.end(); ++x)
        for (const Buf *y = bufs.begin(); y != bufs.end(); ++y)
            if (x != y && x->out && overlap(span(x->p, x->rows, x->cols, x->ld, x->eb),
                                            span(y->p, y->rows, y->cols, y->ld, y->eb)))
                return fail(GEMM_ERR_UNSUPPORTED, "%s overlaps %s", x->name, y->name);
    return GEMM_OK;
}

inline gemm_status_t check_gfx950() // (the device's own check, once per call)
{
    int dev = 0;
    return check_device(&dev, nullptr);
}

inline gemm_status_t launched(hipError_t e)
{
    return e == hipSuccess ? ok() : hip_fail(e, "kernel launch");
}

#define CHECK(x)                     \
    do {                             \
        const gemm_status_t st_ = x; \
        if (st_ != GEMM_OK)          \
            return st_;              \
    } while (0)

} // namespace stg

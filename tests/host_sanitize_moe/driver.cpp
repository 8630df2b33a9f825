// Host-only driver of the mixture-of-experts entry points (moe_api.cpp) for an
// AddressSanitizer / UndefinedBehaviorSanitizer build: the HIP runtime and
// the dense launchers are the stubs of ../host_sanitize/driver.cpp, the
// launchers of moe_args.hpp are stubbed here and check what the kernels rely
// on.  Seeded calls with sizes, leading dimensions, types and pointers from
// extreme sets; exit status 0 means no sanitizer report and no failed
// expectation.
#define main dense_main
#include "../host_sanitize/driver.cpp"
#undef main

#include "gemm_moe.h"
#include "moe_args.hpp"

namespace stg {
hipError_t launch_route(const RouteArgs &a, const RowsArgs *r, hipStream_t)
{
    EXPECT(a.slots >= 0 && a.slots <= INT32_MAX && a.groups >= 1 && a.groups <= ROUTE_MAX_GROUPS);
    EXPECT(a.offsets && (a.slots == 0 || (a.ids && a.order && a.pos)));
    EXPECT(a.chunk >= 512 && a.chunk % 512 == 0 && a.chunks <= 256);
    EXPECT((int64_t)a.chunk * a.chunks >= a.slots);
    EXPECT(a.slots <= ROUTE_SMALL || a.counts);
    if (r) {
        EXPECT(r->cols >= 0 && r->cols <= (1 << 23) && r->ld_in >= r->cols && r->ld_out >= r->cols);
        EXPECT(r->cols == 0 || a.slots == 0 || (r->in && r->out));
    }
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_combine(const RowsArgs &a, hipStream_t)
{
    EXPECT(a.tokens > 0 && a.cols > 0 && a.pos && a.out && (a.rows == 0 || a.in));
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_combine_backward(const RowsArgs &a, hipStream_t)
{
    EXPECT(a.tokens > 0 && a.pos && a.weights && a.dw);
    EXPECT(a.cols == 0 || (a.in && (a.rows == 0 || (a.in2 && a.out))));
    ++g_launches;
    return hipSuccess;
}
static hipError_t q8(const Q8Args &a)
{
    EXPECT(a.rows > 0 && a.cols > 0 && (!a.codes == !a.scales));
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_q8_store(const Q8Args &a, hipStream_t) { return q8(a); }
hipError_t launch_q8_load(const Q8Args &a, hipStream_t) { return q8(a); }
hipError_t launch_swiglu(const Q8Args &a, hipStream_t)
{
    EXPECT(a.cols % 2 == 0 && a.out);
    return q8(a);
}
hipError_t launch_swiglu_backward(const Q8Args &a, hipStream_t) { return launch_swiglu(a, nullptr); }
hipError_t launch_grouped(int f, const GroupedArgs &a, hipStream_t)
{
    EXPECT(f >= 0 && f < GF_COUNT && a.groups >= 1 && a.groups <= 65535 && a.N > 0 && a.D);
    EXPECT((a.weights_mode ? a.K : a.rows) > 0 && a.ldd >= a.N && a.lda >= a.K && a.offsets);
    EXPECT(a.num_cu == 256);
    if (f != GF_GENERIC) {
        // 16-byte chunks inside the rows, 32-bit offsets
        EXPECT(a.K % 8 == 0 && a.lda % 8 == 0 && a.ldb % 8 == 0 && a.lda < (1 << 21) &&
               a.ldb < (1 << 21));
        EXPECT(!(a.weights_mode || a.b_row) || a.N % 8 == 0);
        EXPECT((uintptr_t)a.A % 16 == 0 && (uintptr_t)a.B % 16 == 0);
    }
    EXPECT(f != GF_SKINNY || !a.weights_mode);
    // a grid of 2^32 - 1 threads
    const int64_t g = a.groups < a.rows ? a.groups : a.rows;
    const int64_t b = f == GF_TILED_256 ? 256 : f == GF_TILED_128 ? 128 : 64;
    const int64_t nb = f == GF_SKINNY ? 32 : b;
    const int64_t tiles =
        a.weights_mode ? ((a.K + b - 1) / b * ((a.N + b - 1) / b) + 7) / 8 * 8 * a.groups
                       : ((a.rows + b - 1) / b + g) * ((a.N + nb - 1) / nb) + 256;
    EXPECT(tiles * (b == 64 && f != GF_SKINNY ? 256 : 512) < ((int64_t)1 << 32));
    ++g_launches;
    return hipSuccess;
}
} // namespace stg

// A fake address, sometimes NULL, misaligned or another buffer's.
static void *ptr(int i)
{
    switch (rnd() % 24) {
    case 0: return nullptr;
    case 1: return (char *)fake(i) + 1 + rnd() % 15;
    case 2: return fake((int)(rnd() % 8) + 1);
    default: return fake(i);
    }
}
static bool status_ok(gemm_status_t s)
{
    return s == GEMM_OK || s == GEMM_ERR_NULL_POINTER || s == GEMM_ERR_INVALID_VALUE ||
           s == GEMM_ERR_UNSUPPORTED || s == GEMM_ERR_MISALIGNED;
}
static const int64_t MOE_SIZES[] = {-1, 0, 1, 2, 3, 8, 64, 72, 100, 1024, 4097, 65536, 1 << 23,
                                    (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX, INT64_MIN};
static const int64_t MOE_LD[] = {0, 0, 0, 0, 8, 64, 8192, (int64_t)1 << 22, INT64_MAX, -1};
static int64_t size() { return rnd() % 3 ? MOE_SIZES[1 + rnd() % 11] : pick(MOE_SIZES); }
static int32_t type() { return rnd() % 4 ? (rnd() & 1 ? GEMM_F16 : GEMM_BF16) : pick(TYPES); }

int main(int argc, char **argv)
{
    const long iters = argc > 1 ? atol(argv[1]) : 100000;
    long good = 0;
    for (long i = 0; i < iters; ++i) {
        const int64_t t = size(), k = 1 + (int64_t)(rnd() % 9), g = size(), c = size(), r = size();
        const int32_t ty = type(), ib = rnd() % 8 ? (rnd() & 1 ? 4 : 8) : 3;
        size_t n = 0;
        gemm_status_t s = gemm_moe_sort_workspace(t, k, g, &n);
        EXPECT(status_ok(s));
        EXPECT(s != GEMM_OK || n <= (size_t)256 * 1024 * 4);
        s = gemm_moe_sort(t, k, g, ib, ptr(1), (int32_t *)ptr(2), (int32_t *)ptr(3),
                          (int32_t *)ptr(4), ptr(5), nullptr);
        EXPECT(status_ok(s));
        good += s == GEMM_OK;
        s = gemm_moe_dispatch(t, k, g, c, ty, ib, ptr(1), ptr(6), pick(MOE_LD), (int32_t *)ptr(2),
                              (int32_t *)ptr(3), (int32_t *)ptr(4), ptr(7), pick(MOE_LD), ptr(5),
                              nullptr);
        EXPECT(status_ok(s));
        good += s == GEMM_OK;
        s = gemm_moe_combine(t, k, c, ty, (int32_t *)ptr(1), rnd() & 1 ? (float *)ptr(2) : nullptr,
                             ptr(3), pick(MOE_LD), r, ptr(4), pick(MOE_LD), nullptr);
        EXPECT(status_ok(s));
        good += s == GEMM_OK;
        s = gemm_moe_combine_backward(t, k, c, ty, (int32_t *)ptr(1), (float *)ptr(2), ptr(3),
                                      pick(MOE_LD), ptr(4), pick(MOE_LD), r, ptr(5), pick(MOE_LD),
                                      (float *)ptr(6), nullptr);
        EXPECT(status_ok(s));
        good += s == GEMM_OK;
        uint8_t *q = (uint8_t *)ptr(2), *sc = (uint8_t *)ptr(3);
        s = gemm_q8_store(r, c, ty, ptr(1), pick(MOE_LD), q, sc, nullptr);
        EXPECT(status_ok(s));
        s = gemm_q8_load(r, c, ty, q, sc, ptr(1), pick(MOE_LD), nullptr);
        EXPECT(status_ok(s));
        s = gemm_swiglu(r, c, ty, ptr(1), pick(MOE_LD), ptr(4), pick(MOE_LD), q, sc, nullptr);
        EXPECT(status_ok(s));
        good += s == GEMM_OK;
        s = gemm_swiglu_backward(r, c, ty, q, sc, ptr(1), pick(MOE_LD), ptr(4), pick(MOE_LD),
                                 rnd() & 1 ? ptr(5) : nullptr, pick(MOE_LD), nullptr);
        EXPECT(status_ok(s));
        good += s == GEMM_OK;

        gemm_grouped_desc_t d{};
        d.mode = rnd() % 16 ? (int32_t)(rnd() & 1) : 7;
        d.groups = rnd() % 8 ? 1 + (int32_t)(rnd() % 100) : (int32_t)g;
        d.rows = size();
        d.N = size();
        d.K = size();
        d.a_type = ty;
        d.b_type = d.mode && rnd() & 1 ? GEMM_F8_E4M3 : rnd() % 8 ? ty : type();
        d.d_type = rnd() & 1 ? GEMM_F32 : type();
        d.b_layout = d.mode ? 0 : (int32_t)(rnd() & 1);
        d.has_c = d.mode ? (int32_t)(rnd() & 1) : 0;
        d.algo = rnd() & 1 ? 0 : (int32_t)(rnd() % 8) - 1;
        d.lda = pick(MOE_LD);
        d.ldb = pick(MOE_LD);
        d.ldd = pick(MOE_LD);
        const gemm_status_t v = gemm_grouped_validate_desc(&d);
        gemm_grouped_plan_t *p = nullptr;
        s = gemm_grouped_plan(&d, &p);
        EXPECT(s == v || (v == GEMM_OK && s == GEMM_ERR_UNSUPPORTED && d.algo));
        EXPECT((s == GEMM_OK) == (p != nullptr));
        if (p) {
            char name[64];
            EXPECT(gemm_grouped_plan_describe(p, name, sizeof name) == GEMM_OK && name[0]);
            s = gemm_grouped_run(p, ptr(1), ptr(2), (uint8_t *)ptr(3), (int32_t *)ptr(4), ptr(5),
                                 rnd() & 1 ? fake(5) : ptr(6), nullptr);
            EXPECT(status_ok(s));
            good += s == GEMM_OK;
            EXPECT(gemm_grouped_plan_destroy(p) == GEMM_OK);
        }
    }
    EXPECT(good > iters / 4); // the sets reach the launchers
    printf("moe host driver: %ld rounds, %ld accepted calls, %ld launches, %s\n", iters, good,
           g_launches, g_fail ? "FAILED" : "ok");
    return g_fail;
}

// Host-only driver of the entry points over a vocabulary (vocab_api.cpp) for an
// AddressSanitizer / UndefinedBehaviorSanitizer build: the HIP runtime and
// the dense launchers are the stubs of ../host_sanitize/driver.cpp, the
// launchers of vocab_args.hpp are stubbed here and check what the kernels rely
// on, above all that every part of a workspace lies inside it.  Seeded calls
// with sizes, leading dimensions, types and pointers from extreme sets; exit
// status 0 means no sanitizer report and no failed expectation.
#define main dense_main
#include "../host_sanitize/driver.cpp"
#undef main

#include "gemm_vocab.h"
#include "vocab_args.hpp"

static uintptr_t g_ws; // the workspace of the call under way, and its bytes
static size_t g_bytes;

namespace stg {
static bool inside(const void *p, int64_t n, size_t size)
{
    const uintptr_t a = (uintptr_t)p;
    return n >= 0 && a >= g_ws && a % 16 == 0 && a - g_ws <= g_bytes &&
           (size_t)n * size <= g_bytes - (a - g_ws);
}

hipError_t launch_embed(const EmbedArgs &a, hipStream_t)
{
    EXPECT(a.tokens > 0 && a.tokens <= (1 << 25) && a.cols > 0 && a.cols <= (1 << 23));
    EXPECT(a.vocab >= 0 && a.vocab <= EMBED_MAX_VOCAB && a.ids && a.out && (a.in || a.vocab == 0));
    EXPECT(a.ld_in >= a.cols && a.ld_out >= a.cols);
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_embed_backward(const EmbedArgs &a, hipStream_t)
{
    EXPECT(a.vocab > 0 && a.vocab <= EMBED_MAX_VOCAB && a.cols > 0 && a.out);
    EXPECT(a.tokens > 0 || !a.accumulate);
    EXPECT(a.tokens == 0 || (a.ids && a.in));
    if (a.tokens > EMBED_SMALL) {
        const int64_t lows = (int64_t)1 << a.lo_bits;
        EXPECT(lows <= EMBED_MAX_BINS && 1 << a.hi_bits <= EMBED_MAX_BINS);
        EXPECT(lows << a.hi_bits >= a.vocab); // every id has a bin in both passes
        EXPECT(a.chunk % 512 == 0 && a.chunks <= 256 && (int64_t)a.chunk * a.chunks >= a.tokens);
        EXPECT(inside(a.counts, a.chunks * lows, 4) && inside(a.bounds, lows + 1, 4));
        EXPECT(inside(a.binned, a.tokens, 8) && inside(a.order, a.tokens, 4));
        EXPECT(inside(a.key, a.tokens, 4));
        EXPECT(inside(a.part, (a.tokens + EMBED_RUN - 1) / EMBED_RUN * 2 * a.cols, 4));
        // one launch holds 2^32 - 1 threads: the runs' join is the largest
        EXPECT((a.tokens + EMBED_RUN - 1) / EMBED_RUN * 512 < ((int64_t)1 << 32));
    }
    ++g_launches;
    return hipSuccess;
}

static void check_args(const XentArgs &a, bool backward)
{
    EXPECT(a.tokens >= 0 && a.tokens <= (1 << 20) && a.hp % 8 == 0 && a.hp >= a.hidden);
    EXPECT(a.prep > 0 && a.prep % XENT_STEP == 0);
    EXPECT(inside(a.count, 2, 4) && inside(a.pos, a.tokens, 4) && inside(a.map, a.tokens, 4));
    EXPECT(inside(a.tgt, a.tokens, 4) && a.ldc >= a.hp && inside(a.Xc, a.tokens * a.ldc, 2));
    if (backward) {
        EXPECT(inside(a.ca, a.tokens, 4) && inside(a.cb, a.tokens, 4) && inside(a.cl, a.tokens, 4));
        EXPECT(a.gmaxes >= 1 && a.gmaxes * a.prep >= a.tokens && inside(a.gmax, a.gmaxes, 4));
    } else {
        EXPECT(a.part_tiles > 0 && inside(a.part, a.part_tiles * a.tokens * 2, 4));
        EXPECT(inside(a.zt, a.tokens, 4) && a.lse);
        // what the kernels read where it lies
        EXPECT(!a.direct || (a.tokens <= 64 && a.hidden % 8 == 0 && a.ldx % 8 == 0 &&
                             (uintptr_t)a.X % 16 == 0));
    }
}
static void check_piece(int tile, const XentArgs &a, const XentPiece &p)
{
    EXPECT(p.n > 0 && p.v0 >= 0 && p.v0 + p.n <= a.vocab && (p.loose || p.ldw % 8 == 0) && p.ldw < (1 << 21));
    if (p.loose)
        EXPECT(!p.G && a.tokens <= XENT_STREAM_ROWS && p.ldw >= a.hidden && p.ldw < (1 << 21));
    else
        EXPECT((uintptr_t)p.W % 16 == 0 && p.ldw >= a.hp);
    EXPECT(tile >= 0 && (tile < XT_COUNT || (tile == XT_STREAM && a.tokens <= XENT_STREAM_ROWS)));
    if (tile < XT_COUNT) {
        const int64_t b = xent_edge(tile);
        EXPECT((a.tokens + b - 1) / b * ((p.n + b - 1) / b) * 512 < ((int64_t)1 << 32));
    }
}
hipError_t launch_xent_prepare(const XentArgs &a, bool backward, hipStream_t)
{
    check_args(a, backward);
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_xent_copy(const XentCopy &c, hipStream_t)
{
    EXPECT(c.W && c.n > 0 && c.ldw >= c.hidden && c.ldo >= c.hp && inside(c.out, c.n * c.ldo, 2));
    return hipSuccess;
}
hipError_t launch_xent_stats(int tile, const XentArgs &a, const XentPiece &p, hipStream_t)
{
    check_args(a, false);
    check_piece(tile, a, p);
    const int64_t parts = tile == XT_STREAM ? xent_streams(p.n, a.dx.num_cu)
                                            : (p.n + xent_edge(tile) - 1) / xent_edge(tile);
    EXPECT(p.tile0 >= 0 && p.tile0 + parts <= a.part_tiles);
    return hipSuccess;
}
hipError_t launch_xent_loss(const XentArgs &a, hipStream_t)
{
    check_args(a, false);
    return hipSuccess;
}
static void check_g(const XentArgs &a, const XentPiece &p)
{
    check_args(a, true);
    EXPECT(p.ldg % 256 == 0 && p.ldg >= p.n && p.ldg <= (1 << 20) && inside(p.G, a.tokens * p.ldg, 2));
}
hipError_t launch_xent_g(int tile, const XentArgs &a, const XentPiece &p, hipStream_t)
{
    check_piece(tile, a, p);
    check_g(a, p);
    return hipSuccess;
}
// acc holds the parts that any number of rows chooses
static void check_acc(const XentArgs &a, const float *acc)
{
    const XentSplits &x = a.dx;
    EXPECT(x.cols > 0 && x.most >= 1 && x.slots > 0 && x.edge >= 64);
    for (int64_t n : {(int64_t)1, a.tokens / 3, a.tokens / 2, a.tokens - 1, a.tokens}) {
        if (n < 1)
            continue;
        const int s = xent_splits((int)n, x.edge, x.tiles_n, x.cols, x.slots, x.most);
        EXPECT(s >= 1 && s <= x.most && inside(acc, s * n * a.hp, 4));
        EXPECT((n + x.edge - 1) / x.edge * x.tiles_n * s <= x.wgs);
    }
    EXPECT((int64_t)x.wgs * 512 < ((int64_t)1 << 32));
}
hipError_t launch_xent_dx(int tile, const XentArgs &a, const XentPiece &p, const XentDx &d, hipStream_t)
{
    check_piece(tile, a, p);
    check_g(a, p);
    check_acc(a, d.acc);
    EXPECT(d.add == (p.v0 > 0) && tile < XT_COUNT && xent_edge(tile) == a.dx.edge);
    return hipSuccess;
}
hipError_t launch_xent_dw(int tile, const XentArgs &a, const XentPiece &p, const XentDw &d, hipStream_t)
{
    check_g(a, p);
    EXPECT(d.dW && d.ldd >= a.hidden && tile <= XT_STREAM);
    if (tile == XT_STREAM) {
        EXPECT(a.tokens > 0 && a.tokens <= XENT_DW_ROWS && a.hidden % 8 == 0 && d.vec);
        EXPECT((uintptr_t)d.dW % 16 == 0 && d.ldd * (d.d_kind == OUT_F32 ? 4 : 2) % 16 == 0);
        return hipSuccess;
    }
    const int64_t b = xent_edge(tile);
    EXPECT((p.n + b - 1) / b * ((a.hp + b - 1) / b) * 512 < ((int64_t)1 << 32));
    EXPECT(!d.vec || ((uintptr_t)d.dW % 8 == 0 && d.ldd % 4 == 0));
    return hipSuccess;
}
hipError_t launch_xent_out(const XentArgs &a, const XentOut &o, hipStream_t)
{
    check_args(a, true);
    check_acc(a, o.acc);
    EXPECT(o.dX && o.ldd >= a.hidden);
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
static void *ws(size_t bytes)
{
    void *p = rnd() % 16 ? fake(9) : ptr(9);
    g_ws = (uintptr_t)p;
    g_bytes = bytes;
    return p;
}
static bool status_ok(gemm_status_t s)
{
    return s == GEMM_OK || s == GEMM_ERR_NULL_POINTER || s == GEMM_ERR_INVALID_VALUE ||
           s == GEMM_ERR_UNSUPPORTED || s == GEMM_ERR_MISALIGNED;
}
static const int64_t V_SIZES[] = {1, 2, 7, 16, 17, 64, 65, 100, 777, 1024, 1025, 4096, 50021, 65536,
                                  131072, 1 << 20, (1 << 20) + 1, 1 << 24, 1 << 25, -1, 0,
                                  (int64_t)1 << 31, INT64_MAX, INT64_MIN};
static const int64_t V_LD[] = {0, 0, 0, 0, 0, 8, 72, 4096, 8192, (int64_t)1 << 21, INT64_MAX, -1};
static int64_t size() { return rnd() % 8 ? V_SIZES[rnd() % 16] : pick(V_SIZES); }
static int32_t ftype() { return rnd() % 8 ? (rnd() % 3 == 0 ? GEMM_F32 : rnd() & 1 ? GEMM_F16 : GEMM_BF16) : pick(TYPES); }

int main(int argc, char **argv)
{
    const long iters = argc > 1 ? atol(argv[1]) : 100000;
    long good = 0;
    for (long i = 0; i < iters; ++i) {
        const int64_t t = size(), v = size(), c = size();
        const int32_t ib = rnd() % 8 ? (rnd() & 1 ? 4 : 8) : 3;
        size_t n = 0;
        gemm_status_t s = gemm_embed(t, v, c, ftype(), ftype(), ib, ptr(1), ptr(2), pick(V_LD), ptr(3),
                                     pick(V_LD), 2.0f, nullptr);
        EXPECT(status_ok(s));
        good += s == GEMM_OK;
        s = gemm_embed_workspace(t, v, c, &n);
        EXPECT(status_ok(s));
        s = gemm_embed_backward(t, v, c, ftype(), ftype(), ib, ptr(1), ptr(2), pick(V_LD), ptr(3),
                                pick(V_LD), (int32_t)(rnd() % 9) % 2, ws(n), 1.0f, nullptr);
        EXPECT(status_ok(s));
        good += s == GEMM_OK;

        gemm_xent_desc_t d{};
        d.tokens = size();
        d.vocab = size();
        d.hidden = size();
        d.x_type = rnd() % 8 ? (rnd() & 1 ? GEMM_F16 : GEMM_BF16) : pick(TYPES);
        d.dx_type = ftype();
        d.dw_type = ftype();
        d.id_bytes = ib;
        d.accumulate = (int32_t)(rnd() & 1);
        d.unaligned = rnd() % 4 == 0;
        d.ldx = pick(V_LD);
        d.ldw = pick(V_LD);
        d.lddx = pick(V_LD);
        d.lddw = pick(V_LD);
        d.piece = rnd() & 1 ? 0 : size();
        d.scale = 1.0f;
        const gemm_status_t valid = gemm_xent_validate_desc(&d);
        gemm_xent_plan_t *p = nullptr;
        s = gemm_xent_plan(&d, &p);
        EXPECT(s == valid && (s == GEMM_OK) == (p != nullptr));
        if (!p)
            continue;
        char name[96];
        EXPECT(gemm_xent_plan_describe(p, name, sizeof name) == GEMM_OK && name[0]);
        size_t f = 0, b = 0;
        EXPECT(gemm_xent_workspace(p, &f, &b) == GEMM_OK && f > 0 && b > 0);
        s = gemm_xent_forward(p, ptr(1), ptr(2), ptr(3), rnd() & 1 ? (float *)ptr(4) : nullptr,
                              (float *)ptr(5), ws(f), nullptr);
        EXPECT(status_ok(s));
        good += s == GEMM_OK;
        s = gemm_xent_backward(p, ptr(1), ptr(2), ptr(3), (float *)ptr(4), (float *)ptr(5),
                               rnd() & 1 ? (float *)ptr(6) : nullptr, rnd() % 4 ? ptr(7) : nullptr,
                               rnd() % 4 ? ptr(8) : nullptr, ws(b), nullptr);
        EXPECT(status_ok(s));
        good += s == GEMM_OK;
        EXPECT(gemm_xent_plan_destroy(p) == GEMM_OK);
    }
    EXPECT(good > iters / 4); // the sets reach the launchers
    printf("vocab host driver: %ld rounds, %ld accepted calls, %ld launches, %s\n", iters, good,
           g_launches, g_fail ? "FAILED" : "ok");
    return g_fail;
}

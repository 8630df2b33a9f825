// C ABI of the mixture-of-experts operators: argument checks, plan choice and
// launch.  The operations are documented in include/gemm_moe.h.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>

#include "api_checks.hpp"
#include "gemm_moe.h"
#include "kernel_args.hpp"
#include "moe_args.hpp"

using namespace stg;

struct gemm_grouped_plan {
    gemm_grouped_desc_t d; // normalised: packed leading dimensions filled in
    int family;            // stg::GroupedFamily
    int device, num_cu;
    char name[64];
};

namespace {

// ---------------------------------------------------------------- routing

gemm_status_t check_route(int64_t tokens, int64_t topk)
{
    if (tokens < 0 || topk < 1)
        return fail(GEMM_ERR_INVALID_VALUE, "tokens must be >= 0 and topk >= 1");
    if (smul(tokens, topk) > INT32_MAX)
        return fail(GEMM_ERR_UNSUPPORTED, "tokens * topk must be below 2^31");
    return GEMM_OK;
}

gemm_status_t check_groups(int64_t groups)
{
    if (groups < 1)
        return fail(GEMM_ERR_INVALID_VALUE, "groups must be >= 1");
    if (groups > ROUTE_MAX_GROUPS)
        return fail(GEMM_ERR_UNSUPPORTED, "at most %d groups", ROUTE_MAX_GROUPS);
    return GEMM_OK;
}

gemm_status_t check_rows_type(int64_t cols, int32_t type)
{
    if (type < GEMM_F16 || type > GEMM_U8)
        return fail(GEMM_ERR_INVALID_VALUE, "unknown dtype code");
    if (!is_16bit(type))
        return fail(GEMM_ERR_UNSUPPORTED, "type must be f16 or bf16");
    if (cols < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "negative number of columns");
    if (cols > (1 << 23))
        return fail(GEMM_ERR_UNSUPPORTED, "at most 2^23 columns");
    return GEMM_OK;
}

size_t sort_workspace(int64_t slots, int64_t groups)
{
    if (slots <= ROUTE_SMALL)
        return 0;
    return (size_t)(ceil_div(slots, route_chunk(slots)) * groups) * sizeof(int32_t);
}

// Checks of gemm_moe_sort and gemm_moe_dispatch, and the launch arguments.
gemm_status_t make_route(RouteArgs &a, int64_t tokens, int64_t topk, int64_t groups,
                         int32_t id_bytes, const void *ids, int32_t *offsets, int32_t *order,
                         int32_t *pos, void *workspace)
{
    CHECK(check_route(tokens, topk));
    CHECK(check_groups(groups));
    if (id_bytes != 4 && id_bytes != 8)
        return fail(GEMM_ERR_INVALID_VALUE, "id_bytes must be 4 or 8");
    a.tokens = tokens;
    a.topk = topk;
    a.slots = tokens * topk;
    a.groups = (int)groups;
    a.id8 = id_bytes == 8;
    a.ids = ids;
    a.offsets = offsets;
    a.order = order;
    a.pos = pos;
    a.chunk = (int)route_chunk(a.slots);
    a.chunks = (int)ceil_div(a.slots, a.chunk);
    a.counts = (int32_t *)workspace;
    return GEMM_OK;
}

} // namespace

extern "C" {

gemm_status_t gemm_moe_sort_workspace(int64_t tokens, int64_t topk, int64_t groups, size_t *bytes)
{
    if (!bytes)
        return fail(GEMM_ERR_NULL_POINTER, "bytes is NULL");
    CHECK(check_route(tokens, topk));
    CHECK(check_groups(groups));
    *bytes = sort_workspace(tokens * topk, groups);
    return ok();
}

gemm_status_t gemm_moe_sort(int64_t tokens, int64_t topk, int64_t groups, int32_t id_bytes,
                            const void *ids, int32_t *offsets, int32_t *order, int32_t *pos,
                            void *workspace, gemm_stream_t stream)
{
    RouteArgs a{};
    CHECK(make_route(a, tokens, topk, groups, id_bytes, ids, offsets, order, pos, workspace));
    const int64_t n = a.slots, wn = (int64_t)sort_workspace(n, groups) / 4;
    CHECK(check_buffers({{"ids", ids, n, 1, 1, id_bytes, false},
                         {"offsets", offsets, groups + 1, 1, 1, 4, true},
                         {"order", order, n, 1, 1, 4, true},
                         {"pos", pos, n, 1, 1, 4, true},
                         {"workspace", workspace, wn, 1, 1, 4, true}}));
    CHECK(check_gfx950());
    return launched(launch_route(a, nullptr, (hipStream_t)stream));
}

gemm_status_t gemm_moe_dispatch(int64_t tokens, int64_t topk, int64_t groups, int64_t cols,
                                int32_t type, int32_t id_bytes, const void *ids, const void *X,
                                int64_t ldx, int32_t *offsets, int32_t *order, int32_t *pos,
                                void *Xs, int64_t ldxs, void *workspace, gemm_stream_t stream)
{
    RouteArgs a{};
    CHECK(make_route(a, tokens, topk, groups, id_bytes, ids, offsets, order, pos, workspace));
    CHECK(check_rows_type(cols, type));
    CHECK(check_matrix("X", tokens, cols, &ldx));
    CHECK(check_matrix("Xs", a.slots, cols, &ldxs));
    const int64_t n = a.slots, wn = (int64_t)sort_workspace(n, groups) / 4;
    CHECK(check_buffers({{"ids", ids, n, 1, 1, id_bytes, false},
                         {"X", X, tokens, cols, ldx, 2, false},
                         {"offsets", offsets, groups + 1, 1, 1, 4, true},
                         {"order", order, n, 1, 1, 4, true},
                         {"pos", pos, n, 1, 1, 4, true},
                         {"Xs", Xs, n, cols, ldxs, 2, true},
                         {"workspace", workspace, wn, 1, 1, 4, true}}));
    CHECK(check_gfx950());
    RowsArgs r{};
    r.tokens = tokens;
    r.topk = topk;
    r.cols = cols;
    r.rows = n;
    r.pos = pos;
    r.in = X;
    r.ld_in = ldx;
    r.out = Xs;
    r.ld_out = ldxs;
    return launched(launch_route(a, &r, (hipStream_t)stream));
}

gemm_status_t gemm_moe_combine(int64_t tokens, int64_t topk, int64_t cols, int32_t type,
                               const int32_t *pos, const float *weights, const void *Ys,
                               int64_t ldys, int64_t rows, void *Y, int64_t ldy,
                               gemm_stream_t stream)
{
    CHECK(check_route(tokens, topk));
    CHECK(check_rows_type(cols, type));
    CHECK(check_matrix("Ys", rows, cols, &ldys));
    CHECK(check_matrix("Y", tokens, cols, &ldy));
    const int64_t n = tokens * topk;
    CHECK(check_buffers({{"pos", pos, n, 1, 1, 4, false},
                         {"weights", weights, weights ? n : 0, 1, 1, 4, false},
                         {"Ys", Ys, rows, cols, ldys, 2, false},
                         {"Y", Y, tokens, cols, ldy, 2, true}}));
    if (tokens == 0 || cols == 0)
        return ok();
    CHECK(check_gfx950());
    RowsArgs r{};
    r.tokens = tokens;
    r.topk = topk;
    r.cols = cols;
    r.rows = rows;
    r.pos = pos;
    r.weights = weights;
    r.in = Ys;
    r.ld_in = ldys;
    r.out = Y;
    r.ld_out = ldy;
    r.bf16 = type == GEMM_BF16;
    return launched(launch_combine(r, (hipStream_t)stream));
}

gemm_status_t gemm_moe_combine_backward(int64_t tokens, int64_t topk, int64_t cols, int32_t type,
                                        const int32_t *pos, const float *weights, const void *dY,
                                        int64_t lddy, const void *Ys, int64_t ldys, int64_t rows,
                                        void *dYs, int64_t lddys, float *dw, gemm_stream_t stream)
{
    CHECK(check_route(tokens, topk));
    CHECK(check_rows_type(cols, type));
    CHECK(check_matrix("dY", tokens, cols, &lddy));
    CHECK(check_matrix("Ys", rows, cols, &ldys));
    CHECK(check_matrix("dYs", rows, cols, &lddys));
    const int64_t n = tokens * topk;
    CHECK(check_buffers({{"pos", pos, n, 1, 1, 4, false},
                         {"weights", weights, n, 1, 1, 4, false},
                         {"dY", dY, tokens, cols, lddy, 2, false},
                         {"Ys", Ys, rows, cols, ldys, 2, false},
                         {"dYs", dYs, rows, cols, lddys, 2, true},
                         {"dw", dw, n, 1, 1, 4, true}}));
    if (tokens == 0)
        return ok();
    CHECK(check_gfx950());
    RowsArgs r{};
    r.tokens = tokens;
    r.topk = topk;
    r.cols = cols;
    r.rows = rows;
    r.pos = pos;
    r.weights = weights;
    r.in = dY;
    r.ld_in = lddy;
    r.in2 = Ys;
    r.ld_in2 = ldys;
    r.out = dYs;
    r.ld_out = lddys;
    r.dw = dw;
    r.bf16 = type == GEMM_BF16;
    return launched(launch_combine_backward(r, (hipStream_t)stream));
}

// ---------------------------------------------------------------- grouped products

static bool normalise(gemm_grouped_desc_t &d)
{
    const bool w = d.mode == GEMM_GROUPED_WEIGHTS;
    const int64_t b_min = !w && d.b_layout == GEMM_COL_MAJOR ? d.K : d.N;
    auto fix = [](int64_t &ld, int64_t mn) {
        if (ld == 0)
            ld = mn > 0 ? mn : 1;
        return ld >= mn && ld > 0;
    };
    const bool oka = fix(d.lda, d.K), okb = fix(d.ldb, b_min), okd = fix(d.ldd, d.N);
    return oka && okb && okd;
}

gemm_status_t gemm_grouped_validate_desc(const gemm_grouped_desc_t *desc)
{
    if (!desc)
        return fail(GEMM_ERR_NULL_POINTER, "desc is NULL");
    gemm_grouped_desc_t d = *desc;
    if (d.mode != GEMM_GROUPED_ROWS && d.mode != GEMM_GROUPED_WEIGHTS)
        return fail(GEMM_ERR_INVALID_VALUE, "unknown mode");
    const bool w = d.mode == GEMM_GROUPED_WEIGHTS;
    if (d.rows < 0 || d.N < 0 || d.K < 0 || d.rows > INT32_MAX || d.N > INT32_MAX ||
        d.K > INT32_MAX)
        return fail(GEMM_ERR_INVALID_VALUE, "rows, N and K must be in 0 .. 2^31 - 1");
    if (d.groups < 1 || d.groups > 65535)
        return fail(GEMM_ERR_INVALID_VALUE, "groups must be in 1 .. 65535");
    auto dtype_ok = [](int t) { return t >= GEMM_F16 && t <= GEMM_U8; };
    if (!dtype_ok(d.a_type) || !dtype_ok(d.b_type) || !dtype_ok(d.d_type))
        return fail(GEMM_ERR_INVALID_VALUE, "unknown dtype code");
    if (d.b_layout != GEMM_ROW_MAJOR && d.b_layout != GEMM_COL_MAJOR)
        return fail(GEMM_ERR_INVALID_VALUE, "unknown layout code");
    if (d.has_c != 0 && d.has_c != 1)
        return fail(GEMM_ERR_INVALID_VALUE, "has_c must be 0 or 1");
    if (d.algo < GEMM_ALGO_AUTO || d.algo > GEMM_ALGO_TILED_256)
        return fail(GEMM_ERR_INVALID_VALUE, "unknown algo code");
    if (d.lda < 0 || d.ldb < 0 || d.ldd < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "negative leading dimension");
    if (d.lda > MAX_ELEMS || d.ldb > MAX_ELEMS || d.ldd > MAX_ELEMS)
        return fail(GEMM_ERR_INVALID_VALUE, "leading dimension above 2^40");
    if (!normalise(d))
        return fail(GEMM_ERR_INVALID_VALUE, "leading dimension smaller than the matrix extent");
    const int64_t b_rows = w ? d.rows
                             : smul(d.groups, d.b_layout == GEMM_COL_MAJOR ? d.N : d.K);
    const int64_t d_rows = w ? smul(d.groups, d.K) : d.rows;
    if (smul(d.rows, d.lda) > MAX_ELEMS || smul(b_rows, d.ldb) > MAX_ELEMS ||
        smul(d_rows, d.ldd) > MAX_ELEMS)
        return fail(GEMM_ERR_INVALID_VALUE, "a matrix spans more than 2^40 elements");
    if (!is_16bit(d.a_type))
        return fail(GEMM_ERR_UNSUPPORTED, "A must be f16 or bf16");
    if (d.d_type != GEMM_F32 && !is_16bit(d.d_type))
        return fail(GEMM_ERR_UNSUPPORTED, "D must be f32, f16 or bf16");
    if (d.b_type != d.a_type && !(w && d.b_type == GEMM_F8_E4M3))
        return fail(GEMM_ERR_UNSUPPORTED,
                    "B must have A's type (or, for the weights' product, be e4m3 codes)");
    if (d.b_type == GEMM_F8_E4M3 && d.ldb != (d.N > 0 ? d.N : 1))
        return fail(GEMM_ERR_UNSUPPORTED, "8-bit B must be packed (ldb == N)");
    if (!w && d.has_c)
        return fail(GEMM_ERR_UNSUPPORTED, "C applies to the weights' product only");
    if (w && d.b_layout != GEMM_ROW_MAJOR)
        return fail(GEMM_ERR_UNSUPPORTED, "the weights' product takes a row-major B");
    // one launch holds 2^32 - 1 threads: below 2^23 64 x 64 tiles every kernel's
    // grid fits (the skinny one's narrower strips are checked by the plan)
    const int64_t tiles = w ? smul(smul(ceil_div(d.K, 64), ceil_div(d.N, 64)), d.groups)
                            : smul(ceil_div(d.rows, 64) + (d.groups < d.rows ? d.groups : d.rows),
                                   ceil_div(d.N, 64));
    if (tiles >= (1 << 23))
        return fail(GEMM_ERR_UNSUPPORTED, "more output tiles than one launch holds");
    return ok();
}

// Can the LDS-tiled kernels serve this descriptor (ignoring pointer
// alignment)?  They move 16-byte chunks: along K of a K-contiguous operand,
// along N (K for A) of an MN-major one; offsets inside a tile's rows take
// 32 bits.
static bool grouped_tiled_ok(const gemm_grouped_desc_t &d)
{
    const bool w = d.mode == GEMM_GROUPED_WEIGHTS;
    const bool b_mn = w || d.b_layout == GEMM_ROW_MAJOR;
    const int64_t lim = (int64_t)1 << 21; // 256 rows of 2-byte elements below 2^30
    return d.K % 8 == 0 && d.lda % 8 == 0 && d.ldb % 8 == 0 && (!b_mn || d.N % 8 == 0) &&
           d.lda < lim && d.ldb < lim;
}

// The family for a descriptor the tiled kernels take, from its sizes alone
// (the plan cannot see the groups' bounds; every family serves groups of any
// length).  Times are us on MI355X.
static int choose_family(const gemm_grouped_desc_t &d, int num_cu)
{
    if (d.mode == GEMM_GROUPED_WEIGHTS) {
        // With few tiles a tile's way through the rows is the time, which
        // smaller tiles shorten: 4 groups of 3400 rows, 704 x 480, 34 with 64,
        // 68 with 128; 2048 x 1024, 65 and 59.  Two workgroups of 64 x 64 tiles
        // (64 KB of LDS) run on a compute unit at once, and yet the border is
        // three tiles per compute unit: over drawn shapes (some 90 to each
        // quarter, 16-bit / 8-bit B) 64's time over 128's is, as a geometric
        // mean, 0.79 / 0.79 from 1.5 to 2 tiles per compute unit, 0.90 / 0.93,
        // 0.97 / 0.95, 1.00 / 0.99, 0.99 / 1.01 in the quarters from 2 to 3, 1.02 /
        // 1.05 from 3 to 3.5 and 1.06 / 1.17 from 4 to 6.  The same for 128
        // against 256: 4 groups of 2048 rows, 2048 x 1024, 57 and 75; 3 of
        // 1200, 5904 x 448, 67 and 85; 2048 x 4096, 199 and 144; drawn shapes 0.66 /
        // 0.64 from 1.5 to 2, 0.77-0.83 / 0.71-0.77 from 2 to 3.
        const int64_t t64 = d.groups * ceil_div(d.K, 64) * ceil_div(d.N, 64);
        const int64_t t128 = d.groups * ceil_div(d.K, 128) * ceil_div(d.N, 128);
        const int64_t t256 = d.groups * ceil_div(d.K, 256) * ceil_div(d.N, 256);
        if (t64 <= 3 * num_cu)
            return GF_TILED_64;
        // (Where K or N ends in the first half of a 128 and has few, 64 wastes
        // less: 8 groups of 1320 rows, 1032 x 264, 31 and 51.)
        if (t128 <= 3 * num_cu)
            return t64 * 10 <= t128 * 24 ? GF_TILED_64 : GF_TILED_128;
        // Many tiles: 256 moves less per product, 128 wastes less at the
        // edges and, two to a compute unit, hides its stores better, which
        // counts where the groups are short: 40 groups of 365 rows, 2136 x
        // 384, 116 and 92; 11 of 285, 2952 x 1352, 78 and 67; 17 groups of 36
        // rows, 488 x 3720, 50 and 47 (16 of 62 rows, 4096 x 2048, whole cache
        // lines: 196 and 254); 3 groups of 1400, 6400 x 1240, 110 and 137.
        const bool lines = d.ldd * (d.d_type == GEMM_F32 ? 4 : 2) % 128 == 0;
        return (lines || d.rows >= 256 * (int64_t)d.groups) && t256 * 33 <= t128 * 10
                   ? GF_TILED_256
                   : GF_TILED_128; // at most 6/5 of the area
    }
    // Rows: groups that can have rows, and the row tiles expected of them
    // (each wastes half a tile).
    const int64_t g = d.groups < d.rows ? d.groups : d.rows;
    auto expect = [&](int64_t b) { return (d.rows / b + (g + 1) / 2) * ceil_div(d.N, b); };
    // Few tiles: time is one workgroup's way through K.  Up to 16 rows per
    // group and 64 tiles the skinny kernel, whose waves split K (4 groups, 1024
    // x 2048: 4 rows 6.0 against 9.6, 16 rows 7.2 and 9.7, 64 rows 9.7 and 9.8;
    // 38 groups, 272 x 288, 3.9 and 4.9; past those its strips of 32 columns no
    // longer run at once: 6 groups, 2520 x 264, 11.1 and 5.0), else 64 x 64
    // tiles (367 rows, 352 x 4880, 24 against 45 with 128; 6 groups of 324,
    // 1072 x 1616, 26 and 25).
    if (expect(64) <= 2 * num_cu)
        return d.rows <= 16 * g && expect(64) * 4 <= num_cu ? GF_SKINNY : GF_TILED_64;
    // Few rows per group: bound by B's stream.  32 groups, 4096 x 2048, with
    // 64 / 128 / 256: 4 rows each 109 / 123 / 122, 16 rows 114 / 125 / 132, 32
    // rows 131 / 132 / 135; row-major B, read in runs of a tile's width: 2
    // rows 84 / 89 / 88, 4 rows 110 / 109 / 99, 16 rows 131 / 138 / 108, but
    // only while the last round of 256-wide tiles is mostly full: 27 groups of
    // 16 rows, K 4096, N 2048 (216 tiles) 95 / 99 / 86, N 2816 (297) 125 / 137
    // / 154, N 1048 (135) 58 / 55 / 74.
    if (d.rows < 32 * g) {
        const int64_t t = g * ceil_div(d.N, 256);
        return d.b_layout == GEMM_ROW_MAJOR && d.rows >= 4 * g &&
                       t * 5 >= ceil_div(t, num_cu) * num_cu * 4
                   ? GF_TILED_256
                   : GF_TILED_64;
    }
    // 8 groups of 256 rows, 2048 x 1024, 19 with 128 and 20 with 256, x 4096
    // 77 and 67; 15 groups of 208, 1504 x 408, 15 and 17; 8 of 1024, 2048 x
    // 1024, 52 and 47; 4 of 800, 2472 x 136, 15 and 18.
    return expect(128) <= (d.K <= 512 ? 3 : 1) * (int64_t)num_cu ? GF_TILED_128 : GF_TILED_256;
}

static const char *grouped_family_name(int f)
{
    static const char *const n[GF_COUNT] = {"generic", "skinny", "tiled64", "tiled128",
                                             "tiled256"};
    return n[f];
}

gemm_status_t gemm_grouped_plan(const gemm_grouped_desc_t *desc, gemm_grouped_plan_t **out)
{
    if (!out)
        return fail(GEMM_ERR_NULL_POINTER, "out is NULL");
    *out = nullptr;
    CHECK(gemm_grouped_validate_desc(desc));
    gemm_grouped_desc_t d = *desc;
    normalise(d);
    int dev = 0;
    DeviceInfo di;
    CHECK(check_device(&dev, &di));
    const bool tiled = grouped_tiled_ok(d);
    // (can serve; strips of 32 columns, 512 threads each)
    const bool skinny =
        tiled && d.mode == GEMM_GROUPED_ROWS &&
        smul(ceil_div(d.rows, 64) + (d.groups < d.rows ? d.groups : d.rows), ceil_div(d.N, 32)) <
            (1 << 22);
    const int auto_fam = tiled ? choose_family(d, di.num_cu) : GF_GENERIC;
    const int auto_tiled = auto_fam == GF_SKINNY ? GF_TILED_64 : auto_fam;
    int fam = -1;
    switch (d.algo) {
    case GEMM_ALGO_AUTO: fam = auto_fam; break;
    case GEMM_ALGO_SKINNY: fam = skinny ? GF_SKINNY : -1; break;
    case GEMM_ALGO_GENERIC: fam = GF_GENERIC; break;
    case GEMM_ALGO_TILED: fam = tiled ? auto_tiled : -1; break;
    case GEMM_ALGO_TILED_128: fam = tiled ? GF_TILED_128 : -1; break;
    case GEMM_ALGO_TILED_256: fam = tiled ? GF_TILED_256 : -1; break;
    default: fam = -1;
    }
    // Tuning override, as in gemm_plan: STGEMM_FORCE_KERNEL=<family name>
    // replaces the choice for descriptors that family can serve.
    if (const char *force = getenv("STGEMM_FORCE_KERNEL"))
        for (int f = 0; f < GF_COUNT; ++f)
            if (strcmp(force, grouped_family_name(f)) == 0 &&
                (f == GF_GENERIC || (f == GF_SKINNY ? skinny : tiled)))
                fam = f;
    if (fam < 0)
        return fail(GEMM_ERR_UNSUPPORTED, "requested algorithm cannot serve this problem");
    gemm_grouped_plan_t *p = new (std::nothrow) gemm_grouped_plan_t();
    if (!p)
        return fail(GEMM_ERR_INVALID_VALUE, "out of host memory");
    p->d = d;
    p->device = dev;
    p->num_cu = di.num_cu;
    p->family = fam;
    snprintf(p->name, sizeof p->name, "grouped_%s_%s_%s%s%s",
             d.mode == GEMM_GROUPED_WEIGHTS ? "weights" : "rows", grouped_family_name(fam),
             d.a_type == GEMM_BF16 ? "bf16" : "f16", d.b_type == GEMM_F8_E4M3 ? "xe4m3" : "",
             d.mode == GEMM_GROUPED_ROWS && d.b_layout == GEMM_ROW_MAJOR ? "_brow" : "");
    static const bool log = [] {
        const char *v = getenv("GEMM_LOG");
        return v && *v && strcmp(v, "0") != 0;
    }();
    if (log)
        fprintf(stderr, "[stgemm] grouped plan rows=%lld N=%lld K=%lld groups=%d -> %s\n",
                (long long)d.rows, (long long)d.N, (long long)d.K, d.groups, p->name);
    *out = p;
    return ok();
}

gemm_status_t gemm_grouped_plan_destroy(gemm_grouped_plan_t *plan)
{
    delete plan;
    return ok();
}

gemm_status_t gemm_grouped_plan_describe(const gemm_grouped_plan_t *plan, char *buf, size_t len)
{
    if (!plan || !buf)
        return fail(GEMM_ERR_NULL_POINTER, "plan or buf is NULL");
    if (len == 0)
        return fail(GEMM_ERR_INVALID_VALUE, "len is 0");
    snprintf(buf, len, "%s", plan->name);
    return ok();
}

gemm_status_t gemm_grouped_run(const gemm_grouped_plan_t *plan, const void *A, const void *B,
                               const uint8_t *scales, const int32_t *offsets, const void *C,
                               void *D, gemm_stream_t stream)
{
    if (!plan)
        return fail(GEMM_ERR_NULL_POINTER, "plan is NULL");
    const gemm_grouped_desc_t &d = plan->d;
    const bool w = d.mode == GEMM_GROUPED_WEIGHTS, q8 = d.b_type == GEMM_F8_E4M3;
    const int64_t m = w ? d.K : d.rows;
    if (m == 0 || d.N == 0)
        return ok();
    const int64_t db = d.d_type == GEMM_F32 ? 4 : 2;
    const int64_t d_rows = w ? (int64_t)d.groups * d.K : d.rows;
    const int64_t b_cols = !w && d.b_layout == GEMM_COL_MAJOR ? d.K : d.N;
    const int64_t b_rows = w ? d.rows
                             : (int64_t)d.groups * (d.b_layout == GEMM_COL_MAJOR ? d.N : d.K);
    // C shares D's leading dimension: C == D (every element read before it is
    // written, by the same lane) is fine, any other overlap is not
    const bool in_place = d.has_c && C == D;
    if (d.has_c && !C)
        return fail(GEMM_ERR_NULL_POINTER, "C is NULL but the plan reads C");
    CHECK(check_buffers({{"A", A, d.rows, d.K, d.lda, 2, false},
                         {"B", B, b_rows, b_cols, d.ldb, q8 ? 1 : 2, false},
                         {"scales", scales, q8 ? d.rows : 0, ceil_div(d.N, 32), ceil_div(d.N, 32),
                          1, false},
                         {"offsets", offsets, d.groups + 1, 1, 1, 4, false},
                         {"C", C, d.has_c && !in_place ? d_rows : 0, d.N, d.ldd, db, false},
                         {"D", D, d_rows, d.N, d.ldd, db, true}}));
    GroupedArgs a{};
    a.weights_mode = w;
    a.groups = d.groups;
    a.rows = d.rows;
    a.N = d.N;
    a.K = d.K;
    a.A = A;
    a.B = B;
    a.bs = q8 ? scales : nullptr;
    a.offsets = offsets;
    a.C = d.has_c ? C : nullptr;
    a.D = D;
    a.lda = d.lda;
    a.ldb = d.ldb;
    a.ldd = d.ldd;
    a.b_row = d.b_layout == GEMM_ROW_MAJOR;
    a.bf16 = d.a_type == GEMM_BF16;
    a.d_kind = d.d_type == GEMM_F32 ? OUT_F32 : d.d_type == GEMM_F16 ? OUT_F16 : OUT_BF16;
    // the vector epilogue addresses 257 rows of C and D with 32-bit offsets
    a.num_cu = plan->num_cu;
    a.vec = (!d.has_c || aligned(C, 4 * (size_t)db)) && aligned(D, 4 * (size_t)db) &&
            d.ldd % 4 == 0 && d.ldd * db < 0x7fffffff / 257;
    a.whole_lines = aligned(D, 128) && (d.ldd * db) % 128 == 0;
    int fam = plan->family;
    if (fam != GF_GENERIC && (!aligned(A, 16) || !aligned(B, 16)))
        fam = GF_GENERIC;
    return launched(launch_grouped(fam, a, (hipStream_t)stream));
}

// ---------------------------------------------------------------- 8-bit checkpoints

// The sizes of a checkpointed rows x cols tensor.
static gemm_status_t check_q8(int64_t rows, int64_t cols, int32_t type)
{
    CHECK(check_rows_type(cols, type));
    if (rows < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "negative number of rows");
    if (smul(rows, cols) > MAX_ELEMS)
        return fail(GEMM_ERR_INVALID_VALUE, "a matrix spans more than 2^40 elements");
    return GEMM_OK;
}

gemm_status_t gemm_q8_store(int64_t rows, int64_t cols, int32_t type, const void *X, int64_t ldx,
                            uint8_t *codes, uint8_t *scales, gemm_stream_t stream)
{
    CHECK(check_q8(rows, cols, type));
    CHECK(check_matrix("X", rows, cols, &ldx));
    const int64_t nb = ceil_div(cols, 32);
    CHECK(check_buffers({{"X", X, rows, cols, ldx, 2, false},
                         {"codes", codes, rows, cols, cols, 1, true},
                         {"scales", scales, rows, nb, nb, 1, true}}));
    if (rows == 0 || cols == 0)
        return ok();
    CHECK(check_gfx950());
    Q8Args a{};
    a.rows = rows;
    a.cols = cols;
    a.bf16 = type == GEMM_BF16;
    a.x = X;
    a.ldx = ldx;
    a.codes = codes;
    a.scales = scales;
    return launched(launch_q8_store(a, (hipStream_t)stream));
}

gemm_status_t gemm_q8_load(int64_t rows, int64_t cols, int32_t type, const uint8_t *codes,
                           const uint8_t *scales, void *X, int64_t ldx, gemm_stream_t stream)
{
    CHECK(check_q8(rows, cols, type));
    CHECK(check_matrix("X", rows, cols, &ldx));
    const int64_t nb = ceil_div(cols, 32);
    CHECK(check_buffers({{"codes", codes, rows, cols, cols, 1, false},
                         {"scales", scales, rows, nb, nb, 1, false},
                         {"X", X, rows, cols, ldx, 2, true}}));
    if (rows == 0 || cols == 0)
        return ok();
    CHECK(check_gfx950());
    Q8Args a{};
    a.rows = rows;
    a.cols = cols;
    a.bf16 = type == GEMM_BF16;
    a.codes = const_cast<uint8_t *>(codes);
    a.scales = const_cast<uint8_t *>(scales);
    a.out = X;
    a.ldo = ldx;
    return launched(launch_q8_load(a, (hipStream_t)stream));
}

gemm_status_t gemm_swiglu(int64_t rows, int64_t cols, int32_t type, const void *GU, int64_t ldgu,
                          void *H, int64_t ldh, uint8_t *codes, uint8_t *scales,
                          gemm_stream_t stream)
{
    CHECK(check_q8(rows, cols, type));
    CHECK(check_matrix("GU", rows, 2 * cols, &ldgu));
    CHECK(check_matrix("H", rows, cols, &ldh));
    const int64_t nb = ceil_div(2 * cols, 32), keep = codes || scales ? rows : 0;
    CHECK(check_buffers({{"GU", GU, rows, 2 * cols, ldgu, 2, false},
                         {"H", H, rows, cols, ldh, 2, true},
                         {"codes", codes, keep, 2 * cols, 2 * cols, 1, true},
                         {"scales", scales, keep, nb, nb, 1, true}}));
    if (rows == 0 || cols == 0)
        return ok();
    CHECK(check_gfx950());
    Q8Args a{};
    a.rows = rows;
    a.cols = 2 * cols;
    a.bf16 = type == GEMM_BF16;
    a.x = GU;
    a.ldx = ldgu;
    a.codes = codes;
    a.scales = scales;
    a.out = H;
    a.ldo = ldh;
    return launched(launch_swiglu(a, (hipStream_t)stream));
}

gemm_status_t gemm_swiglu_backward(int64_t rows, int64_t cols, int32_t type, const uint8_t *codes,
                                   const uint8_t *scales, const void *dH, int64_t lddh, void *dGU,
                                   int64_t lddgu, void *H, int64_t ldh, gemm_stream_t stream)
{
    CHECK(check_q8(rows, cols, type));
    CHECK(check_matrix("dH", rows, cols, &lddh));
    CHECK(check_matrix("dGU", rows, 2 * cols, &lddgu));
    CHECK(check_matrix("H", rows, cols, &ldh));
    const int64_t nb = ceil_div(2 * cols, 32);
    CHECK(check_buffers({{"codes", codes, rows, 2 * cols, 2 * cols, 1, false},
                         {"scales", scales, rows, nb, nb, 1, false},
                         {"dH", dH, rows, cols, lddh, 2, false},
                         {"dGU", dGU, rows, 2 * cols, lddgu, 2, true},
                         {"H", H, H ? rows : 0, cols, ldh, 2, true}}));
    if (rows == 0 || cols == 0)
        return ok();
    CHECK(check_gfx950());
    Q8Args a{};
    a.rows = rows;
    a.cols = 2 * cols;
    a.bf16 = type == GEMM_BF16;
    a.codes = const_cast<uint8_t *>(codes);
    a.scales = const_cast<uint8_t *>(scales);
    a.x = dH;
    a.ldx = lddh;
    a.out = dGU;
    a.ldo = lddgu;
    a.out2 = H;
    a.ldo2 = ldh;
    return launched(launch_swiglu_backward(a, (hipStream_t)stream));
}

} // extern "C"

// C ABI of the operators over a vocabulary: argument checks, plan choice,
// workspace layout and launches.  The operations are documented in
// include/gemm_vocab.h.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>

#include "api_checks.hpp"
#include "gemm_vocab.h"
#include "vocab_args.hpp"

using namespace stg;

struct gemm_xent_plan {
    gemm_xent_desc_t d; // normalised: packed leading dimensions filled in
    int64_t hp;         // hidden in whole 16-byte chunks
    int copy;           // W goes through the workspace
    int loose;          // but not forward: the streaming kernel reads it where it lies
    int stats, g, dx, dw; // XentTile of each product
    int dw_tile;        // of dW where it is not aligned to 16 bytes
    int64_t piece;      // columns of a piece
    XentSplits split;   // of dX's sums, by the rows that have a target
    int64_t acc;        // fp32 values that they take
    int device;
    char name[96];
};

namespace {

bool is_float(int t) { return t == GEMM_F32 || is_16bit(t); }
int64_t float_bytes(int t) { return t == GEMM_F32 ? 4 : 2; }
int out_kind(int t) { return t == GEMM_F32 ? OUT_F32 : t == GEMM_F16 ? OUT_F16 : OUT_BF16; }

// ---------------------------------------------------------------- embedding

gemm_status_t check_embed(int64_t tokens, int64_t vocab, int64_t cols)
{
    if (tokens < 0 || vocab < 0 || cols < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "negative size");
    if (tokens > (1 << 25) || vocab > EMBED_MAX_VOCAB || cols > (1 << 23))
        return fail(GEMM_ERR_UNSUPPORTED, "at most 2^25 tokens, 2^20 rows and 2^23 columns");
    return GEMM_OK;
}

gemm_status_t check_embed_types(int32_t e_type, int32_t y_type, int32_t id_bytes)
{
    for (int32_t t : {e_type, y_type}) {
        if (t < GEMM_F16 || t > GEMM_U8)
            return fail(GEMM_ERR_INVALID_VALUE, "unknown dtype code");
        if (!is_float(t))
            return fail(GEMM_ERR_UNSUPPORTED, "types must be f32, f16 or bf16");
    }
    if (id_bytes != 4 && id_bytes != 8)
        return fail(GEMM_ERR_INVALID_VALUE, "id_bytes must be 4 or 8");
    return GEMM_OK;
}

// Hands out 256-byte aligned parts of a workspace, or counts their bytes.
struct Parts {
    uint8_t *base;
    size_t at = 0;
    template <class T>
    void take(T *&p, int64_t n)
    {
        p = base ? (T *)(base + at) : nullptr;
        at += ((size_t)n * sizeof(T) + 255) / 256 * 256;
    }
};

// The sort's sizes and the workspace of the gradient.  It depends on the number of
// tokens alone whether there is one, also where the kernels group up to 2048
// tokens without it (embed_small).
size_t embed_parts(EmbedArgs &a, void *workspace)
{
    if (a.tokens <= EMBED_SMALL)
        return 0;
    int bits = 1;
    while (((int64_t)1 << bits) < a.vocab)
        ++bits;
    a.hi_bits = bits / 2;
    a.lo_bits = bits - a.hi_bits;
    const int64_t c = ceil_div(a.tokens, 256);
    a.chunk = (int)(c <= 1024 ? 1024 : ceil_div(c, 512) * 512); // eight waves, 64 at a time
    a.chunks = (int)ceil_div(a.tokens, a.chunk);
    Parts p{(uint8_t *)workspace};
    p.take(a.counts, (int64_t)a.chunks << a.lo_bits);
    p.take(a.bounds, ((int64_t)1 << a.lo_bits) + 1);
    p.take(a.binned, a.tokens);
    p.take(a.order, a.tokens);
    p.take(a.key, a.tokens);
    p.take(a.part, ceil_div(a.tokens, EMBED_RUN) * 2 * a.cols);
    return p.at;
}

} // namespace

extern "C" {

gemm_status_t gemm_embed(int64_t tokens, int64_t vocab, int64_t cols, int32_t e_type,
                         int32_t y_type, int32_t id_bytes, const void *ids, const void *E,
                         int64_t lde, void *Y, int64_t ldy, float scale, gemm_stream_t stream)
{
    CHECK(check_embed(tokens, vocab, cols));
    CHECK(check_embed_types(e_type, y_type, id_bytes));
    CHECK(check_matrix("E", vocab, cols, &lde));
    CHECK(check_matrix("Y", tokens, cols, &ldy));
    CHECK(check_buffers({{"ids", ids, tokens, 1, 1, id_bytes, false},
                         {"E", E, vocab, cols, lde, float_bytes(e_type), false},
                         {"Y", Y, tokens, cols, ldy, float_bytes(y_type), true}}));
    if (tokens == 0 || cols == 0)
        return ok();
    CHECK(check_gfx950());
    EmbedArgs a{};
    a.tokens = tokens;
    a.vocab = vocab;
    a.cols = cols;
    a.id8 = id_bytes == 8;
    a.ids = ids;
    a.e_kind = out_kind(e_type);
    a.y_kind = out_kind(y_type);
    a.in = E;
    a.ld_in = lde;
    a.out = Y;
    a.ld_out = ldy;
    a.scale = scale;
    return launched(launch_embed(a, (hipStream_t)stream));
}

gemm_status_t gemm_embed_workspace(int64_t tokens, int64_t vocab, int64_t cols, size_t *bytes)
{
    if (!bytes)
        return fail(GEMM_ERR_NULL_POINTER, "bytes is NULL");
    CHECK(check_embed(tokens, vocab, cols));
    EmbedArgs a{};
    a.tokens = tokens;
    a.vocab = vocab;
    a.cols = cols;
    *bytes = embed_parts(a, nullptr);
    return ok();
}

gemm_status_t gemm_embed_backward(int64_t tokens, int64_t vocab, int64_t cols, int32_t y_type,
                                  int32_t e_type, int32_t id_bytes, const void *ids,
                                  const void *dY, int64_t lddy, void *dE, int64_t ldde,
                                  int32_t accumulate, void *workspace, float scale,
                                  gemm_stream_t stream)
{
    CHECK(check_embed(tokens, vocab, cols));
    CHECK(check_embed_types(e_type, y_type, id_bytes));
    if (accumulate != 0 && accumulate != 1)
        return fail(GEMM_ERR_INVALID_VALUE, "accumulate must be 0 or 1");
    CHECK(check_matrix("dY", tokens, cols, &lddy));
    CHECK(check_matrix("dE", vocab, cols, &ldde));
    EmbedArgs a{};
    a.tokens = tokens;
    a.vocab = vocab;
    a.cols = cols;
    const int64_t bytes = (int64_t)embed_parts(a, workspace);
    CHECK(check_buffers({{"ids", ids, tokens, 1, 1, id_bytes, false},
                         {"dY", dY, tokens, cols, lddy, float_bytes(y_type), false},
                         {"dE", dE, vocab, cols, ldde, float_bytes(e_type), true},
                         {"workspace", workspace, bytes, 1, 1, 1, true, 16}}));
    if (vocab == 0 || cols == 0 || (tokens == 0 && accumulate))
        return ok();
    CHECK(check_gfx950());
    a.id8 = id_bytes == 8;
    a.ids = ids;
    a.e_kind = out_kind(e_type);
    a.y_kind = out_kind(y_type);
    a.in = dY;
    a.ld_in = lddy;
    a.out = dE;
    a.ld_out = ldde;
    a.scale = scale;
    a.accumulate = accumulate;
    return launched(launch_embed_backward(a, (hipStream_t)stream));
}

// ---------------------------------------------------------------- linear cross entropy

static bool normalise(gemm_xent_desc_t &d)
{
    auto fix = [&](int64_t &ld) {
        if (ld == 0)
            ld = d.hidden;
        return ld >= d.hidden;
    };
    const bool x = fix(d.ldx), w = fix(d.ldw), dx = fix(d.lddx), dw = fix(d.lddw);
    return x && w && dx && dw;
}

gemm_status_t gemm_xent_validate_desc(const gemm_xent_desc_t *desc)
{
    if (!desc)
        return fail(GEMM_ERR_NULL_POINTER, "desc is NULL");
    gemm_xent_desc_t d = *desc;
    if (d.tokens < 0 || d.vocab < 1 || d.hidden < 1)
        return fail(GEMM_ERR_INVALID_VALUE, "tokens must be >= 0, vocab and hidden >= 1");
    auto dtype_ok = [](int t) { return t >= GEMM_F16 && t <= GEMM_U8; };
    if (!dtype_ok(d.x_type) || !dtype_ok(d.dx_type) || !dtype_ok(d.dw_type))
        return fail(GEMM_ERR_INVALID_VALUE, "unknown dtype code");
    if (d.id_bytes != 4 && d.id_bytes != 8)
        return fail(GEMM_ERR_INVALID_VALUE, "id_bytes must be 4 or 8");
    if ((d.accumulate != 0 && d.accumulate != 1) || (d.unaligned != 0 && d.unaligned != 1))
        return fail(GEMM_ERR_INVALID_VALUE, "accumulate and unaligned must be 0 or 1");
    if (d.ldx < 0 || d.ldw < 0 || d.lddx < 0 || d.lddw < 0 || d.piece < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "negative leading dimension or piece");
    if (!normalise(d))
        return fail(GEMM_ERR_INVALID_VALUE, "leading dimension smaller than the matrix extent");
    for (int64_t ld : {d.ldx, d.ldw, d.lddx, d.lddw})
        if (ld > MAX_ELEMS || smul(d.tokens > d.vocab ? d.tokens : d.vocab, ld) > MAX_ELEMS)
            return fail(GEMM_ERR_INVALID_VALUE, "a matrix spans more than 2^40 elements");
    if (d.tokens > (1 << 20) || d.vocab > (1 << 24) || d.hidden > (1 << 15))
        return fail(GEMM_ERR_UNSUPPORTED, "at most 2^20 tokens, 2^24 columns and 2^15 hidden values");
    if (!is_16bit(d.x_type))
        return fail(GEMM_ERR_UNSUPPORTED, "X must be f16 or bf16");
    if (!is_float(d.dx_type) || !is_float(d.dw_type))
        return fail(GEMM_ERR_UNSUPPORTED, "dX and dW must be f32, f16 or bf16");
    // (2^31 threads in 256 x 256 tiles)
    if (smul(ceil_div(d.tokens, 256), ceil_div(d.vocab, 256)) > (1 << 20))
        return fail(GEMM_ERR_UNSUPPORTED, "more logits than one launch holds");
    return ok();
}

static int64_t tiles(int t, int64_t m, int64_t n)
{
    return ceil_div(m, xent_edge(t)) * ceil_div(n, xent_edge(t));
}

// What a product of m x n outputs and a sum of k takes in a tile's rounds of
// workgroups, us: a 64-value step of the sum and the rest of a tile's way (its
// first operands, its epilogue), with one workgroup of 256 x 256 on a compute
// unit and two of the others.  Fitted on the measured kernels, for their order: it
// is within some 25 % of most, and 40 to 65 % above where few tiles have a long
// sum (the last one here).  265 tokens, 19890 x 840, dW 32 / 31 / 54 us for
// 256 / 128 / 64 (measured 38, 31, 44); 3 tokens, 172148 x 72, 31 / 21 (41, 25);
// 137, 32408 x 7096, 186 / 243 (220, 249); logits of 260, 58186 x 88, 24 / 23 /
// 43 (26, 24, 35); 442, 90142 x 456, 62 / 79 (63, 77); 556, 1379 x 7920, 189 /
// 118 / 54 (129, 72, 38).
static double tile_time(int t, int64_t m, int64_t n, int64_t k, int64_t parts, int num_cu)
{
    static const double step[XT_COUNT] = {0.4, 0.9, 1.45}, rest[XT_COUNT] = {4, 6, 9};
    const int64_t slots = t == XT_256 ? num_cu : 2 * num_cu;
    return (double)ceil_div(tiles(t, m, n) * parts, slots) *
           ((double)ceil_div(ceil_div(k, parts), 64) * step[t] + rest[t]);
}

static int best_tile(int64_t m, int64_t n, int64_t k, int num_cu)
{
    int best = XT_64;
    for (int t = XT_128; t < XT_COUNT; ++t)
        if (tile_time(t, m, n, k, 1, num_cu) < tile_time(best, m, n, k, 1, num_cu))
            best = t;
    return best;
}

// Tile of the logits' product of `n` columns.  Up to 16 rows the streaming
// kernel, but 64 x 64 tiles for long rows of a W of 512 MB and more: 1 row,
// 131072 x 4096, 183 us and 166; 16 rows 204 and 168; 16, 65536 x 4096, 104 and
// 100; 4, 32768 x 8192, 100 and 104; 10, 50021 x 1416, 38 and 37; 9, 200000 x
// 512, 39 and 49; 1, 32768 x 2048, 25 and 32.
static int choose_logits(int64_t tokens, int64_t n, int64_t hp, int num_cu)
{
    if (tokens <= XENT_STREAM_ROWS)
        return hp >= 2048 && n * hp >= (1 << 28) ? XT_64 : XT_STREAM;
    return tokens <= 64 ? XT_64 : best_tile(tokens, n, hp, num_cu);
}

// Parts of dX's sum over `cols` columns that any number of rows may choose:
// 1024 columns each at least, 128 (which k_xent_out adds up) and four rounds of
// workgroups at most.
static XentSplits dx_split(int tile, int64_t hp, int64_t cols, int num_cu)
{
    const int e = xent_edge(tile), slots = tile == XT_256 ? num_cu : 2 * num_cu;
    const int tiles_n = (int)ceil_div(hp, e);
    int64_t most = ceil_div(cols, 1024);
    most = most < 4 * slots / tiles_n ? most : 4 * slots / tiles_n;
    most = most < 128 ? most : 128;
    return {e, tiles_n, (int)cols, slots, most < 1 ? 1 : (int)most, 0, num_cu};
}

static int choose_dx(int64_t tokens, int64_t hp, int64_t cols, int num_cu)
{
    int best = XT_64;
    double least = 0;
    for (int t = XT_64; t < XT_COUNT; ++t) {
        const XentSplits x = dx_split(t, hp, cols, num_cu);
        const int s = xent_splits((int)tokens, x.edge, x.tiles_n, x.cols, x.slots, x.most);
        // (each part is written and read again, at 5 TB/s)
        const double us =
            tile_time(t, tokens, hp, cols, s, num_cu) + 8e-6 / 5 * (double)(s * tokens * hp);
        if (t == XT_64 || us < least) {
            best = t;
            least = us;
        }
    }
    return best;
}

static void choose(gemm_xent_plan_t &p, int num_cu)
{
    const gemm_xent_desc_t &d = p.d;
    p.hp = ceil_div(d.hidden, 8) * 8;
    // the main loop addresses 256 rows of W with 32-bit offsets
    p.copy = d.hidden % 8 != 0 || d.ldw % 8 != 0 || d.ldw >= (1 << 21) || d.unaligned;
    // G of a piece: 512 MB, W's copy too
    int64_t width = ((int64_t)1 << 28) / (d.tokens > 0 ? d.tokens : 1);
    if (p.copy && width > ((int64_t)1 << 28) / p.hp)
        width = ((int64_t)1 << 28) / p.hp;
    if (width > (1 << 20))
        width = 1 << 20;
    width = width < 2048 ? 2048 : width / 256 * 256;
    if (d.piece > 0)
        width = d.piece > (1 << 20) ? 1 << 20 : ceil_div(d.piece, 256) * 256;
    const int64_t n = ceil_div(d.vocab, width);
    p.piece = ceil_div(ceil_div(d.vocab, n), 256) * 256;
    const int64_t cols = d.vocab < p.piece ? d.vocab : p.piece;
    p.stats = choose_logits(d.tokens, p.copy ? cols : d.vocab, p.hp, num_cu);
    if (p.copy && d.tokens <= XENT_STREAM_ROWS) // (no copy of W: see loose)
        p.stats = XT_STREAM;
    p.g = choose_logits(d.tokens, cols, p.hp, num_cu);
    p.dw = p.dw_tile = best_tile(cols, p.hp, d.tokens, num_cu);
    const int64_t dw_row = d.lddw * float_bytes(d.dw_type);
    if (d.tokens > 0 && d.tokens <= XENT_DW_ROWS && d.hidden % 8 == 0 && dw_row % 16 == 0)
        p.dw = XT_STREAM;
    p.dx = choose_dx(d.tokens, p.hp, cols, num_cu);
    if (const char *force = getenv("STGEMM_FORCE_KERNEL")) {
        static const char *const names[XT_COUNT] = {"tiled64", "tiled128", "tiled256"};
        for (int t = 0; t < XT_COUNT; ++t)
            if (strcmp(force, names[t]) == 0)
                p.stats = p.g = p.dw = p.dw_tile = p.dx = t;
    }
    p.loose = p.copy && p.stats == XT_STREAM && d.tokens <= XENT_STREAM_ROWS && d.ldw < (1 << 21);
    // dX's sums run over the piece's columns, cut where its tiles would leave
    // compute units idle.  The kernels choose by the rows that have a target;
    // here every number of them needs room.
    p.split = dx_split(p.dx, p.hp, cols, num_cu);
    const XentSplits &x = p.split;
    const int e = x.edge;
    p.acc = 0;
    for (int64_t n = 0; n < d.tokens;) {
        n = n + e < d.tokens ? n + e : d.tokens;
        const int s = xent_splits((int)n, e, x.tiles_n, x.cols, x.slots, x.most);
        const int wgs = (int)ceil_div(n, e) * x.tiles_n * s;
        p.acc = s * n * p.hp > p.acc ? s * n * p.hp : p.acc;
        p.split.wgs = wgs > p.split.wgs ? wgs : p.split.wgs;
    }
}

static bool copy_forward(const gemm_xent_plan_t &p) { return p.copy && !p.loose; }

// Maxima and sums per row that the statistics of n columns leave.
static int64_t stats_parts(const gemm_xent_plan_t &p, int64_t n)
{
    return p.stats == XT_STREAM ? xent_streams(n, p.split.num_cu) : ceil_div(n, xent_edge(p.stats));
}

// The workspace of a call: args' pointers into it, its bytes.
static size_t xent_parts(const gemm_xent_plan_t &p, bool backward, void *workspace, XentArgs &a,
                         XentPiece &piece, float *&acc, uint16_t *&copy)
{
    const gemm_xent_desc_t &d = p.d;
    Parts w{(uint8_t *)workspace};
    w.take(a.count, 2);
    w.take(a.pos, d.tokens);
    w.take(a.map, d.tokens);
    w.take(a.tgt, d.tokens);
    a.ldc = xent_pitch(d.hidden);
    w.take(a.Xc, d.tokens * a.ldc);
    if (backward) {
        w.take(a.ca, d.tokens);
        w.take(a.cb, d.tokens);
        w.take(a.cl, d.tokens);
        a.gmaxes = d.tokens > 0 ? ceil_div(d.tokens, xent_prep(d.tokens)) : 1;
        w.take(a.gmax, a.gmaxes);
        w.take(acc, p.acc);
        w.take(piece.G, d.tokens * p.piece);
        piece.ldg = p.piece;
    } else {
        const int64_t full = d.vocab / p.piece;
        a.part_tiles = copy_forward(p) ? full * stats_parts(p, p.piece) + stats_parts(p, d.vocab - full * p.piece)
                              : stats_parts(p, d.vocab);
        w.take(a.zt, d.tokens);
        w.take(a.part, a.part_tiles * d.tokens * 2);
    }
    if (backward ? p.copy : copy_forward(p))
        w.take(copy, (d.vocab < p.piece ? d.vocab : p.piece) * a.ldc);
    return w.at;
}

gemm_status_t gemm_xent_plan(const gemm_xent_desc_t *desc, gemm_xent_plan_t **out)
{
    if (!out)
        return fail(GEMM_ERR_NULL_POINTER, "out is NULL");
    *out = nullptr;
    CHECK(gemm_xent_validate_desc(desc));
    int dev = 0;
    DeviceInfo di;
    CHECK(check_device(&dev, &di));
    gemm_xent_plan_t *p = new (std::nothrow) gemm_xent_plan_t();
    if (!p)
        return fail(GEMM_ERR_INVALID_VALUE, "out of host memory");
    p->d = *desc;
    normalise(p->d);
    p->device = dev;
    choose(*p, di.num_cu);
    auto logits = [](int t) { return t == XT_STREAM ? XENT_STREAM_ROWS : xent_edge(t); };
    char dw[16] = "rows";
    if (p->dw != XT_STREAM)
        snprintf(dw, sizeof dw, "%d", xent_edge(p->dw));
    snprintf(p->name, sizeof p->name, "xent_%s_stats%d_g%d_dx%d_dw%s%s",
             p->d.x_type == GEMM_BF16 ? "bf16" : "f16", logits(p->stats), logits(p->g),
             xent_edge(p->dx), dw, p->copy ? "_copy" : "");
    static const bool log = [] {
        const char *v = getenv("GEMM_LOG");
        return v && *v && strcmp(v, "0") != 0;
    }();
    if (log)
        fprintf(stderr, "[stgemm] xent plan tokens=%lld vocab=%lld hidden=%lld piece=%lld -> %s\n",
                (long long)p->d.tokens, (long long)p->d.vocab, (long long)p->d.hidden,
                (long long)p->piece, p->name);
    *out = p;
    return ok();
}

gemm_status_t gemm_xent_plan_destroy(gemm_xent_plan_t *plan)
{
    delete plan;
    return ok();
}

gemm_status_t gemm_xent_plan_describe(const gemm_xent_plan_t *plan, char *buf, size_t len)
{
    if (!plan || !buf)
        return fail(GEMM_ERR_NULL_POINTER, "plan or buf is NULL");
    if (len == 0)
        return fail(GEMM_ERR_INVALID_VALUE, "len is 0");
    snprintf(buf, len, "%s", plan->name);
    return ok();
}

gemm_status_t gemm_xent_workspace(const gemm_xent_plan_t *plan, size_t *forward, size_t *backward)
{
    if (!plan)
        return fail(GEMM_ERR_NULL_POINTER, "plan is NULL");
    XentArgs a{};
    XentPiece p{};
    float *acc;
    uint16_t *copy;
    if (forward)
        *forward = xent_parts(*plan, false, nullptr, a, p, acc, copy);
    if (backward)
        *backward = xent_parts(*plan, true, nullptr, a, p, acc, copy);
    return ok();
}

static void fill_args(XentArgs &a, const gemm_xent_plan_t &p, const void *X, const void *targets)
{
    a.tokens = p.d.tokens;
    a.vocab = p.d.vocab;
    a.hidden = p.d.hidden;
    a.hp = p.hp;
    a.id8 = p.d.id_bytes == 8;
    a.bf16 = p.d.x_type == GEMM_BF16;
    a.X = X;
    a.ldx = p.d.ldx;
    a.targets = targets;
    a.prep = xent_prep(p.d.tokens);
    a.dx = p.split;
    a.scale = p.d.scale;
}

// A call's device, and W's alignment.
static gemm_status_t check_call(const gemm_xent_plan_t &p, const void *W)
{
    int dev = 0;
    CHECK(check_device(&dev, nullptr));
    if (dev != p.device)
        return fail(GEMM_ERR_DEVICE, "the plan was made on device %d, the current one is %d", p.device,
                    dev);
    if (!p.copy && !aligned(W, 16))
        return fail(GEMM_ERR_MISALIGNED, "W is not aligned to 16 bytes and the plan has unaligned = 0");
    return GEMM_OK;
}

// W's rows of a piece: where they lie, or copied.
static hipError_t take_w(const gemm_xent_plan_t &p, bool copies, const void *W, uint16_t *copy,
                         XentPiece &piece, hipStream_t s)
{
    const uint16_t *w = (const uint16_t *)W + piece.v0 * p.d.ldw;
    piece.W = copies ? copy : w;
    piece.ldw = copies ? xent_pitch(p.d.hidden) : p.d.ldw;
    return copies ? launch_xent_copy({w, p.d.ldw, piece.n, p.d.hidden, p.hp, copy, piece.ldw}, s)
                  : hipSuccess;
}

#define LAUNCH(x)                                 \
    do {                                          \
        const hipError_t e_ = x;                  \
        if (e_ != hipSuccess)                     \
            return hip_fail(e_, "kernel launch"); \
    } while (0)

gemm_status_t gemm_xent_forward(const gemm_xent_plan_t *plan, const void *X, const void *W,
                                const void *targets, float *loss, float *lse, void *workspace,
                                gemm_stream_t stream)
{
    if (!plan)
        return fail(GEMM_ERR_NULL_POINTER, "plan is NULL");
    const gemm_xent_desc_t &d = plan->d;
    const hipStream_t s = (hipStream_t)stream;
    XentArgs a{};
    XentPiece p{};
    float *acc;
    uint16_t *copy = nullptr;
    if (d.tokens == 0)
        return ok();
    const int64_t bytes = (int64_t)xent_parts(*plan, false, workspace, a, p, acc, copy);
    CHECK(check_buffers({{"X", X, d.tokens, d.hidden, d.ldx, 2, false},
                         {"W", W, d.vocab, d.hidden, d.ldw, 2, false},
                         {"targets", targets, d.tokens, 1, 1, d.id_bytes, false},
                         {"loss", loss, loss ? d.tokens : 0, 1, 1, 4, true},
                         {"lse", lse, d.tokens, 1, 1, 4, true},
                         {"workspace", workspace, bytes, 1, 1, 1, true, 16}}));
    CHECK(check_call(*plan, W));
    fill_args(a, *plan, X, targets);
    a.loss = loss;
    a.lse = lse;
    // (one tile of rows: nothing is gained by skipping some)
    a.direct = d.tokens <= 64 && d.hidden % 8 == 0 && d.ldx % 8 == 0 && d.ldx < (1 << 21) &&
               aligned(X, 16);
    if (!a.direct)
        LAUNCH(launch_xent_prepare(a, false, s));
    const bool copies = copy_forward(*plan);
    const int64_t step = copies ? plan->piece : d.vocab;
    p.loose = plan->loose;
    for (p.v0 = 0; p.v0 < d.vocab; p.v0 += step) {
        p.n = d.vocab - p.v0 < step ? d.vocab - p.v0 : step;
        LAUNCH(take_w(*plan, copies, W, copy, p, s));
        LAUNCH(launch_xent_stats(plan->stats, a, p, s));
        p.tile0 += stats_parts(*plan, p.n);
    }
    return launched(launch_xent_loss(a, s));
}

gemm_status_t gemm_xent_backward(const gemm_xent_plan_t *plan, const void *X, const void *W,
                                 const void *targets, const float *lse, const float *dloss,
                                 const float *dlse, void *dX, void *dW, void *workspace,
                                 gemm_stream_t stream)
{
    if (!plan)
        return fail(GEMM_ERR_NULL_POINTER, "plan is NULL");
    const gemm_xent_desc_t &d = plan->d;
    const hipStream_t s = (hipStream_t)stream;
    XentArgs a{};
    XentPiece p{};
    float *acc = nullptr;
    uint16_t *copy = nullptr;
    const int64_t t = d.tokens, bytes = (int64_t)xent_parts(*plan, true, workspace, a, p, acc, copy);
    const int64_t wb = float_bytes(d.dw_type);
    CHECK(check_buffers({{"X", X, t, d.hidden, d.ldx, 2, false},
                         {"W", W, d.vocab, d.hidden, d.ldw, 2, false},
                         {"targets", targets, t, 1, 1, d.id_bytes, false},
                         {"lse", lse, t, 1, 1, 4, false},
                         {"dloss", dloss, t, 1, 1, 4, false},
                         {"dlse", dlse, dlse ? t : 0, 1, 1, 4, false},
                         {"dX", dX, dX ? t : 0, d.hidden, d.lddx, float_bytes(d.dx_type), true},
                         {"dW", dW, dW ? d.vocab : 0, d.hidden, d.lddw, wb, true},
                         {"workspace", workspace, bytes, 1, 1, 1, true, 16}}));
    CHECK(check_call(*plan, W));
    if (!dX && !dW)
        return ok();
    fill_args(a, *plan, X, targets);
    a.lse_in = lse;
    a.dloss = dloss;
    a.dlse = dlse;
    LAUNCH(launch_xent_prepare(a, true, s));
    for (p.v0 = 0; p.v0 < d.vocab; p.v0 += plan->piece) {
        p.n = d.vocab - p.v0 < plan->piece ? d.vocab - p.v0 : plan->piece;
        LAUNCH(take_w(*plan, plan->copy, W, copy, p, s));
        if (t > 0)
            LAUNCH(launch_xent_g(plan->g, a, p, s));
        if (dX && t > 0)
            LAUNCH(launch_xent_dx(plan->dx, a, p, {acc, p.v0 > 0}, s));
        if (dW) {
            uint8_t *w = (uint8_t *)dW + p.v0 * d.lddw * wb;
            // the vector epilogue addresses 257 rows of dW with 32-bit offsets
            const int vec = aligned(w, 4 * (size_t)wb) && d.lddw % 4 == 0 &&
                            d.lddw * wb < 0x7fffffff / 257;
            const int lines = aligned(w, 128) && (d.lddw * wb) % 128 == 0;
            // (the streaming kernel stores 16 bytes at a time)
            const int tile = vec && aligned(w, 16) ? plan->dw : plan->dw_tile;
            LAUNCH(launch_xent_dw(tile, a, p,
                                  {w, d.lddw, out_kind(d.dw_type), d.accumulate, vec, lines}, s));
        }
    }
    if (dX && t > 0)
        LAUNCH(launch_xent_out(a, {acc, dX, d.lddx, out_kind(d.dx_type)}, s));
    return ok();
}

} // extern "C"

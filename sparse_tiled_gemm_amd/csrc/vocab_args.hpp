// Argument blocks and launchers of the operators over a vocabulary
// (vocab_api.cpp calls them; kernels_embed.hip and kernels_xent*.hip define
// them).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernel_args.hpp"

namespace stg {

// ---------------------------------------------------------------- embedding

constexpr int64_t EMBED_MAX_VOCAB = (int64_t)1 << 20;
// up to this many tokens the gradient needs no workspace
constexpr int EMBED_SMALL = 1024;
// Tokens that the gradient groups without a sort, every one looking through all
// ids: 512 tokens, 2048 columns 6.8 us.  Added to an fp32 table, us without and
// with the sort: 1100 tokens 17-19 / 36-39, 1500 21 / 37, 2048 25-29 / 36-39 (64 to
// 2048 columns); more columns are more workgroups that look: 2048, 4096 51, but
// 1000, 8192 34.  The sizes decide, and the ids may turn it: with half of the
// tokens one id, whose rows four waves sum, 1500 30-42 / 36, 2048 37-56 / 37; with all
// of them 1500 47-77 / 29, 2048 60-102 / 29.
inline bool embed_small(int64_t tokens, int64_t cols)
{
    return tokens <= EMBED_SMALL || (tokens <= 2048 && cols <= 2048);
}
// sorted positions whose rows one wave sums
constexpr int EMBED_RUN = 32;
constexpr int EMBED_MAX_BINS = 1024; // of either pass of the sort

struct EmbedArgs {
    int64_t tokens, vocab, cols;
    int id8;
    const void *ids;
    int e_kind, y_kind; // OutKind: of the table (its gradient), of Y (dY)
    const void *in;     // E; backward: dY
    int64_t ld_in;
    void *out; // Y; backward: dE
    int64_t ld_out;
    float scale;
    int accumulate;
    // backward, more than EMBED_SMALL tokens (the workspace): ids are cut into
    // low bits (the first pass) and high ones (the second)
    int lo_bits, hi_bits;
    int chunk, chunks;    // tokens per workgroup of the first pass
    int32_t *counts;      // [chunks][1 << lo_bits]
    int32_t *bounds;      // [(1 << lo_bits) + 1] first place of each bin
    struct Binned {
        int32_t id, token;
    } *binned;            // [tokens] tokens by low bits
    int32_t *order, *key; // [tokens] tokens by id, and their ids
    float *part;          // [runs][2][cols] sums that go on in another run
};

hipError_t launch_embed(const EmbedArgs &a, hipStream_t s);
hipError_t launch_embed_backward(const EmbedArgs &a, hipStream_t s);

// ---------------------------------------------------------------- linear cross entropy

// Workgroup tiles of a product.
enum XentTile {
    XT_64 = 0,
    XT_128,
    XT_256,
    XT_COUNT,
    XT_STREAM = XT_COUNT // few rows, no tiles: the logits of up to 16 (columns in
                         // turn), dW of up to 128 (rows in turn)
};
inline int xent_edge(int t) { return t == XT_256 ? 256 : t == XT_128 ? 128 : 64; }

// tokens of a step of the preparing kernel, and of one of its workgroups: more
// where looking through all targets before them would count
constexpr int XENT_STEP = 32;
inline int xent_prep(int64_t tokens) { return tokens <= 32768 ? XENT_STEP : 8 * XENT_STEP; }

// Parts that dX's sum over `cols` columns of a piece is cut into, for n rows of
// tiles of `edge` and tiles_n columns of them: those that fill 1 to 4 rounds of
// the chip's `slots` workgroups, or one, whichever is cheapest, a tile's way
// costing some 600 columns besides.  Sizes are below 2^21, tiles at most 2^23.
inline __host__ __device__ int xent_splits(int n, int edge, int tiles_n, int cols, int slots, int most)
{
    const int tiles = (n + edge - 1) / edge * tiles_n;
    int best = 1, cost = INT32_MAX;
    for (int r = 0; r <= 4; ++r) {
        int s = r == 0 || tiles == 0 ? 1 : slots * r / tiles;
        s = s < 1 ? 1 : s > most ? most : s;
        const float c = (float)((tiles * s + slots - 1) / slots) * (float)((cols + s - 1) / s + 600);
        if (c < (float)cost) {
            cost = c < 2e9f ? (int)c : INT32_MAX;
            best = s;
        }
    }
    return best;
}
struct XentSplits {
    int edge, tiles_n, cols, slots, most;
    int wgs; // workgroups at most: tiles times parts
    int num_cu;
};
// Workgroups of the streaming kernel, four waves with 16 columns at a time
// each: two to a compute unit.
constexpr int XENT_STREAM_ROWS = 16;
constexpr int XENT_DW_ROWS = 128; // rows of dW's streaming kernel
inline int64_t xent_streams(int64_t n, int num_cu)
{
    const int64_t g = (n + 63) / 64;
    return g < 2 * num_cu ? g : 2 * num_cu;
}

struct XentArgs {
    int64_t tokens, vocab, hidden, hp; // hp: hidden in whole 16-byte chunks
    int id8, bf16;
    const void *X, *targets;
    int64_t ldx;
    int prep;   // tokens per workgroup of the preparing kernel
    int direct; // forward, few tokens: X is read where it lies, every token is a row
    XentSplits dx;
    float scale;
    const float *lse_in, *dloss, *dlse; // backward
    float *loss, *lse;                  // forward
    // the workspace: rows are the tokens with a target, in order
    int32_t *count;       // rows, and (backward) parts of dX's sum
    int32_t *pos, *map;   // row of a token (-1: none), token of a row
    int32_t *tgt;         // target of a row
    float *ca, *cb, *cl;  // of a row: dloss + dlse, dloss, lse / ln 2
    float *gmax;          // largest |ca|, |cb| of each workgroup's tokens
    int64_t gmaxes;
    uint16_t *Xc;         // rows x hp, ldc apart: whole cache lines (xent_pitch)
    int64_t ldc;
    float *zt;            // target's logit of a row
    float *part;          // [tile column][row] maximum and sum
    int64_t part_tiles;
};

// One piece of the vocabulary: columns v0 .. v0 + n - 1.
struct XentPiece {
    const void *W; // its first row, rows 16-byte aligned unless loose
    int64_t ldw;
    int loose; // forward, few rows: W is read where it lies, aligned or not
    int64_t v0, n;
    int64_t tile0; // forward: its first tile column in XentArgs::part
    uint16_t *G;   // backward: rows x ldg
    int64_t ldg;
};

// Elements between the rows of X and of a piece of W in the workspace: rows on
// cache lines (those of 1416 values, 22.1 lines, cost the products 15 %).
inline int64_t xent_pitch(int64_t hidden) { return (hidden + 63) / 64 * 64; }

// W's rows v0 .. v0 + n - 1 (hidden values each) to out (hp each, zeros at
// the end, ldo apart)
struct XentCopy {
    const uint16_t *W;
    int64_t ldw, n, hidden, hp;
    uint16_t *out;
    int64_t ldo;
};

struct XentDx { // acc[split] (+)= G W
    float *acc; // [splits][rows][hp]
    int add;    // add to what acc holds
};
struct XentDw {
    void *dW; // the piece's first row
    int64_t ldd;
    int d_kind, add, vec, whole_lines;
};
struct XentOut { // dX = the sum of acc, scaled, by token
    const float *acc;
    void *dX;
    int64_t ldd;
    int d_kind;
};

hipError_t launch_xent_prepare(const XentArgs &a, bool backward, hipStream_t s);
hipError_t launch_xent_copy(const XentCopy &c, hipStream_t s);
hipError_t launch_xent_stats(int tile, const XentArgs &a, const XentPiece &p, hipStream_t s);
hipError_t launch_xent_loss(const XentArgs &a, hipStream_t s);
hipError_t launch_xent_g(int tile, const XentArgs &a, const XentPiece &p, hipStream_t s);
hipError_t launch_xent_dx(int tile, const XentArgs &a, const XentPiece &p, const XentDx &d,
                          hipStream_t s);
hipError_t launch_xent_dw(int tile, const XentArgs &a, const XentPiece &p, const XentDw &d,
                          hipStream_t s);
hipError_t launch_xent_out(const XentArgs &a, const XentOut &o, hipStream_t s);

} // namespace stg

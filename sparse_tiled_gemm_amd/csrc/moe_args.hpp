// Argument blocks and launchers of the mixture-of-experts operators
// (moe_api.cpp calls them; kernels_route.hip, kernels_q8.hip and
// kernels_grouped*.hip define them).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace stg {

// ---------------------------------------------------------------- routing

constexpr int ROUTE_MAX_GROUPS = 1024;
// up to this many slots every workgroup counts all of them for itself, in one
// launch; more are sorted in chunks by two launches
constexpr int ROUTE_SMALL = 4096;

struct RouteArgs {
    int64_t tokens, topk, slots;
    int groups, id8; // id8: ids are int64
    const void *ids;
    int32_t *offsets, *order, *pos;
    // chunked sort: slots per chunk, chunks, counts[chunk][group]
    int chunk, chunks;
    int32_t *counts;
};
// Slots per chunk of the chunked sort: at least 1024, at most 256 chunks
inline int64_t route_chunk(int64_t slots)
{
    const int64_t c = (slots + 255) / 256;
    return c <= 1024 ? 1024 : (c + 511) / 512 * 512;
}

struct RowsArgs { // rows of 16-bit elements moved between token and sorted order
    int64_t tokens, topk, cols, rows;
    const int32_t *pos;
    const float *weights;
    const void *in, *in2; // dispatch: X; combine: Ys; backward: dY, Ys
    int64_t ld_in, ld_in2;
    void *out; // dispatch: Xs; combine: Y; backward: dYs
    int64_t ld_out;
    float *dw;
    int bf16;
};

// the sort; `copy` (dispatch) may be null
hipError_t launch_route(const RouteArgs &a, const RowsArgs *copy, hipStream_t s);
hipError_t launch_combine(const RowsArgs &a, hipStream_t s);
hipError_t launch_combine_backward(const RowsArgs &a, hipStream_t s);

// ---------------------------------------------------------------- 8-bit checkpoints

struct Q8Args {
    int64_t rows, cols; // cols: of the checkpointed tensor (swiglu: 2 x the width of H)
    int bf16;
    const void *x; // store: X, swiglu: GU, backward: dH
    int64_t ldx;
    uint8_t *codes, *scales; // (read only in load and backward)
    void *out;               // load: X, swiglu: H, backward: dGU
    int64_t ldo;
    void *out2; // backward: H
    int64_t ldo2;
};
hipError_t launch_q8_store(const Q8Args &a, hipStream_t s);
hipError_t launch_q8_load(const Q8Args &a, hipStream_t s);
hipError_t launch_swiglu(const Q8Args &a, hipStream_t s);
hipError_t launch_swiglu_backward(const Q8Args &a, hipStream_t s);

// ---------------------------------------------------------------- grouped products

enum GroupedFamily {
    GF_GENERIC = 0,
    GF_SKINNY,    // rows: few per group
    GF_TILED_64,  // 64 x 64 tiles: few tiles
    GF_TILED_128, // 128 x 128 tiles, two workgroups per compute unit
    GF_TILED_256, // 256 x 256 tiles, one
    GF_COUNT
};

struct GroupedArgs {
    int weights_mode; // 0: ROWS, 1: WEIGHTS
    int groups;
    int64_t rows, N, K;
    const void *A, *B;
    const uint8_t *bs; // scales of an 8-bit B, else null
    const int32_t *offsets;
    const void *C;
    void *D;
    int64_t lda, ldb, ldd;
    int b_row; // ROWS: B_g is K x N (row-major)
    int bf16;  // A's type
    int d_kind; // OutKind
    int num_cu; // compute units of the device
    int vec;    // rows of C and D allow the vector epilogue (EpiArgs::vec)
    int whole_lines; // D's rows start on cache lines
};
// one-launch grid limits and operand requirements are checked by the plan
hipError_t launch_grouped_rows(int family, const GroupedArgs &a, hipStream_t s);    // tiled
hipError_t launch_grouped_skinny(const GroupedArgs &a, hipStream_t s); // rows
hipError_t launch_grouped_weights(int family, const GroupedArgs &a, hipStream_t s); // tiled
hipError_t launch_grouped(int family, const GroupedArgs &a, hipStream_t s);

} // namespace stg

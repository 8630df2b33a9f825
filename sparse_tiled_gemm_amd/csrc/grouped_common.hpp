// Pieces shared by the grouped-product kernels: which group a workgroup's
// tile belongs to, and the 8-bit B operand.
#pragma once
#include "device_common.hpp"
#include "moe_args.hpp"
#include "q8.hpp"

namespace stg {

// Rows [r0, r1) of group g, from bounds clamped to the matrix.
struct GroupRows {
    int g;
    int64_t r0, r1;
    int tm; // tile of the group
};

__device__ STG_AI inline void group_bounds(const GroupedArgs &a, int g, int &b, int &e)
{
    const int rows = (int)a.rows;
    b = min(max(a.offsets[g], 0), rows);
    e = max(min(max(a.offsets[g + 1], 0), rows), b);
}

// Tile `tile` of the groups' BM-row tiles counted one group after the other;
// false past the last one.  The groups are scanned 64 at a time, one per
// lane; every lane of the wave gets the (uniform) answer.
template <int BM>
__device__ STG_AI inline bool find_tile(const GroupedArgs &a, int tile, int lane, GroupRows &out)
{
    int done = 0; // tiles of the groups before g0
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
        int b = 0, e = 0;
        if (g0 + lane < a.groups)
            group_bounds(a, g0 + lane, b, e);
        const int n = (e - b + BM - 1) / BM;
        int incl = n;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int y = __shfl_up(incl, d);
            incl += lane >= d ? y : 0;
        }
        const uint64_t past = __ballot(done + incl > tile);
        if (past) {
            const int l = __builtin_ctzll(past);
            out.g = g0 + l;
            out.r0 = __builtin_amdgcn_readlane(b, l);
            out.r1 = __builtin_amdgcn_readlane(e, l);
            out.tm = tile - done - __builtin_amdgcn_readlane(incl - n, l);
            return true;
        }
        done += __builtin_amdgcn_readlane(incl, 63);
    }
    return false;
}

// Row tiles of BM rows that the groups of `rows` rows can need.
template <int BM>
inline int64_t max_row_tiles(const GroupedArgs &a)
{
    return (a.rows + BM - 1) / BM + (a.groups < a.rows ? a.groups : a.rows);
}

// The epilogue of group g's output: plain store, with C added where given.
// r0: first row of D (ROWS) of the tile's group; M: its rows.
__device__ STG_AI inline EpiArgs group_epilogue(const GroupedArgs &a, int g, int64_t r0, int64_t M)
{
    EpiArgs e;
    const int db = a.d_kind == OUT_F32 ? 4 : 2;
    const int64_t first = a.weights_mode ? (int64_t)g * a.K : r0;
    e.M = M;
    e.N = a.N;
    e.C = a.C ? (const uint8_t *)a.C + first * a.ldd * db : nullptr;
    e.ldc = a.ldd;
    e.bias = nullptr;
    e.alpha = 1.0f;
    e.relu = 0;
    e.d_kind = a.d_kind;
    e.D = (uint8_t *)a.D + first * a.ldd * db;
    e.ldd = a.ldd;
    e.vec = 0;
    e.sat = 0;
    e.c_kind = a.d_kind == OUT_F32 ? 0 : a.d_kind == OUT_F16 ? 1 : 2;
    return e;
}

} // namespace stg

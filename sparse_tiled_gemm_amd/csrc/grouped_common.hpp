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

// BM-row tiles of a group of n rows.  SHORT: only those with more than BM/2
// rows (long); a remainder of at most BM/2 is a short tile.
template <int BM, bool SHORT>
__device__ STG_AI inline int long_tiles(int n)
{
    return SHORT ? (n + BM / 2 - 1) / BM : (n + BM - 1) / BM;
}
template <int BM>
__device__ STG_AI inline int short_tiles(int n)
{
    return (n + BM - 1) / BM - (n + BM / 2 - 1) / BM;
}

// Long and short tiles of all groups.
template <int BM, bool SHORT>
__device__ STG_AI inline void count_tiles(const GroupedArgs &a, int lane, int &n_long, int &n_short)
{
    int l = 0, s = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64)
        if (g0 + lane < a.groups) {
            int b, e;
            group_bounds(a, g0 + lane, b, e);
            l += long_tiles<BM, SHORT>(e - b);
            s += SHORT ? short_tiles<BM>(e - b) : 0;
        }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        l += __shfl_xor(l, d);
        if (SHORT)
            s += __shfl_xor(s, d);
    }
    n_long = __builtin_amdgcn_readfirstlane(l);
    n_short = __builtin_amdgcn_readfirstlane(s);
}

// Tile `tile` of the groups' long tiles counted one group after the other,
// then (SHORT, from n_long on) of their short ones; false past the last.  The
// groups are scanned 64 at a time, one per lane; every lane of the wave gets
// the (uniform) answer.
template <int BM, bool SHORT = false>
__device__ STG_AI inline bool find_tile(const GroupedArgs &a, int tile, int n_long, int lane,
                                        GroupRows &out)
{
    const bool second = SHORT && tile >= n_long;
    if (second)
        tile -= n_long;
    int done = 0; // tiles of the groups before g0
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
        int b = 0, e = 0;
        if (g0 + lane < a.groups)
            group_bounds(a, g0 + lane, b, e);
        const int n = second ? short_tiles<BM>(e - b) : long_tiles<BM, SHORT>(e - b);
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
            out.tm = second ? (int)((out.r1 - out.r0) / BM)
                            : tile - done - __builtin_amdgcn_readlane(incl - n, l);
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

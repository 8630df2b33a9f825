// Pieces of the stable counting sorts (kernels_route.hip, kernels_embed.hip).
#pragma once
#include "device_common.hpp"

namespace stg {

// Lanes of this wave that hold the same group (none for g < 0); bits: those of
// a group's number.
__device__ STG_AI inline uint64_t same_group(int g, int bits)
{
    uint64_t m = __ballot(g >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t v = __ballot((g >> b) & 1);
        m &= (g >> b) & 1 ? v : ~v;
    }
    return g >= 0 ? m : 0;
}

__device__ STG_AI inline int lanes_below(uint64_t m)
{
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                     __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// v[0 .. n) (LDS) becomes its exclusive prefix sum and v[n] the total; all
// NT threads of the workgroup call it after a barrier; it ends with one.
// tmp: NT / 64 ints.
template <int NT>
__device__ STG_AI inline void scan_lds(int *v, int n, int *tmp, int tid)
{
    const int lane = tid & 63, wave = tid >> 6;
    int base = 0;
    for (int i0 = 0; i0 < n; i0 += NT) {
        const int i = i0 + tid;
        const int x = i < n ? v[i] : 0;
        int incl = x;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int y = __shfl_up(incl, d);
            if (lane >= d)
                incl += y;
        }
        if (lane == 63)
            tmp[wave] = incl;
        __syncthreads();
        int before = base;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) {
            const int t = tmp[w];
            before += w < wave ? t : 0;
            base += t;
        }
        if (i < n)
            v[i] = before + incl - x;
        __syncthreads();
    }
    if (tid == 0)
        v[n] = base;
    __syncthreads();
}

} // namespace stg

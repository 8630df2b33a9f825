// The LDS-tiled grouped product of the rows (k_grouped_tiled): A is
// K-contiguous, B_g either K-contiguous (N x K) or MN-major (K x N).
#include "grouped_tiled.hpp"

namespace stg {

template <class OP, int BLAY, int BM, int BN>
static hipError_t launch_t(const GroupedArgs &a, hipStream_t s)
{
    const int tiles_n = (int)((a.N + BN - 1) / BN);
    const int64_t tiles = max_row_tiles<BM>(a) * tiles_n;
    constexpr bool SHORT = BM == 256;
    const int64_t extra = SHORT ? a.num_cu / 2 : 0; // second halves of the last long tiles
    const dim3 grid((unsigned)((tiles + extra + 7) / 8 * 8 + 8));
    hipLaunchKernelGGL((k_grouped_tiled<OP, false, GL_K, BLAY, BM, BN, SHORT>), grid, dim3(512), 0, s,
                       a, 0, tiles_n);
    return hipGetLastError();
}

template <class OP, int BLAY>
static hipError_t launch_small(const GroupedArgs &a, hipStream_t s)
{
    const int tiles_n = (int)((a.N + 63) / 64);
    const dim3 grid((unsigned)((max_row_tiles<64>(a) * tiles_n + 7) / 8 * 8));
    hipLaunchKernelGGL((k_grouped_small<OP, false, GL_K, BLAY>), grid, dim3(256), 0, s, a, 0, tiles_n);
    return hipGetLastError();
}

template <class OP>
static hipError_t launch_op(int family, const GroupedArgs &a, hipStream_t s)
{
    if (family == GF_TILED_256)
        return a.b_row ? launch_t<OP, GL_MN, 256, 256>(a, s) : launch_t<OP, GL_K, 256, 256>(a, s);
    if (family == GF_TILED_64)
        return a.b_row ? launch_small<OP, GL_MN>(a, s) : launch_small<OP, GL_K>(a, s);
    return a.b_row ? launch_t<OP, GL_MN, 128, 128>(a, s) : launch_t<OP, GL_K, 128, 128>(a, s);
}

hipError_t launch_grouped_rows(int family, const GroupedArgs &a, hipStream_t s)
{
    return a.bf16 ? launch_op<Op16BF16>(family, a, s) : launch_op<Op16F16>(family, a, s);
}

} // namespace stg

// The LDS-tiled grouped product of the weights' gradient (k_grouped_tiled):
// both operands MN-major, the sum runs over the group's rows; B in 16 bits
// or as codes and scales of an 8-bit checkpoint.
#include "grouped_tiled.hpp"

namespace stg {

template <class OP, int BLAY, int BM, int BN>
static hipError_t launch_t(const GroupedArgs &a, hipStream_t s)
{
    const int tiles_m = (int)((a.K + BM - 1) / BM), tiles_n = (int)((a.N + BN - 1) / BN);
    const int64_t per_xcd = ((int64_t)tiles_m * tiles_n + 7) / 8;
    const dim3 grid((unsigned)(per_xcd * 8 * a.groups));
    hipLaunchKernelGGL((k_grouped_tiled<OP, true, GL_MN, BLAY, BM, BN, false>), grid, dim3(512), 0, s, a,
                       tiles_m, tiles_n);
    return hipGetLastError();
}

template <class OP, int BLAY>
static hipError_t launch_small(const GroupedArgs &a, hipStream_t s)
{
    const int tiles_m = (int)((a.K + 63) / 64), tiles_n = (int)((a.N + 63) / 64);
    const int64_t per_xcd = ((int64_t)tiles_m * tiles_n + 7) / 8;
    const dim3 grid((unsigned)(per_xcd * 8 * a.groups));
    hipLaunchKernelGGL((k_grouped_small<OP, true, GL_MN, BLAY>), grid, dim3(256), 0, s, a, tiles_m,
                       tiles_n);
    return hipGetLastError();
}

template <class OP>
static hipError_t launch_op(int family, const GroupedArgs &a, hipStream_t s)
{
    if (family == GF_TILED_256)
        return a.bs ? launch_t<OP, GL_Q8, 256, 256>(a, s) : launch_t<OP, GL_MN, 256, 256>(a, s);
    if (family == GF_TILED_64)
        return a.bs ? launch_small<OP, GL_Q8>(a, s) : launch_small<OP, GL_MN>(a, s);
    return a.bs ? launch_t<OP, GL_Q8, 128, 128>(a, s) : launch_t<OP, GL_MN, 128, 128>(a, s);
}

hipError_t launch_grouped_weights(int family, const GroupedArgs &a, hipStream_t s)
{
    return a.bf16 ? launch_op<Op16BF16>(family, a, s) : launch_op<Op16F16>(family, a, s);
}

} // namespace stg

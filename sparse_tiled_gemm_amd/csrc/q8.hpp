// Values of the 8-bit checkpoints (gemm_moe.h): scale bytes and clamping.
#pragma once
#include "device_common.hpp"

namespace stg {

// A scale byte's 2^(s - 127); 255 is NaN, 0 the subnormal 2^-127.
__device__ STG_AI inline float e8m0(uint32_t s)
{
    const uint32_t b = s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : s << 23;
    return __builtin_bit_cast(float, b);
}

// The largest scale byte under which every code's value lies in the type's
// range: 448 * 2^(byte - 127).
template <bool BF>
constexpr uint32_t MAX_SCALE = BF ? 246 : 134;

// x clamped to the finite range of the 16-bit type (NaN stays NaN).
template <bool BF>
__device__ STG_AI inline float clamp16(float x)
{
    constexpr float big = BF ? 0x1.FEp127f : 65504.0f;
    x = x > big ? big : x;
    return x < -big ? -big : x;
}

} // namespace stg

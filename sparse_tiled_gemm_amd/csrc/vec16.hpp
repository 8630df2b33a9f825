// Eight 16-bit elements as one 16-byte access at any element-aligned
// address, and their conversion to and from fp32.
#pragma once
#include "device_common.hpp"

namespace stg {

struct __attribute__((packed, aligned(2))) u4_any_t {
    u4_t v;
};

// The first n (1..8) of the eight elements at p; zeros after them.
__device__ STG_AI inline u4_t load8(const uint16_t *p, int n)
{
    if (n >= 8)
        return ((const u4_any_t *)p)->v;
    u4_t v{};
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n)
            v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    return v;
}

__device__ STG_AI inline void store8(uint16_t *p, u4_t v, int n)
{
    if (n >= 8) {
        ((u4_any_t *)p)->v = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n)
            p[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
}

template <bool BF>
__device__ STG_AI inline float widen(uint32_t h)
{
    return BF ? __builtin_bit_cast(float, h << 16)
              : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

template <bool BF>
__device__ STG_AI inline void widen8(u4_t v, float (&f)[8])
{
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint32_t w = v[e >> 1];
        f[e] = widen<BF>(w & 0xFFFFu);
        f[e + 1] = BF ? __builtin_bit_cast(float, w & 0xFFFF0000u) : widen<BF>(w >> 16);
    }
}

// Rounded to nearest even.
template <bool BF>
__device__ STG_AI inline u4_t narrow8(const float (&f)[8])
{
    u4_t v;
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        v[e >> 1] = BF ? f32_to_bf16_bits(f[e]) | ((uint32_t)f32_to_bf16_bits(f[e + 1]) << 16)
                       : f32_to_f16_bits(f[e]) | ((uint32_t)f32_to_f16_bits(f[e + 1]) << 16);
    return v;
}

} // namespace stg

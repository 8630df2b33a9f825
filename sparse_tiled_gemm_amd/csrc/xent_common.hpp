// Pieces shared by the kernels of the linear cross entropy.
#pragma once
#include "device_common.hpp"
#include "vocab_args.hpp"

namespace stg {

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

__device__ STG_AI inline int xent_target(const XentArgs &a, int64_t t)
{
    // -1: none
    if (a.id8) {
        const int64_t v = ((const int64_t *)a.targets)[t];
        return v >= 0 && v < a.vocab ? (int)v : -1;
    }
    const int32_t v = ((const int32_t *)a.targets)[t];
    return v >= 0 && v < a.vocab ? v : -1;
}

// The logits' gradient enters its products as a 16-bit value relative to the
// call's largest coefficient: |G| <= 2 F with F = 1, or 2^14 for fp16, whose
// normal values then begin at 2^-28 of that coefficient (a probability of 4e-9)
// instead of 2^-14.
__device__ STG_AI inline float xent_unit(const XentArgs &a) { return a.bf16 ? 1.0f : 16384.0f; }

// The largest coefficient of the call; every wave computes it.
__device__ STG_AI inline float xent_gmax(const XentArgs &a, int lane)
{
    float g = 0.0f;
    for (int64_t i = lane; i < a.gmaxes; i += 64)
        g = __builtin_fmaxf(g, a.gmax[i]);
#pragma unroll
    for (int d = 32; d; d >>= 1)
        g = __builtin_fmaxf(g, __shfl_xor(g, d));
    return g;
}

// What a product of G is multiplied by.
__device__ STG_AI inline float xent_factor(const XentArgs &a, int lane)
{
    return xent_gmax(a, lane) / xent_unit(a) * a.scale;
}

} // namespace stg

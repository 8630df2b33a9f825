// Pieces shared by the kernels of the linear cross entropy.
#pragma once
#include "vocab_id.hpp"

namespace stg {

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

// Token t's target, -1: none.
__device__ STG_AI inline int xent_target(const XentArgs &a, int64_t t)
{
    return vocab_id(a.targets, a.id8, a.vocab, t);
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

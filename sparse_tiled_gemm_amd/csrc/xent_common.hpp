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

// Rows, and a row's target.
__device__ STG_AI inline int xent_rows(const XentArgs &a)
{
    return a.direct ? (int)a.tokens : __builtin_amdgcn_readfirstlane(*a.count);
}
__device__ STG_AI inline int xent_row_target(const XentArgs &a, int64_t row)
{
    return a.direct ? xent_target(a, row) : a.tgt[row];
}

// What a sum of exponentials is relative to: their largest argument m, but zero
// where that is infinite.  All -inf then sum to zero, and one +inf makes the sum
// +inf as the definition does (relative to itself it would be a NaN).
__device__ STG_AI inline float sum_ref(float m)
{
    return __builtin_fabsf(m) == __builtin_inff() ? 0.0f : m;
}

// The logits' gradient enters its products as a 16-bit value relative to the
// call's largest coefficient: |G| <= 2 F with F = 1, or 2^14 for fp16, whose
// normal values then begin at 2^-28 of that coefficient (a probability of 4e-9)
// instead of 2^-14.  (16 bits, because the matrix instructions take both operands
// of one type: G in two halves would make five products of three.  512 tokens,
// 8192 x 256, errors against 64 bits relative to the result: 16-bit outputs 2.0e-3
// for bf16 and 2.75e-4 for fp16, where rounding them alone gives 1.66e-3 and
// 2.3e-4; fp32 outputs 1.1e-3 and 1.5e-4.)
__device__ STG_AI inline float xent_unit(const XentArgs &a) { return a.bf16 ? 1.0f : 16384.0f; }

// The largest finite coefficient of the call, 1 if there is none but zeros
// (an infinity or NaN stays what it is in its own row); every wave computes it,
// the first 256 values from loads that were begun earlier.
struct Gmax {
    float v[4];
};
__device__ STG_AI inline Gmax load_gmax(const XentArgs &a, int lane)
{
    Gmax g;
#pragma unroll
    for (int i = 0; i < 4; ++i) // (past the end: the last one again)
        g.v[i] = a.gmax[min((int64_t)lane + 64 * i, a.gmaxes - 1)];
    return g;
}
__device__ STG_AI inline float xent_gmax(const XentArgs &a, const Gmax &first, int lane)
{
    float g = __builtin_fmaxf(__builtin_fmaxf(first.v[0], first.v[1]),
                              __builtin_fmaxf(first.v[2], first.v[3]));
    for (int64_t i = lane + 256; i < a.gmaxes; i += 64)
        g = __builtin_fmaxf(g, a.gmax[i]);
#pragma unroll
    for (int d = 32; d; d >>= 1)
        g = __builtin_fmaxf(g, __shfl_xor(g, d));
    return g > 0.0f ? g : 1.0f;
}

// What a product of G is multiplied by.
__device__ STG_AI inline float xent_factor(const XentArgs &a, const Gmax &first, int lane)
{
    return xent_gmax(a, first, lane) / xent_unit(a) * a.scale;
}

} // namespace stg

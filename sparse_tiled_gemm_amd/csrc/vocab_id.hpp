// Token ids and targets (kernels_embed.hip, kernels_xent*.hip).
#pragma once
#include "device_common.hpp"
#include "vocab_args.hpp"

namespace stg {

// ids[t], -1 if it is not in 0 .. vocab-1 (vocab < 2^31); id8: 64-bit ids.  Both
// words are loaded whatever the size, so that no branch stands between several
// loads.
__device__ STG_AI inline int vocab_id(const void *ids, int id8, int64_t vocab, int64_t t)
{
    const int32_t *p = (const int32_t *)ids + (t << id8);
    int32_t lo = p[0], hi = p[id8];
    asm("" : "+v"(lo), "+v"(hi)); // (neither load waits for the other's value)
    return ((hi & -id8) == 0) & ((uint32_t)lo < (uint32_t)vocab) ? lo : -1;
}

} // namespace stg

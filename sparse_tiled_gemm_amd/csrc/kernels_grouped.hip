// Products of a mixture-of-experts MLP over ragged groups of rows
// (gemm_moe.h, "grouped products"): the generic kernel, which serves every
// size, stride and alignment, and the dispatch over the kernel families.
#include "grouped_common.hpp"
#include "internal.hpp"

namespace stg {

// One wave per 32 x 32 output tile, operands read element by element.
// W: the weights' product (the sum runs over the group's rows); Q8: B holds
// E4M3 codes with scales.
template <class OP, bool W, bool Q8>
__global__ __launch_bounds__(256) void k_grouped_generic(GroupedArgs a, int tiles_n)
{
    constexpr int LE = 8, KI = 16; // K per lane and per instruction
    constexpr bool BF = std::is_same<OP, OpBF16>::value;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tn = blockIdx.x % tiles_n, rest = blockIdx.x / tiles_n;
    GroupRows t;
    int64_t m0, M, K;
    if constexpr (W) {
        const int tiles_m = (int)((a.K + 63) / 64);
        int b, e;
        t.g = rest / tiles_m;
        group_bounds(a, t.g, b, e);
        t.r0 = b;
        t.r1 = e;
        m0 = (int64_t)(rest % tiles_m) * 64;
        M = a.K;
        K = t.r1 - t.r0;
    } else {
        if (!find_tile<64>(a, rest, 0, lane, t))
            return;
        m0 = (int64_t)t.tm * 64;
        M = t.r1 - t.r0;
        K = a.K;
    }
    m0 += (wave >> 1) * 32;
    const int64_t n0 = (int64_t)tn * 64 + (wave & 1) * 32;
    if (m0 >= M || n0 >= a.N)
        return; // whole wave idle
    const int64_t am = m0 + (lane & 31), bn = n0 + (lane & 31);
    const bool a_ok = am < M, b_ok = bn < a.N;
    const uint16_t *A = (const uint16_t *)a.A + t.r0 * a.lda;
    const int64_t a_rs = W ? 1 : a.lda, a_cs = W ? a.lda : 1;
    // B's group: a matrix of its own, or (W) the group's rows
    const bool b_row = W || a.b_row;
    const int64_t b_first = W ? t.r0 : (int64_t)t.g * (b_row ? a.K : a.N);
    const int64_t b_rs = b_row ? a.ldb : 1, b_cs = b_row ? 1 : a.ldb;
    const uint8_t *B = (const uint8_t *)a.B + b_first * a.ldb * (Q8 ? 1 : 2);
    const int64_t nb = (a.N + 31) / 32;
    typename OP::acc_t acc = {};
    for (int64_t k0 = 0; k0 < K; k0 += KI) {
        uint32_t fa[4], fb[4];
        const int64_t kb = k0 + (lane >> 5) * LE;
        load_frag_strided<2, LE>(fa, A, a_ok, am * a_rs, a_cs, kb, K);
        if constexpr (Q8) {
#pragma unroll
            for (int j = 0; j < LE; ++j) {
                float v = 0.0f;
                if (b_ok && kb + j < K) {
                    const int c = B[(kb + j) * b_rs + bn];
                    v = __builtin_amdgcn_cvt_pk_f32_fp8(c, false)[0] *
                        e8m0(a.bs[(t.r0 + kb + j) * nb + bn / 32]);
                    v = clamp16<BF>(v);
                }
                const uint32_t h = BF ? f32_to_bf16_bits(v) : f32_to_f16_bits(v);
                fb[j / 2] = j & 1 ? fb[j / 2] | (h << 16) : h;
            }
        } else {
            load_frag_strided<2, LE>(fb, B, b_ok, bn * b_cs, b_rs, kb, K);
        }
        acc = OP::mma(fa, fb, acc);
    }
    typename OP::acc_t grid[1][1] = {{acc}};
    epilogue_grid<OP, 1, 1>(group_epilogue(a, t.g, t.r0, M), grid, m0, n0, lane);
}

template <class OP>
static hipError_t launch_generic(const GroupedArgs &a, hipStream_t s)
{
    const int tiles_n = (int)((a.N + 63) / 64);
    const int64_t tiles = a.weights_mode ? (a.K + 63) / 64 * a.groups : max_row_tiles<64>(a);
    const dim3 grid((unsigned)(tiles * tiles_n));
    if (!a.weights_mode)
        hipLaunchKernelGGL((k_grouped_generic<OP, false, false>), grid, dim3(256), 0, s, a, tiles_n);
    else if (a.bs)
        hipLaunchKernelGGL((k_grouped_generic<OP, true, true>), grid, dim3(256), 0, s, a, tiles_n);
    else
        hipLaunchKernelGGL((k_grouped_generic<OP, true, false>), grid, dim3(256), 0, s, a, tiles_n);
    return hipGetLastError();
}

hipError_t launch_grouped(int family, const GroupedArgs &a, hipStream_t s)
{
    if (family == GF_SKINNY)
        return launch_grouped_skinny(a, s);
    if (family != GF_GENERIC)
        return a.weights_mode ? launch_grouped_weights(family, a, s)
                              : launch_grouped_rows(family, a, s);
    return a.bf16 ? launch_generic<OpBF16>(a, s) : launch_generic<OpF16>(a, s);
}

} // namespace stg

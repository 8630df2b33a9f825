// Linear cross entropy: the two products of the logits' gradient G, on the
// grouped products' main loop (grouped_tiled.hpp).
//  - dX: acc[split] (+)= G W over a part of the piece's columns, fp32 in the
//    workspace (the pieces add up there; splits fill the chip where there are
//    few tiles), joined and rounded by k_xent_out;
//  - dW = G^T X: the sum runs over all rows, so a piece's part of dW is
//    complete and rounded at once.
#include "grouped_tiled.hpp"
#include "xent_common.hpp"

namespace stg {

// The piece's columns in whole 16-byte chunks (G's are written that far).
__device__ STG_AI inline int64_t chunks8(int64_t n) { return (n + 7) & ~(int64_t)7; }

struct DxTile {
    GroupedArgs g;
    EpiArgs e;
    int64_t K, KB;
};
// Operands of split `split` of dX's product; K 0: nothing to add.
__device__ STG_AI inline DxTile dx_tile(const XentArgs &a, const XentPiece &p, const XentDx &d, int n,
                                        int split, int splits)
{
    DxTile x{};
    const int64_t per = ((p.n + splits - 1) / splits + 63) / 64 * 64;
    const int64_t k0 = split * per, kb = min(per, p.n - k0);
    x.KB = kb > 0 ? kb : 0;
    x.K = chunks8(x.KB);
    x.g.N = a.hp;
    x.g.A = p.G + k0;
    x.g.lda = p.ldg;
    x.g.B = (const uint16_t *)p.W + k0 * p.ldw;
    x.g.ldb = p.ldw;
    x.g.K = x.K;
    x.e.M = n;
    x.e.N = a.hp;
    x.e.alpha = 1.0f;
    x.e.d_kind = OUT_F32;
    x.e.D = d.acc + (int64_t)split * n * a.hp;
    x.e.ldd = x.e.ldc = a.hp;
    x.e.C = d.add ? x.e.D : nullptr;
    x.e.vec = 1;
    return x;
}

__device__ STG_AI inline GroupedArgs dw_args(const XentArgs &a, const XentPiece &p)
{
    GroupedArgs g{};
    g.weights_mode = 1;
    g.K = chunks8(p.n);
    g.N = a.hp;
    g.A = p.G;
    g.lda = p.ldg;
    g.B = a.Xc;
    g.ldb = a.ldc;
    return g;
}
__device__ STG_AI inline EpiArgs dw_epilogue(const XentArgs &a, const XentPiece &p, const XentDw &d)
{
    EpiArgs e{};
    e.M = p.n;
    e.N = a.hidden;
    e.alpha = 1.0f;
    e.d_kind = d.d_kind;
    e.D = d.dW;
    e.ldd = e.ldc = d.ldd;
    e.C = d.add ? d.dW : nullptr;
    e.c_kind = d.d_kind == OUT_F32 ? 0 : d.d_kind == OUT_F16 ? 1 : 2;
    e.vec = d.vec;
    return e;
}

template <class OP, bool DW, int BM, int BN>
__global__ __launch_bounds__(512, BM * BN >= 256 * 128 ? 2 : 4) void
k_xent_grad(XentArgs a, XentPiece p, XentDx dx, XentDw dw, int tiles_n)
{
    constexpr int AB = region_bytes<BM / 2, BN / 4>(), BB = region_bytes<BN / 2, BN / 4>();
    __shared__ __attribute__((aligned(1024))) uint8_t a00[AB], a10[AB], a01[AB], a11[AB], b00[BB],
        b10[BB], b01[BB], b11[BB];
    const Regions L = {a00, a10, a01, a11, b00, b10, b01, b11};
    constexpr int ALAY = DW ? GL_MN : GL_K;
    typedef TileShape<OP, DW, ALAY, GL_MN, BM, BN> S;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = __builtin_amdgcn_readfirstlane(*a.count);
    const int tiles_m = (int)(((DW ? p.n : (int64_t)n) + BM - 1) / BM);
    const int tiles = tiles_m * tiles_n, splits = DW ? 1 : __builtin_amdgcn_readfirstlane(a.count[1]);
    const int id = xcd_tile(blockIdx.x, tiles * splits);
    if (id < 0)
        return;
    int tm, tn;
    tile_of(id % tiles, tiles_m, tiles_n, tm, tn);
    const int64_t m = wave_uniform((int64_t)tm * BM), c = wave_uniform((int64_t)tn * BN);
    typename OP::acc_t acc[S::FM][S::FN];
    const GroupRows t = {0, 0, n, 0};
    if constexpr (DW) {
        const GroupedArgs g = dw_args(a, p);
        const Gmax first = load_gmax(a, lane); // (nothing waits for it later)
        tile_sum<OP, true, GL_MN, GL_MN, BM, BN>(g, t, m, c, g.K, n, n, lane, wave, L, acc);
        const float f = xent_factor(a, first, lane);
#pragma unroll
        for (int i = 0; i < S::FM; ++i)
#pragma unroll
            for (int j = 0; j < S::FN; ++j)
                acc[i][j] *= f;
        store_acc<OP, S>(dw_epilogue(a, p, dw), dw.whole_lines, m, c, acc, lane, wave,
                         wave_slab(L, wave));
    } else {
        const DxTile x = dx_tile(a, p, dx, n, id / tiles, splits);
        if (x.K == 0 && dx.add)
            return;
        tile_sum<OP, false, GL_K, GL_MN, BM, BN>(x.g, t, m, c, n, x.K, x.KB, lane, wave, L, acc);
        store_acc<OP, S>(x.e, 0, m, c, acc, lane, wave, wave_slab(L, wave));
    }
}

template <class OP, bool DW>
__global__ __launch_bounds__(256, 2) void k_xent_grad_small(XentArgs a, XentPiece p, XentDx dx,
                                                            XentDw dw, int tiles_n)
{
    __shared__ __attribute__((aligned(1024))) uint8_t s0[16384], s1[16384], s2[16384], s3[16384];
    constexpr int ALAY = DW ? GL_MN : GL_K;
    typedef SmallShape<OP, DW, ALAY, GL_MN> S;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = __builtin_amdgcn_readfirstlane(*a.count);
    const int tiles_m = (int)(((DW ? p.n : (int64_t)n) + 63) / 64);
    const int tiles = tiles_m * tiles_n, splits = DW ? 1 : __builtin_amdgcn_readfirstlane(a.count[1]);
    const int id = xcd_tile(blockIdx.x, tiles * splits);
    if (id < 0)
        return;
    int tm, tn;
    tile_of(id % tiles, tiles_m, tiles_n, tm, tn);
    const int64_t m = wave_uniform((int64_t)tm * 64), c = wave_uniform((int64_t)tn * 64);
    typename OP::acc_t acc[2][2];
    const GroupRows t = {0, 0, n, 0};
    uint8_t *slab = wave == 0 ? s0 : wave == 1 ? s1 : wave == 2 ? s2 : s3;
    if constexpr (DW) {
        const GroupedArgs g = dw_args(a, p);
        const Gmax first = load_gmax(a, lane);
        small_sum<OP, true, GL_MN, GL_MN>(g, t, m, c, g.K, n, n, lane, wave, s0, s1, s2, s3, acc);
        const float f = xent_factor(a, first, lane);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] *= f;
        store_acc<OP, S>(dw_epilogue(a, p, dw), dw.whole_lines, m, c, acc, lane, wave,
                         (uint32_t *)slab);
    } else {
        const DxTile x = dx_tile(a, p, dx, n, id / tiles, splits);
        if (x.K == 0 && dx.add)
            return;
        small_sum<OP, false, GL_K, GL_MN>(x.g, t, m, c, n, x.K, x.KB, lane, wave, s0, s1, s2, s3, acc);
        store_acc<OP, S>(x.e, 0, m, c, acc, lane, wave, (uint32_t *)slab);
    }
}

template <class OP, bool DW>
static hipError_t launch_t(int tile, const XentArgs &a, const XentPiece &p, const XentDx &dx,
                           const XentDw &dw, hipStream_t s)
{
    const int64_t b = xent_edge(tile);
    const int tiles_n = (int)((a.hp + b - 1) / b);
    const int64_t wgs = DW ? (p.n + b - 1) / b * tiles_n : a.dx.wgs;
    const dim3 grid((unsigned)((wgs + 7) / 8 * 8));
    if (tile == XT_256)
        hipLaunchKernelGGL((k_xent_grad<OP, DW, 256, 256>), grid, dim3(512), 0, s, a, p, dx, dw,
                           tiles_n);
    else if (tile == XT_128)
        hipLaunchKernelGGL((k_xent_grad<OP, DW, 128, 128>), grid, dim3(512), 0, s, a, p, dx, dw,
                           tiles_n);
    else
        hipLaunchKernelGGL((k_xent_grad_small<OP, DW>), grid, dim3(256), 0, s, a, p, dx, dw, tiles_n);
    return hipGetLastError();
}

hipError_t launch_xent_dx(int tile, const XentArgs &a, const XentPiece &p, const XentDx &d,
                          hipStream_t s)
{
    return a.bf16 ? launch_t<Op16BF16, false>(tile, a, p, d, XentDw{}, s)
                  : launch_t<Op16F16, false>(tile, a, p, d, XentDw{}, s);
}

hipError_t launch_xent_dw(int tile, const XentArgs &a, const XentPiece &p, const XentDw &d,
                          hipStream_t s)
{
    return a.bf16 ? launch_t<Op16BF16, true>(tile, a, p, XentDx{}, d, s)
                  : launch_t<Op16F16, true>(tile, a, p, XentDx{}, d, s);
}

} // namespace stg

// Linear cross entropy: the logits' tiles.  The product X W^T runs on the
// grouped products' main loop (grouped_tiled.hpp) as one group; what becomes of
// a tile is decided in registers, so that no logit reaches memory:
//  - forward: every row's maximum m and sum of exp(z - m) over the tile's
//    columns, and its target's logit;
//  - backward: G = (dloss + dlse) exp(z - lse) - [target] dloss in 16 bits,
//    for the two products that follow.
#include "grouped_tiled.hpp"
#include "xent_common.hpp"

namespace stg {

// Reductions over the 16 lanes that share an accumulator's rows (DPP: lanes
// 1 and 2 apart, then the mirrored half and whole row).
template <int CTRL>
__device__ STG_AI inline float dpp(float x)
{
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}
__device__ STG_AI inline float max16(float x)
{
    x = __builtin_fmaxf(x, dpp<0xB1>(x));
    x = __builtin_fmaxf(x, dpp<0x4E>(x));
    x = __builtin_fmaxf(x, dpp<0x141>(x));
    return __builtin_fmaxf(x, dpp<0x140>(x));
}
__device__ STG_AI inline float sum16(float x)
{
    x += dpp<0xB1>(x);
    x += dpp<0x4E>(x);
    x += dpp<0x141>(x);
    return x + dpp<0x140>(x);
}

// Statistics of the tile at (m_blk, n_blk), tile column tn; n: rows.  lds: BM
// ints, GN * BM pairs of floats (16-byte aligned).
template <class OP, class S>
__device__ STG_AI inline void tile_stats(const XentArgs &a, const XentPiece &p, int n, int64_t m_blk,
                                         int64_t n_blk, int tn,
                                         typename OP::acc_t (&acc)[S::FM][S::FN], int lane, int wave,
                                         int *tgt, float *st)
{
    static_assert(S::PA == 1 && S::PB == 1, "a wave's block is one piece");
    const int tid = threadIdx.x, l16 = lane & 15, q = lane >> 4;
    const int rb = wave / S::GN * S::WM, cb = wave % S::GN * S::WN;
    if (tid < S::BM) // targets relative to the tile's columns
        tgt[tid] = m_blk + tid < n ? (int)(a.tgt[m_blk + tid] - (p.v0 + n_blk)) : -1;
    __syncthreads();
    const int left = (int)min((int64_t)S::BN, p.n - n_blk) - cb - l16; // columns from this lane's on
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
        const i4_t tg = *(const i4_t *)(tgt + rb + 16 * i + 4 * q);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float z[S::FN], m = -INFINITY, s = 0.0f;
#pragma unroll
            for (int j = 0; j < S::FN; ++j) {
                z[j] = 16 * j < left ? acc[i][j][r] * a.scale : -INFINITY;
                m = __builtin_fmaxf(m, z[j]);
            }
            const int d = tg[r] - cb - l16;
            if ((uint32_t)d < (uint32_t)S::WN && (d & 15) == 0) {
                float x = z[0];
#pragma unroll
                for (int j = 1; j < S::FN; ++j)
                    x = d >> 4 == j ? z[j] : x;
                a.zt[m_blk + rb + 16 * i + 4 * q + r] = x;
            }
            m = max16(m);
            const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int j = 0; j < S::FN; ++j)
                s += __builtin_amdgcn_exp2f((z[j] - ref) * LOG2E);
            s = sum16(s);
            if (l16 == 0) {
                float *o = st + ((wave % S::GN) * S::BM + rb + 16 * i + 4 * q + r) * 2;
                o[0] = m;
                o[1] = s;
            }
        }
    }
    __syncthreads();
    if (tid < S::BM && m_blk + tid < n) {
        float m = -INFINITY, s = 0.0f;
#pragma unroll
        for (int w = 0; w < S::GN; ++w)
            m = __builtin_fmaxf(m, st[(w * S::BM + tid) * 2]);
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int w = 0; w < S::GN; ++w)
            s += st[(w * S::BM + tid) * 2 + 1] *
                 __builtin_amdgcn_exp2f((st[(w * S::BM + tid) * 2] - ref) * LOG2E);
        float *o = a.part + ((p.tile0 + tn) * a.tokens + m_blk + tid) * 2;
        o[0] = m;
        o[1] = s;
    }
}

// The tile's G in place of its sums.  rows: four arrays of BM values in LDS.
template <class OP, class S>
__device__ STG_AI inline void tile_g(const XentArgs &a, const XentPiece &p, int n, int64_t m_blk,
                                     int64_t n_blk, typename OP::acc_t (&acc)[S::FM][S::FN], int lane,
                                     int wave, float *rows)
{
    static_assert(S::PA == 1 && S::PB == 1, "a wave's block is one piece");
    const int tid = threadIdx.x, l16 = lane & 15, q = lane >> 4;
    const int rb = wave / S::GN * S::WM, cb = wave % S::GN * S::WN;
    const float gmax = xent_gmax(a, lane);
    if (tid < S::BM) {
        const int64_t row = m_blk + tid;
        const bool in = row < n;
        const float f = xent_unit(a);
        // (gmax 0: every coefficient is)
        rows[tid] = in && gmax != 0.0f ? a.ca[row] / gmax * f : 0.0f;
        rows[S::BM + tid] = in && gmax != 0.0f ? a.cb[row] / gmax * f : 0.0f;
        rows[2 * S::BM + tid] = in ? a.cl[row] : 0.0f;
        ((int *)rows)[3 * S::BM + tid] = in ? (int)(a.tgt[row] - (p.v0 + n_blk)) : -1;
    }
    __syncthreads();
    const int left = (int)min((int64_t)S::BN, p.n - n_blk) - cb - l16;
    const float k = a.scale * LOG2E;
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
        const float *at = rows + rb + 16 * i + 4 * q;
        const f4_t ca = *(const f4_t *)at, cbv = *(const f4_t *)(at + S::BM);
        const f4_t cl = *(const f4_t *)(at + 2 * S::BM);
        const i4_t tg = *(const i4_t *)(at + 3 * S::BM);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = tg[r] - cb - l16;
#pragma unroll
            for (int j = 0; j < S::FN; ++j) {
                const float e =
                    __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r], k, -cl[r]));
                float g = ca[r] * e;
                g -= d == 16 * j ? cbv[r] : 0.0f;
                acc[i][j][r] = 16 * j < left ? g : 0.0f;
            }
        }
    }
    __syncthreads(); // the rows are read before LDS takes the slabs
}

// (whole rows of G are written, zeros behind the piece's last column)
__device__ STG_AI inline EpiArgs g_epilogue(const XentArgs &a, const XentPiece &p, int n)
{
    EpiArgs e{};
    e.M = n;
    e.N = p.ldg;
    e.alpha = 1.0f;
    e.d_kind = a.bf16 ? OUT_BF16 : OUT_F16;
    e.D = p.G;
    e.ldd = p.ldg;
    e.vec = 1;
    return e;
}

__device__ STG_AI inline GroupedArgs logits_args(const XentArgs &a, const XentPiece &p)
{
    GroupedArgs g{};
    g.N = p.n;
    g.A = a.Xc;
    g.lda = a.hp;
    g.B = p.W;
    g.ldb = p.ldw;
    return g;
}

template <class OP, bool GRAD, int BM, int BN>
__global__ __launch_bounds__(512, BM * BN >= 256 * 128 ? 2 : 4) void k_xent_tiled(XentArgs a,
                                                                                 XentPiece p,
                                                                                 int tiles_n)
{
    constexpr int AB = region_bytes<BM / 2, BN / 4>(), BB = region_bytes<BN / 2, BN / 4>();
    __shared__ __attribute__((aligned(1024))) uint8_t a00[AB], a10[AB], a01[AB], a11[AB], b00[BB],
        b10[BB], b01[BB], b11[BB];
    const Regions L = {a00, a10, a01, a11, b00, b10, b01, b11};
    typedef TileShape<OP, false, GL_K, GL_K, BM, BN> S;
    static_assert(AB >= 4 * BM * 4 && AB >= S::GN * BM * 8, "rows' values");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = __builtin_amdgcn_readfirstlane(*a.count), tiles_m = (n + BM - 1) / BM;
    const int id = xcd_tile(blockIdx.x, tiles_m * tiles_n);
    if (id < 0)
        return;
    int tm, tn;
    tile_of(id, tiles_m, tiles_n, tm, tn);
    const int64_t m = wave_uniform((int64_t)tm * BM), c = wave_uniform((int64_t)tn * BN);
    typename OP::acc_t acc[S::FM][S::FN];
    const GroupRows t = {0, 0, n, 0};
    tile_sum<OP, false, GL_K, GL_K, BM, BN>(logits_args(a, p), t, m, c, n, a.hp, a.hp, lane, wave, L,
                                            acc);
    if constexpr (GRAD) {
        tile_g<OP, S>(a, p, n, m, c, acc, lane, wave, (float *)a00);
        store_acc<OP, S>(g_epilogue(a, p, n), 0, m, c, acc, lane, wave, wave_slab(L, wave));
    } else {
        tile_stats<OP, S>(a, p, n, m, c, tn, acc, lane, wave, (int *)a00, (float *)a10);
    }
}

template <class OP, bool GRAD>
__global__ __launch_bounds__(256, 2) void k_xent_small(XentArgs a, XentPiece p, int tiles_n)
{
    __shared__ __attribute__((aligned(1024))) uint8_t s0[16384], s1[16384], s2[16384], s3[16384];
    typedef SmallShape<OP, false, GL_K, GL_K> S;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = __builtin_amdgcn_readfirstlane(*a.count), tiles_m = (n + 63) / 64;
    const int id = xcd_tile(blockIdx.x, tiles_m * tiles_n);
    if (id < 0)
        return;
    int tm, tn;
    tile_of(id, tiles_m, tiles_n, tm, tn);
    const int64_t m = wave_uniform((int64_t)tm * 64), c = wave_uniform((int64_t)tn * 64);
    typename OP::acc_t acc[2][2];
    const GroupRows t = {0, 0, n, 0};
    small_sum<OP, false, GL_K, GL_K>(logits_args(a, p), t, m, c, n, a.hp, a.hp, lane, wave, s0, s1, s2,
                                     s3, acc);
    if constexpr (GRAD) {
        tile_g<OP, S>(a, p, n, m, c, acc, lane, wave, (float *)s0);
        uint8_t *slab = wave == 0 ? s0 : wave == 1 ? s1 : wave == 2 ? s2 : s3;
        store_acc<OP, S>(g_epilogue(a, p, n), 0, m, c, acc, lane, wave, (uint32_t *)slab);
    } else {
        tile_stats<OP, S>(a, p, n, m, c, tn, acc, lane, wave, (int *)s0, (float *)s1);
    }
}

template <class OP, bool GRAD>
static hipError_t launch_t(int tile, const XentArgs &a, const XentPiece &p, hipStream_t s)
{
    const int64_t b = xent_edge(tile);
    const int tiles_n = (int)((p.n + b - 1) / b);
    const dim3 grid((unsigned)(((a.tokens + b - 1) / b * tiles_n + 7) / 8 * 8));
    if (tile == XT_256)
        hipLaunchKernelGGL((k_xent_tiled<OP, GRAD, 256, 256>), grid, dim3(512), 0, s, a, p, tiles_n);
    else if (tile == XT_128)
        hipLaunchKernelGGL((k_xent_tiled<OP, GRAD, 128, 128>), grid, dim3(512), 0, s, a, p, tiles_n);
    else
        hipLaunchKernelGGL((k_xent_small<OP, GRAD>), grid, dim3(256), 0, s, a, p, tiles_n);
    return hipGetLastError();
}

hipError_t launch_xent_stats(int tile, const XentArgs &a, const XentPiece &p, hipStream_t s)
{
    return a.bf16 ? launch_t<Op16BF16, false>(tile, a, p, s) : launch_t<Op16F16, false>(tile, a, p, s);
}

hipError_t launch_xent_g(int tile, const XentArgs &a, const XentPiece &p, hipStream_t s)
{
    return a.bf16 ? launch_t<Op16BF16, true>(tile, a, p, s) : launch_t<Op16F16, true>(tile, a, p, s);
}

} // namespace stg

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

// x in the places of the tile's columns behind the piece's last one; col: the
// lane's first column in the tile.
template <class OP, class S>
__device__ STG_AI inline void mask_columns(const XentPiece &p, int64_t n_blk, int col,
                                           typename OP::acc_t (&acc)[S::FM][S::FN], float x)
{
    if (n_blk + S::BN <= p.n)
        return;
    const int left = (int)(p.n - n_blk) - col;
#pragma unroll
    for (int j = 0; j < S::FN; ++j)
        if (16 * j >= left)
#pragma unroll
            for (int i = 0; i < S::FM; ++i)
                acc[i][j] = typename OP::acc_t{x, x, x, x};
}

// What the tile's epilogue needs of the row of thread tid (the first BM of a
// workgroup), loaded before the tile's sums so that nothing waits for it.
struct RowVals {
    int tgt; // target relative to the tile's columns
    float ca, cb, cl;
    Gmax gmax;
};
template <bool GRAD, int BM>
__device__ STG_AI inline RowVals load_row(const XentArgs &a, const XentPiece &p, int n, int64_t m_blk,
                                          int64_t n_blk, int tid)
{
    const int64_t row = m_blk + tid;
    RowVals v = {-1, 0.0f, 0.0f, 0.0f, {}};
    if (tid < BM && row < n) {
        v.tgt = (int)(xent_row_target(a, row) - (p.v0 + n_blk));
        if constexpr (GRAD) {
            v.ca = a.ca[row];
            v.cb = a.cb[row];
            v.cl = a.cl[row];
        }
    }
    if constexpr (GRAD)
        v.gmax = load_gmax(a, threadIdx.x & 63);
    return v;
}

// Statistics of the tile at (m_blk, n_blk), tile column tn; n: rows.  lds: BM
// ints, GN * BM pairs of floats (16-byte aligned).
template <class OP, class S>
__device__ STG_AI inline void tile_stats(const XentArgs &a, const XentPiece &p, int n, int64_t m_blk,
                                         int64_t n_blk, int tn, const RowVals &row,
                                         typename OP::acc_t (&acc)[S::FM][S::FN], int lane, int wave,
                                         int *tgt, float *st)
{
    static_assert(S::PA == 1 && S::PB == 1, "a wave's block is one piece");
    const int tid = threadIdx.x, l16 = lane & 15, q = lane >> 4;
    const int rb = wave / S::GN * S::WM, cb = wave % S::GN * S::WN;
    if (tid < S::BM)
        tgt[tid] = row.tgt;
    if (a.scale != 1.0f)
#pragma unroll
        for (int i = 0; i < S::FM; ++i)
#pragma unroll
            for (int j = 0; j < S::FN; ++j)
                acc[i][j] *= a.scale;
    mask_columns<OP, S>(p, n_blk, cb + l16, acc, -INFINITY);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
        const i4_t tg = *(const i4_t *)(tgt + rb + 16 * i + 4 * q);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float m = acc[i][0][r], s = 0.0f;
#pragma unroll
            for (int j = 1; j < S::FN; ++j)
                m = __builtin_fmaxf(m, acc[i][j][r]);
            const int d = tg[r] - cb - l16;
            if ((uint32_t)d < (uint32_t)S::WN && (d & 15) == 0) {
                float x = acc[i][0][r];
#pragma unroll
                for (int j = 1; j < S::FN; ++j)
                    x = d >> 4 == j ? acc[i][j][r] : x;
                a.zt[m_blk + rb + 16 * i + 4 * q + r] = x;
            }
            m = max16(m);
            const float ref = sum_ref(m);
#pragma unroll
            for (int j = 0; j < S::FN; ++j)
                s += __builtin_amdgcn_exp2f((acc[i][j][r] - ref) * LOG2E);
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
        const float ref = sum_ref(m);
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
__device__ STG_AI inline void tile_g(const XentArgs &a, const XentPiece &p, int64_t n_blk,
                                     const RowVals &row, typename OP::acc_t (&acc)[S::FM][S::FN],
                                     int lane, int wave, float *rows)
{
    static_assert(S::PA == 1 && S::PB == 1, "a wave's block is one piece");
    const int tid = threadIdx.x, l16 = lane & 15, q = lane >> 4;
    const int rb = wave / S::GN * S::WM, cb = wave % S::GN * S::WN;
    const float gmax = xent_gmax(a, row.gmax, lane), f = xent_unit(a);
    if (tid < S::BM) {
        rows[tid] = row.ca / gmax * f;
        rows[S::BM + tid] = row.cb / gmax * f;
        rows[2 * S::BM + tid] = row.cl;
        ((int *)rows)[3 * S::BM + tid] = row.tgt;
    }
    __syncthreads();
    const float k = a.scale * LOG2E;
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
        const float *at = rows + rb + 16 * i + 4 * q;
        const f4_t ca = *(const f4_t *)at, cl = *(const f4_t *)(at + 2 * S::BM);
        const i4_t tg = *(const i4_t *)(at + 3 * S::BM);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int j = 0; j < S::FN; ++j)
                acc[i][j][r] =
                    ca[r] * __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r], k, -cl[r]));
            const int d = tg[r] - cb - l16;
            if ((uint32_t)d < (uint32_t)S::WN && (d & 15) == 0) {
                const float x = at[S::BM + r];
#pragma unroll
                for (int j = 0; j < S::FN; ++j)
                    acc[i][j][r] -= d >> 4 == j ? x : 0.0f;
            }
        }
    }
    mask_columns<OP, S>(p, n_blk, cb + l16, acc, 0.0f);
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
    g.A = a.direct ? a.X : a.Xc;
    g.lda = a.direct ? a.ldx : a.ldc;
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
    const int n = xent_rows(a), tiles_m = (n + BM - 1) / BM;
    const int id = xcd_tile(blockIdx.x, tiles_m * tiles_n);
    if (id < 0)
        return;
    int tm, tn;
    tile_of(id, tiles_m, tiles_n, tm, tn);
    const int64_t m = wave_uniform((int64_t)tm * BM), c = wave_uniform((int64_t)tn * BN);
    typename OP::acc_t acc[S::FM][S::FN];
    const GroupRows t = {0, 0, n, 0};
    const RowVals row = load_row<GRAD, BM>(a, p, n, m, c, threadIdx.x);
    tile_sum<OP, false, GL_K, GL_K, BM, BN>(logits_args(a, p), t, m, c, n, a.hp, a.hp, lane, wave, L,
                                            acc);
    if constexpr (GRAD) {
        tile_g<OP, S>(a, p, c, row, acc, lane, wave, (float *)a00);
        store_acc<OP, S>(g_epilogue(a, p, n), 0, m, c, acc, lane, wave, wave_slab(L, wave));
    } else {
        tile_stats<OP, S>(a, p, n, m, c, tn, row, acc, lane, wave, (int *)a00, (float *)a10);
    }
}

template <class OP, bool GRAD>
__global__ __launch_bounds__(256, 2) void k_xent_small(XentArgs a, XentPiece p, int tiles_n)
{
    __shared__ __attribute__((aligned(1024))) uint8_t s0[16384], s1[16384], s2[16384], s3[16384];
    typedef SmallShape<OP, false, GL_K, GL_K> S;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = xent_rows(a), tiles_m = (n + 63) / 64;
    const int id = xcd_tile(blockIdx.x, tiles_m * tiles_n);
    if (id < 0)
        return;
    int tm, tn;
    tile_of(id, tiles_m, tiles_n, tm, tn);
    const int64_t m = wave_uniform((int64_t)tm * 64), c = wave_uniform((int64_t)tn * 64);
    typename OP::acc_t acc[2][2];
    const GroupRows t = {0, 0, n, 0};
    const RowVals row = load_row<GRAD, 64>(a, p, n, m, c, threadIdx.x);
    small_sum<OP, false, GL_K, GL_K>(logits_args(a, p), t, m, c, n, a.hp, a.hp, lane, wave, s0, s1, s2,
                                     s3, acc);
    if constexpr (GRAD) {
        tile_g<OP, S>(a, p, c, row, acc, lane, wave, (float *)s0);
        uint8_t *slab = wave == 0 ? s0 : wave == 1 ? s1 : wave == 2 ? s2 : s3;
        store_acc<OP, S>(g_epilogue(a, p, n), 0, m, c, acc, lane, wave, (uint32_t *)slab);
    } else {
        tile_stats<OP, S>(a, p, n, m, c, tn, row, acc, lane, wave, (int *)s0, (float *)s1);
    }
}

// Up to 16 rows: W's stream is the time.  A wave takes groups of 16 columns in
// turn and copies their K tiles (128 values of 16 columns, 4 KB, 256-byte runs)
// into LDS buffers of its own, three ahead and on into the next group, so that
// the stream stops neither for a barrier nor for an epilogue; X's fragments come
// from L2 beside them.  The statistics are kept per lane while the groups pass,
// the running maximum and the sum relative to it, and joined once at the end:
// one pair per row and workgroup.  Every step has eight (LOOSE: nine)
// vector-memory instructions (past the last one they load zeros without touching
// memory), so a step's have arrived when those of three newer steps are left.
// A wave begins each row at a K tile of its own and goes round (rows of 4096 bytes
// lie alike in the memory's channels, and all waves read the same ones at a time
// otherwise), and an XCD's waves take neighbouring groups.  One row, 32768 x 2048
// (128 MB not in the caches; a plain read of it takes 21 us): the pass 25.3 us,
// without the latter 27.1, without either 33.4; then also with 64-value tiles and
// eight buffers 34.2, with five buffers 35.7, with 64 x 64 tiles 37.0; with four
// times the workgroups, 131072 columns of 4096 207 us for 202.
// LOOSE: W's rows begin at any element.  The copies then begin at the 16 bytes
// that hold a row's first value (all groups of 16 rows lie alike in them) and
// take one piece more, and the fragments are read by dwords from where they
// begin; what lies behind a row is masked.  Four rows, 196647 x 1909,
// fp16: 141 us (5.3 TB/s; a copy of W and the pass over it took 475, unaligned
// loads into registers 455).
constexpr int ST_BUF = 4;
template <class OP, bool GRAD, bool LOOSE>
__global__ __launch_bounds__(256, 2) void k_xent_stream(XentArgs a, XentPiece p, int all_groups)
{
    constexpr bool BF = std::is_same<OP, Op16BF16>::value;
    constexpr int DMAS = LOOSE ? 5 : 4, SB = DMAS * 1024; // copies of a step, their bytes
    __shared__ __attribute__((aligned(1024))) uint8_t b0[4 * SB], b1[4 * SB], b2[4 * SB], b3[4 * SB];
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // every XCD takes an eighth of the groups, its waves every `waves`th of them
    const int xcds = gridDim.x % 8 ? 1 : 8, share = (all_groups + xcds - 1) / xcds;
    const int waves = gridDim.x / xcds * 4;
    const int g0 = blockIdx.x % xcds * share + blockIdx.x / xcds * 4 + wave;
    const int groups = min(all_groups, (int)(blockIdx.x % xcds + 1) * share);
    const int n = xent_rows(a), KT = (int)((a.hp + 127) / 128);
    const int64_t kb = a.hp * 2, ldw = p.ldw * 2, lda = (a.direct ? a.ldx : a.ldc) * 2;
    const __amdgpu_buffer_rsrc_t ra =
        tile_rsrc(a.direct ? a.X : a.Xc, n > 0 ? (n - 1) * lda + kb : 0);
    auto buf = [&](auto slot) STG_AI {
        constexpr int S = decltype(slot)::value;
        return (S == 0 ? b0 : S == 1 ? b1 : S == 2 ? b2 : b3) + wave * SB;
    };
    if (n == 0)
        return;
    // (row l16's values; past the end the last row's, unused)
    const RowVals row = load_row<GRAD, 16>(a, p, n, 0, 0, min(l16, n - 1));
    // the step whose copies are issued next, and the one that is multiplied
    const int va = l16 * (int)lda + q * 16;
    const int turn = g0 % KT;
    int ig = g0, it = turn;
    u4_t fa[ST_BUF][4];
    const int skew = LOOSE ? (int)((uintptr_t)p.W & 15) : 0; // of the first row
    const int hb = (int)a.hidden * 2, lw = (int)ldw;
    // this lane's piece of copy d: byte in the group's rows, and what is left of
    // its row from there
    int piece[DMAS], left[DMAS];
#pragma unroll
    for (int d = 0; d < DMAS; ++d) {
        const int row = d < 4 ? 4 * d + q : l16, chunk = d < 4 ? (l16 ^ row) * 16 : 256;
        const int at = row * lw + skew;
        piece[d] = (LOOSE ? at & ~15 : at) + chunk;
        left[d] = d < 4 || lane < 16 ? (LOOSE ? hb + (at & 15) : (int)kb) - chunk : 0;
    }
    // LOOSE: this lane's fragment begins `sub` bytes into dword `dw` of its 16 bytes
    const int dw = ((l16 * lw + skew) & 15) >> 2, sub = (l16 * lw + skew) & 2;
    auto issue = [&](auto slot) STG_AI {
        constexpr int S = decltype(slot)::value;
        const bool in = ig < groups;
        const int64_t c = (int64_t)ig * 16;
        const __amdgpu_buffer_rsrc_t rb =
            epi_rsrc((const uint8_t *)p.W - skew + (in ? c * ldw : 0),
                     in ? LOOSE ? ((p.n - c - 1) * ldw + hb + skew + 15) & ~(int64_t)15
                                : (p.n - c - 1) * ldw + kb
                        : 0);
#pragma unroll
        for (int d = 0; d < DMAS; ++d)
            dma16(rb, buf(slot) + 1024 * d, it * 256 < left[d] ? piece[d] : (int)0x80000000, it * 256);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool ain = in && it * 256 + 64 * k + q * 16 < kb;
            fa[S][k] = buf_load16(ra, ain ? va + 64 * k : (int)0x80000000, it * 256);
        }
        it = it + 1 < KT ? it + 1 : 0;
        ig += it == turn ? waves : 0;
    };
    auto all = [&](auto &&f) STG_AI {
        [&]<int... I>(std::integer_sequence<int, I...>) STG_AI {
            (f(std::integral_constant<int, I>{}), ...);
        }(std::make_integer_sequence<int, ST_BUF>{});
    };
    in_order();
    all(issue);
    in_order();
    // rows 4 q .. 4 q + 3 are this lane's accumulators
    float ca[4], cb[4], cl[4], m[4], s[4];
    int tgt[4];
    float gmax = 0.0f;
    if constexpr (GRAD)
        gmax = xent_gmax(a, row.gmax, lane);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        tgt[r] = __shfl(row.tgt, 4 * q + r);
        tgt[r] = 4 * q + r < n ? tgt[r] : -1;
        m[r] = -INFINITY;
        s[r] = 0.0f;
        if constexpr (GRAD) {
            const float f = xent_unit(a);
            ca[r] = __shfl(row.ca, 4 * q + r) / gmax * f;
            cb[r] = __shfl(row.cb, 4 * q + r) / gmax * f;
            cl[r] = __shfl(row.cl, 4 * q + r);
        }
    }
    int g = g0, t = turn;
    // (four sums of a quarter of the values each: their roundings are smaller
    // than one sum's, and no product waits for the one before)
    typename OP::acc_t part[4] = {};
    auto finish = [&]() STG_AI { // a group's logits: rows 4 q + r, column l16
        const int col = g * 16 + l16;
        const typename OP::acc_t acc = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            part[k] = typename OP::acc_t{};
        if (g >= groups)
            return;
        if constexpr (GRAD) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float x = ca[r] * __builtin_amdgcn_exp2f(__builtin_fmaf(acc[r], a.scale * LOG2E, -cl[r]));
                x -= tgt[r] == col ? cb[r] : 0.0f;
                x = col < p.n ? x : 0.0f;
                if (4 * q + r < n)
                    p.G[(4 * q + r) * p.ldg + col] = BF ? f32_to_bf16_bits(x) : f32_to_f16_bits(x);
            }
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float z = acc[r] * a.scale;
                if (tgt[r] == col)
                    a.zt[4 * q + r] = z;
                const float x = col < p.n ? z : -INFINITY, mx = __builtin_fmaxf(m[r], x);
                const float ref = sum_ref(mx);
                s[r] = s[r] * __builtin_amdgcn_exp2f((m[r] - ref) * LOG2E) +
                       __builtin_amdgcn_exp2f((x - ref) * LOG2E);
                m[r] = mx;
            }
        }
    };
    auto step = [&](auto slot) STG_AI {
        constexpr int S = decltype(slot)::value;
        in_order();
        STG_WAIT_VMCNT((ST_BUF - 1) * (DMAS + 4));
        in_order();
        u4_t fb[4], x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint8_t *const b = buf(slot);
            if constexpr (LOOSE) {
                uint32_t w[5];
#pragma unroll
                for (int i = 0; i < 5; ++i) {
                    const int chunk = 4 * k + q + ((dw + i) >> 2), in = ((dw + i) & 3) * 4;
                    w[i] = *(const uint32_t *)(b + in + (chunk < 16 ? l16 * 256 + ((chunk ^ l16) << 4)
                                                                    : 4096 + l16 * 16));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    fb[k][i] = __builtin_amdgcn_alignbyte(w[i + 1], w[i], sub);
            } else {
                fb[k] = *(const u4_t *)(b + l16 * 256 + (((4 * k + q) ^ l16) << 4));
            }
            x[k] = fa[S][k];
        }
        wave_lds_sync(); // read before the buffer is copied into again
        if (LOOSE && t == KT - 1)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int n = (int)a.hidden - (t * 128 + 32 * k + 8 * q); // values of the row
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    fb[k][i] &= (2 * i < n ? 0xFFFFu : 0u) | (2 * i + 1 < n ? 0xFFFF0000u : 0u);
            }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            part[k] = OP::mma((const uint32_t *)&x[k], (const uint32_t *)&fb[k], part[k]);
        in_order();
        issue(slot);
        in_order();
        t = t + 1 < KT ? t + 1 : 0;
        if (t == turn) {
            finish();
            g += waves;
        }
    };
    // (without conditions between the steps, from which the compiler would take
    // that fewer loads may be in flight: those past the last group multiply zeros)
    while (g < groups)
        all(step);
    STG_WAIT_VMCNT(0); // copies past the last step, before LDS is reused
    if constexpr (!GRAD) {
        __syncthreads();
        float *st = (float *)b0;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float mx = max16(m[r]), ref = sum_ref(mx);
            const float sum = sum16(s[r] * __builtin_amdgcn_exp2f((m[r] - ref) * LOG2E));
            if (l16 == 0) {
                st[(wave * 16 + 4 * q + r) * 2] = mx;
                st[(wave * 16 + 4 * q + r) * 2 + 1] = sum;
            }
        }
        __syncthreads();
        if (threadIdx.x < n) {
            float mx = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                mx = __builtin_fmaxf(mx, st[(w * 16 + threadIdx.x) * 2]);
            const float ref = sum_ref(mx);
#pragma unroll
            for (int w = 0; w < 4; ++w)
                sum += st[(w * 16 + threadIdx.x) * 2 + 1] *
                       __builtin_amdgcn_exp2f((st[(w * 16 + threadIdx.x) * 2] - ref) * LOG2E);
            float *o = a.part + ((p.tile0 + blockIdx.x) * a.tokens + threadIdx.x) * 2;
            o[0] = mx;
            o[1] = sum;
        }
    }
}

template <class OP, bool GRAD>
static hipError_t launch_t(int tile, const XentArgs &a, const XentPiece &p, hipStream_t s)
{
    if (tile == XT_STREAM) {
        const dim3 grid((unsigned)xent_streams(p.n, a.dx.num_cu));
        const int groups = (int)((p.n + 15) / 16);
        if constexpr (!GRAD)
            if (p.loose) {
                hipLaunchKernelGGL((k_xent_stream<OP, GRAD, true>), grid, dim3(256), 0, s, a, p,
                                   groups);
                return hipGetLastError();
            }
        hipLaunchKernelGGL((k_xent_stream<OP, GRAD, false>), grid, dim3(256), 0, s, a, p, groups);
        return hipGetLastError();
    }
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

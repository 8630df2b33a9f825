// Linear cross entropy: the two products of the logits' gradient G, on the
// grouped products' main loop (grouped_tiled.hpp).
//  - dX: acc[split] (+)= G W over a part of the piece's columns, fp32 in the
//    workspace (the pieces add up there; splits fill the chip where there are
//    few tiles), joined and rounded by k_xent_out;
//  - dW = G^T X: the sum runs over all rows, so a piece's part of dW is
//    complete and rounded at once.
#include "grouped_tiled.hpp"
#include "vec16.hpp"
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

// The lane beside this one's value (1, 0, 3, 2 of each four).
__device__ STG_AI inline u4_t other_lane(u4_t x)
{
    u4_t y;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x[i], 0xB1, 0xF, 0xF, true);
    return y;
}

// dW for up to 128 rows, where its stores are the time.  A wave owns 128 of X's
// columns, whose fragments (the rows are the sum's axis) stay in registers, and
// walks down a range of the vocabulary, 64 rows of dW a step: G's next 64
// columns are copied into an LDS buffer of its own while this step's products
// are stored.  X is the MFMA's first operand, with its columns in an order that
// leaves eight neighbouring values of a row of dW in a lane, so they are stored
// from the registers: lanes of two neighbouring rows exchange 16 bytes first,
// and an instruction writes eight whole cache lines.  No barrier, and a step's
// stores are still on their way while the next one multiplies.  bf16 dW: 40 rows,
// 131072 x 4096, 223 us (4.8 TB/s; tiles of 256 x 256 357, of which little is
// the product; 64 bytes of a line at a time 353, and through the caches 237 with
// what they hold written in the next kernel's time); 93, 52696 x 2048, 45 us
// (96); 16, 48 us (73).
template <class OP, int KT, int DK, bool ADD, int CPOL>
__global__ __launch_bounds__(256, KT == 1 ? 2 : 1) void k_xent_dw_rows(XentArgs a, XentPiece p,
                                                                      XentDw d, int blocks, int per,
                                                                      int wgs)
{
    constexpr bool BF = std::is_same<OP, Op16BF16>::value;
    constexpr int KS = 2 * KT, ES = DK == OUT_F32 ? 4 : 2, NV = ES / 2;
    constexpr int RB = 64 * 128;                     // bytes of 64 rows of G's 64 columns
    constexpr int STORES = 4 * 4 * NV;               // of a step
    __shared__ __attribute__((aligned(1024))) uint8_t b0[4 * KT * RB], b1[4 * KT * RB];
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int id = xcd_tile(blockIdx.x, wgs);
    if (id < 0)
        return;
    const int w = id * 4 + wave, h0 = w % blocks * 128;
    const int64_t v0 = wave_uniform((int64_t)(w / blocks) * per * 64);
    const int64_t v1 = wave_uniform(min(p.n, v0 + (int64_t)per * 64));
    if (v0 >= v1)
        return;
    const int n = __builtin_amdgcn_readfirstlane(*a.count);
    const Gmax first = load_gmax(a, lane);
    typedef Operand<GL_MN, 64, 64, BF, 1, 1, 1> OpG;
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    OpG G;
    G.ld = p.ldg * 2;
    G.k_bytes = n;
    G.base = (const uint8_t *)(p.G + v0);
    G.span = (chunks8(p.n) - v0) * 2;
    G.init(lane, 0, 0);
    auto buf = [&](auto slot) STG_AI {
        return (decltype(slot)::value == 0 ? b0 : b1) + wave * (KT * RB);
    };
    auto copy = [&](auto slot, int64_t v) STG_AI {
        G.base = (const uint8_t *)(p.G + v);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
            G.copy(buf(slot) + kt * RB, I0{}, kt, 0);
    };
    copy(I0{}, v0);
    // fragment i, its row l16: column h0 + 32 (i / 2) + 8 (l16 / 4) + 4 (i % 2)
    // + l16 % 4, so that rows 4 q .. 4 q + 3 of fragments 2 g and 2 g + 1 are
    // columns h0 + 32 g + 8 q .. + 7
    // (zeros behind the last row; columns behind the last one are not stored)
    const __amdgpu_buffer_rsrc_t rx = epi_rsrc(a.Xc, n * a.ldc * 2);
    const int ldc = (int)a.ldc * 2;
    const int x0 = 8 * q * ldc + (h0 + 8 * (l16 >> 2) + (l16 & 3)) * 2;
    u4_t x[8][KS];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                e[j] = __builtin_amdgcn_raw_buffer_load_b16(
                    rx, x0 + 64 * (i >> 1) + 8 * (i & 1) + j * ldc, 32 * s * ldc, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[i][s][j] = e[2 * j] | e[2 * j + 1] << 16;
        }
    const float f = xent_factor(a, first, lane);
    const int ldd = (int)d.ldd * ES;
    // this lane's bytes of the step's first 16 rows: its values' (their first
    // and second 16 bytes for fp32), and of the two stores after an exchange
    // with the lane beside it.  Pair m: columns 64 m + 8 q and 32 behind them,
    // for fp32 32 m + 8 q and 4 behind.
    constexpr int PAIRS = 2 * NV, NEXT = NV == 2 ? 4 : 32, PAIR = NV == 2 ? 32 : 64;
    auto byte_of = [&](int row, int c) STG_AI {
        return c < a.hidden ? row * ldd + c * ES : (int)0x80000000;
    };
    int at[PAIRS], own[PAIRS][2];
#pragma unroll
    for (int m = 0; m < PAIRS; ++m) {
        const int c = h0 + PAIR * m + 8 * q;
        at[m] = byte_of(l16 & ~1, c + (l16 & 1) * NEXT);
        own[m][0] = byte_of(l16, c);
        own[m][1] = byte_of(l16, c + NEXT);
    }
    in_order();
    STG_WAIT_VMCNT(0);
    in_order();

    auto step = [&](auto slot, int64_t v) STG_AI {
        constexpr int P = decltype(slot)::value;
        // (behind the range: copied, not used)
        if (v + 64 < p.n)
            copy(std::integral_constant<int, 1 - P>{}, v + 64);
        const __amdgpu_buffer_rsrc_t rd = epi_rsrc((uint8_t *)d.dW + v * ldd,
                                                   (p.n - v - 1) * ldd + a.hidden * ES);
        // (offsets of rows are added to the lanes': behind a 16-byte store that
        // takes one from a scalar register the compiler overwrites the stored
        // registers at once, and the card then stored what they became)
        u4_t old[2][PAIRS][2];
        auto load_old = [&](auto bc, int r) STG_AI {
            if constexpr (ADD)
#pragma unroll
                for (int m = 0; m < PAIRS; ++m)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        old[decltype(bc)::value][m][k] = buf_load16(rd, own[m][k] + 16 * r * ldd, 0);
        };
        auto rows = [&](auto bc, int r) STG_AI {
            u4_t fg[KS];
            in_order();
#pragma unroll
            for (int s = 0; s < KS; ++s)
                fg[s] = G.read(buf(slot) + s / 2 * RB, r, s % 2);
            in_order();
            __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt(0)
            __builtin_amdgcn_sched_barrier(0);
            typename OP::acc_t acc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[i] = typename OP::acc_t{};
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    acc[i] = OP::mma((const uint32_t *)&x[i][s], (const uint32_t *)&fg[s], acc[i]);
            }
#pragma unroll
            for (int m = 0; m < PAIRS; ++m) {
                u4_t z[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if constexpr (DK == OUT_F32) {
                        f4_t y = acc[2 * m + k] * f;
                        if constexpr (ADD)
                            y += __builtin_bit_cast(f4_t, old[decltype(bc)::value][m][k]);
                        z[k] = __builtin_bit_cast(u4_t, y);
                    } else {
                        float y[8], o[8] = {};
                        if constexpr (ADD)
                            widen8<DK == OUT_BF16>(old[decltype(bc)::value][m][k], o);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            y[e] = acc[4 * m + 2 * k + (e >> 2)][e & 3] * f;
                            if constexpr (ADD)
                                y[e] += o[e];
                        }
                        z[k] = narrow8<DK == OUT_BF16>(y);
                    }
                }
                // the even row's two pieces, then the odd one's
                const bool odd = l16 & 1;
                const u4_t other = other_lane(odd ? z[0] : z[1]);
                const u4_t even_row = odd ? other : z[0], odd_row = odd ? z[1] : other;
                const int to = at[m] + 16 * r * ldd;
                __builtin_amdgcn_raw_buffer_store_b128(even_row, rd, to, 0, CPOL);
                __builtin_amdgcn_raw_buffer_store_b128(odd_row, rd, to + ldd, 0, CPOL);
            }
        };
        load_old(I0{}, 0);
        load_old(I1{}, 1);
        rows(I0{}, 0);
        load_old(I0{}, 2);
        rows(I1{}, 1);
        load_old(I1{}, 3);
        rows(I0{}, 2);
        rows(I1{}, 3);
        in_order();
        STG_WAIT_VMCNT(STORES); // the next step's copies: older than this one's stores
        in_order();
    };
    for (int64_t v = v0; v < v1; v += 128) {
        step(I0{}, v);
        if (v + 64 < v1)
            step(I1{}, v + 64);
    }
    STG_WAIT_VMCNT(0); // copies on their way, before LDS is another's
}

template <class OP, int KT>
static hipError_t launch_rows(const XentArgs &a, const XentPiece &p, const XentDw &d, hipStream_t s)
{
    const int blocks = (int)((a.hp + 127) / 128), steps = (int)((p.n + 63) / 64);
    const int waves = (KT == 1 ? 8 : 4) * a.dx.num_cu;
    int ranges = waves / blocks > 1 ? waves / blocks : 1;
    const int per = (steps + ranges - 1) / ranges;
    ranges = (steps + per - 1) / per;
    const int wgs = (blocks * ranges + 3) / 4;
    const dim3 grid((unsigned)((wgs + 7) / 8 * 8));
    auto go = [&](auto kind, auto add, auto cpol) {
        hipLaunchKernelGGL((k_xent_dw_rows<OP, KT, decltype(kind)::value, decltype(add)::value,
                                           decltype(cpol)::value>),
                           grid, dim3(256), 0, s, a, p, d, blocks, per, wgs);
    };
    auto lines = [&](auto kind, auto add) {
        if (d.whole_lines)
            go(kind, add, std::integral_constant<int, EPI_CPOL>{});
        else
            go(kind, add, std::integral_constant<int, 0>{});
    };
    auto kind = [&](auto k) {
        if (d.add)
            lines(k, std::true_type{});
        else
            lines(k, std::false_type{});
    };
    if (d.d_kind == OUT_F32)
        kind(std::integral_constant<int, OUT_F32>{});
    else if (d.d_kind == OUT_F16)
        kind(std::integral_constant<int, OUT_F16>{});
    else
        kind(std::integral_constant<int, OUT_BF16>{});
    return hipGetLastError();
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
    if (tile == XT_STREAM) {
        if (a.tokens <= 64)
            return a.bf16 ? launch_rows<Op16BF16, 1>(a, p, d, s) : launch_rows<Op16F16, 1>(a, p, d, s);
        return a.bf16 ? launch_rows<Op16BF16, 2>(a, p, d, s) : launch_rows<Op16F16, 2>(a, p, d, s);
    }
    return a.bf16 ? launch_t<Op16BF16, true>(tile, a, p, XentDx{}, d, s)
                  : launch_t<Op16F16, true>(tile, a, p, XentDx{}, d, s);
}

} // namespace stg

// The LDS-tiled grouped product (gemm_moe.h, "grouped products") for 16-bit
// operands on the 16x16x32 MFMA forms: k_grouped_tiled.
//
// A workgroup of eight waves owns a BM x BN tile of one group's output; a
// wave owns a (BM/2) x (BN/4) block of it.  K advances 64 values a tile.
// Both operands go from global memory straight into LDS (16 bytes per lane);
// an operand of a K tile is kept as two regions, the first and the second
// half of every wave's rows (columns), in two buffers, so a K tile is four
// clusters of work, one per quadrant of the wave's block:
//     cluster 0: read A0          MFMA A0 x B0
//     cluster 1: read B1          MFMA A0 x B1
//     cluster 2: read A1          MFMA A1 x B0
//     cluster 3: read the next tile's B0, MFMA A1 x B1
// Each cluster is a memory phase (LDS reads, copies for later) and an MFMA
// phase with a barrier after each.  Waves 0-3 and waves 4-7 -- one of each
// on every SIMD -- run one phase apart, so while one half multiplies the
// other reads, and the matrix pipe is always fed by one of them.
//
// Copies: region R of tile t is read first in cluster n (n = 4t - 1, 4t, 4t
// + 1, 4t + 2 for B0, A0, B1, A1) and is copied in the memory phase of
// cluster n - 6.  With phases counted by barriers, the leading half's
// cluster n reads in phase 2n and the trailing half's in 2n + 1.  What
// cluster n read is in registers by the end of phase 2n + 2 (each MFMA
// phase starts with lgkmcnt(0)), and its place is written again from cluster
// n + 2 on, phase 2n + 4 at the earliest.  A wave waits for its copies of
// cluster n - 6 at the end of its memory phase of cluster n - 1, phase 2n - 1
// at the latest; the barrier there makes them visible to the reads of phase
// 2n and later.
//
// Operand layouts in LDS (both without padding, as the copies need):
//  - K-contiguous (rows of 64 K values = 8 chunks of 16 bytes): chunk c of
//    region row r at slot c ^ (r & 7); a fragment read takes 16 rows at the
//    chunks of four lane groups.
//  - MN-major (64 K rows of the region's columns): 32-byte piece p of K row k
//    at piece p ^ mn_swz(k), chosen so that the eight K rows half a wave
//    touches in one transposing read lie on all eight pieces of a 256-byte
//    window.
// The permutation is applied to the lanes' global addresses.
//
// An 8-bit B (codes and scales of a checkpoint) is loaded into registers
// instead, and brought to 16 bits and stored to LDS four clusters later.
//
// Measured on MI355X (256 x 256 tiles, bf16): one group of 8192^3 1500
// TFLOP/s; rows, 16 groups of 16384 x 4096 x 4096, 483 us, 1138 TFLOP/s (matrix
// pipe busy 65 %, of which the last round of tiles and the padding of ragged
// groups cost about a fifth); weights, 16 groups of 4096 x 2048 fp32 added to
// C over 16384 rows, 370 us, from 8 bits and without C 375 us.
#pragma once
#include "grouped_common.hpp"

namespace stg {

enum { GL_K = 0, GL_MN = 1, GL_Q8 = 2 }; // operand layouts: K-contiguous, MN-major, 8-bit MN-major

// Workgroup id -> tile of `total`, a contiguous run of tiles per XCD (ids go
// round robin over the 8 XCDs); -1 past the end.
__device__ STG_AI inline int xcd_tile(int id, int total)
{
    const int per = (total + 7) >> 3, slot = id >> 3, t = (id & 7) * per + slot;
    return slot < per && t < total ? t : -1;
}

// Tile `t` of tm x tn ones in groups of 8 tile rows walked column by column.
__device__ STG_AI inline void tile_of(int t, int tiles_m, int tiles_n, int &tm, int &tn)
{
    const int per_group = 8 * tiles_n, group = t / per_group, first = group * 8;
    const int rows = min(tiles_m - first, 8), in = t - group * per_group;
    tm = first + in % rows;
    tn = in / rows;
}

// What is left of an operand from p on, [p, end), none if end <= p.  In few
// scalar steps, once per copy (rows left, times the pitch, with 64-bit compares:
// 16 groups of 1024 rows, 4096 x 2048, 392 us and 373 so; one of 5978, 2032
// x 88, 8-bit B, 52.9 and 46.1).
__device__ STG_AI inline __amdgpu_buffer_rsrc_t rest_rsrc(const uint8_t *p, const uint8_t *end)
{
    const int64_t left = end - p;
    const int hi = (int)(left >> 32);
    const uint32_t lo = (uint32_t)left < 0x7fffffffu ? (uint32_t)left : 0x7fffffffu;
    const uint32_t n = (hi > 0 ? 0x7fffffffu : lo) & ~(uint32_t)(hi >> 31);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, (int)n, 0x00020000);
}

// One operand of the tile: where its rows (columns) lie and how it moves.
// LAYOUT: GL_*; R: rows (columns) of a region; PIECE: rows of one wave in it.
// Region row i of half h is tile row at(h, i): K-contiguous operands give each
// wave neighbouring halves, so that its block of the output is one piece; an
// MN-major region is a contiguous run, whose K rows are then fetched in 2 R
// bytes at a time.  SETS: register sets of an 8-bit operand; NW: waves that
// copy; HALVES: 1 for a tile whose operand is one region.
template <int LAYOUT, int R, int PIECE, bool BF, int SETS = 1, int NW = 8, int HALVES = 2>
struct Operand {
    static constexpr bool KC = LAYOUT == GL_K;
    static constexpr int LD = R * 128 / (NW * 1024); // 1 KB copies per wave and region
    static constexpr int VM = LAYOUT == GL_Q8 ? 2 * LD : LD; // vector-memory instructions
    static constexpr int PITCH = R * 2;             // MN-major: bytes of a K row
    static constexpr int CPR = PITCH / 16;          // its 16-byte chunks
    static constexpr int FR = PIECE / 16;           // fragments of a wave
    static constexpr int ROWS = PIECE;
    static_assert(LD >= 1, "a region is at least one copy per wave");

    __device__ STG_AI static int at(int h, int i)
    {
        return KC && HALVES == 2 ? (i / PIECE) * 2 * PIECE + h * PIECE + i % PIECE : h * R + i;
    }

    // (a transposing read touches K rows 8 q + 4 t + 0..3, q = 0, 1 in one
    // half of the wave and 2, 3 in the other)
    __device__ STG_AI static int mn_swz(int k)
    {
        return CPR == 16 ? (k & 3) | (((k >> 3) & 1) << 2) : ((k >> 1) & 1) | (((k >> 3) & 1) << 1);
    }

    const uint8_t *base; // first element of the tile (and of the group's K range)
    int64_t ld;          // bytes between rows (K-contiguous) or K rows
    int64_t k_bytes;     // K-contiguous: bytes of K; MN-major: K rows
    int64_t span;        // K-contiguous: rows that exist; MN-major: bytes of a K row that exist
    const uint8_t *end;  // MN-major: behind the last element that exists
    const uint8_t *sc;   // GL_Q8: scales of the first K row, at the tile's first column's block
    const uint8_t *sc_end;
    int64_t ld_sc;
    int voff[HALVES][LD]; // [half][copy]: byte offset of this lane in the tile
    int soff8[HALVES][LD]; // GL_Q8: offset of its scale
    int kc;              // K-contiguous: byte in the K tile of this lane's chunk
    int rd[FR > 2 ? FR : 2]; // read offsets (K-contiguous: one per K step; else per fragment)
    uint32_t code[SETS][HALVES][LD][2], sbyte[SETS][HALVES][LD]; // GL_Q8: in flight, by half

    // wave_u: the wave's number; part: its place along this operand
    __device__ STG_AI void init(int lane, int wave_u, int part)
    {
        if constexpr (!KC)
            end = base + (k_bytes - 1) * ld + span;
        if constexpr (LAYOUT == GL_Q8)
            sc_end = sc + (k_bytes - 1) * ld_sc + (span + 31) / 32;
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int j = 0; j < LD; ++j) {
                if constexpr (KC) {
                    const int i = (j * NW + wave_u) * 8 + (lane >> 3);
                    const int row = at(h, i);
                    kc = ((lane & 7) ^ ((lane >> 3) & 7)) * 16;
                    voff[h][j] = row * (int)ld + kc;
                } else {
                    const int c = (j * NW + wave_u) * 64 + lane; // chunk of the region
                    const int k = c / CPR;
                    const int i = ((c % CPR) ^ (mn_swz(k) << 1)) * 8; // region column
                    const int col = at(h, i);
                    if constexpr (LAYOUT == GL_Q8) {
                        voff[h][j] = k * (int)ld + col;
                        soff8[h][j] = k * (int)ld_sc + col / 32;
                    } else {
                        voff[h][j] = k * (int)ld + col * 2;
                    }
                }
            }
        const int l16 = lane & 15, q = lane >> 4;
        if constexpr (KC) {
            const int row = part * PIECE + l16;
#pragma unroll
            for (int s = 0; s < 2; ++s)
                rd[s] = row * 128 + (((4 * s + q) ^ (row & 7)) << 4);
        } else {
            const int k = 8 * q + (l16 >> 2), f = mn_swz(k);
#pragma unroll
            for (int r = 0; r < FR; ++r)
                rd[r] = k * PITCH + (((part * FR + r) ^ f) << 5) + (l16 & 3) * 8;
        }
    }

    // Copy half h of K tile kt into `region` (LDS); GL_Q8: into register set Q.
    template <int Q = 0>
    __device__ STG_AI void copy(uint8_t *region, auto half, int kt, int wave_u)
    {
        constexpr int h = decltype(half)::value;
        if constexpr (KC) {
            const __amdgpu_buffer_rsrc_t r = tile_rsrc(base, (span - 1) * ld + k_bytes);
            // chunks past K read zeros: an offset outside every resource
            const bool in = kt * 128 + kc < k_bytes;
#pragma unroll
            for (int j = 0; j < LD; ++j)
                dma16(r, region + (j * NW + wave_u) * 1024, in ? voff[h][j] : (int)0x80000000,
                      kt * 128);
        } else {
            // the tile's K rows start the resource, so that every offset fits
            // 32 bits and K rows past the end lie outside it
            const __amdgpu_buffer_rsrc_t r = rest_rsrc(base + (int64_t)kt * (64 * ld), end);
            if constexpr (LAYOUT == GL_MN) {
#pragma unroll
                for (int j = 0; j < LD; ++j)
                    dma16(r, region + (j * NW + wave_u) * 1024, voff[h][j], 0);
            } else {
                const __amdgpu_buffer_rsrc_t rs = rest_rsrc(sc + (int64_t)kt * (64 * ld_sc), sc_end);
#pragma unroll
                for (int j = 0; j < LD; ++j) {
                    typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
                    const u2_t c = __builtin_bit_cast(
                        u2_t, __builtin_amdgcn_raw_buffer_load_b64(r, voff[h][j], 0, 0));
                    code[Q][h][j][0] = c.x;
                    code[Q][h][j][1] = c.y;
                    sbyte[Q][h][j] = __builtin_amdgcn_raw_buffer_load_b8(rs, soff8[h][j], 0, 0);
                }
            }
        }
    }

    // GL_Q8: half h's codes in register set Q, as 16-bit values into `region`.
    template <int Q = 0>
    __device__ STG_AI void store(uint8_t *region, auto half, int lane, int wave_u)
    {
        constexpr int h = decltype(half)::value;
#pragma unroll
        for (int j = 0; j < LD; ++j) {
            const uint32_t sb = sbyte[Q][h][j];
            u4_t v;
            // scales that cannot take a code past the type's range (448 *
            // 2^(sb - 127)), nor are NaN or subnormal: two values at a time
            if (sb - 1u < (BF ? 246u : 134u)) {
                const float s = __builtin_bit_cast(float, sb << 23);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int c = (int)code[Q][h][j][w >> 1];
                    if constexpr (BF)
                        v[w] = __builtin_bit_cast(
                            uint32_t, w & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, true)
                                            : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, false));
                    else
                        v[w] = __builtin_bit_cast(
                            uint32_t, w & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, s, true)
                                            : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, s, false));
                }
            } else {
                const float s = e8m0(sb);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    typedef float f2_t __attribute__((ext_vector_type(2)));
                    const int c = (int)code[Q][h][j][w >> 1];
                    const f2_t x = w & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(c, true)
                                         : __builtin_amdgcn_cvt_pk_f32_fp8(c, false);
                    const float lo = clamp16<BF>(x.x * s), hi = clamp16<BF>(x.y * s);
                    v[w] = BF ? f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16)
                              : f32_to_f16_bits(lo) | ((uint32_t)f32_to_f16_bits(hi) << 16);
                }
            }
            *(u4_t *)(region + (j * NW + wave_u) * 1024 + lane * 16) = v;
        }
    }

    // Fragment r, K step s of this wave from `region`.
    __device__ STG_AI u4_t read(const uint8_t *region, int r, int s) const
    {
        if constexpr (KC) {
            return *(const u4_t *)(region + rd[s] + r * 16 * 128);
        } else {
            u4_t v;
            lds_read_tr<2>(region + rd[r] + (32 * s) * PITCH, (uint32_t *)&v);
            lds_read_tr<2>(region + rd[r] + (32 * s + 4) * PITCH, (uint32_t *)&v + 2);
            return v;
        }
    }
};

// The LDS regions of a tile, one object per region and buffer: the compiler
// then knows that a copy in flight and a read of another region do not meet.
// [half][buffer] of A, then of B.
struct Regions {
    uint8_t *a00, *a10, *a01, *a11, *b00, *b10, *b01, *b11;
};
// Bytes of a region of R rows (columns): a wave's epilogue slab fits too.
template <int R, int WN>
constexpr int region_bytes()
{
    constexpr int slab = 32 * (WN + 4) * 4;
    return R * 128 > slab ? R * 128 : (slab + 1023) / 1024 * 1024;
}

// A tile's shape and operands: eight waves, 2 x 4, each operand in two halves.
template <class OP, bool W_, int ALAY_, int BLAY_, int BM_, int BN_>
struct TileShape {
    static constexpr bool W = W_, BF = std::is_same<OP, Op16BF16>::value;
    static constexpr int ALAY = ALAY_, BLAY = BLAY_, BM = BM_, BN = BN_;
    static constexpr int GN = 4;                   // waves along N
    static constexpr int WM = BM / 2, WN = BN / 4; // a wave's block
    static constexpr int FM = WM / 16, FN = WN / 16;
    static constexpr int FA = FM / 2, FB = FN / 2; // fragments of one of its halves
    typedef Operand<ALAY, BM / 2, WM / 2, BF> OpA;
    typedef Operand<BLAY, BN / 2, WN / 2, BF> OpB;
    static constexpr int PA = OpA::KC ? 1 : 2, PB = OpB::KC ? 1 : 2; // pieces the block lies in
};
// The 64 x 64 tile: four waves, 2 x 2, each operand one region.
template <class OP, bool W_, int ALAY_, int BLAY_>
struct SmallShape {
    static constexpr bool W = W_, BF = std::is_same<OP, Op16BF16>::value;
    static constexpr int ALAY = ALAY_, BLAY = BLAY_, BM = 64, BN = 64;
    static constexpr int GN = 2, WM = 32, WN = 32, FM = 2, FN = 2;
    typedef Operand<ALAY, BM, WM, BF, 1, 4, 1> OpA;
    typedef Operand<BLAY, BN, WN, BF, 2, 4, 1> OpB;
    static constexpr int PA = 1, PB = 1;
};

// The operands of the tile of group t at (m_blk, n_blk); M, K: its group's
// rows (of the output) and sum.
template <class S>
__device__ STG_AI inline void set_operands(typename S::OpA &A, typename S::OpB &B,
                                           const GroupedArgs &a, const GroupRows &t, int64_t m_blk,
                                           int64_t n_blk, int64_t M, int64_t K, int lane, int wave)
{
    A.ld = a.lda * 2;
    if constexpr (S::ALAY == GL_K) {
        A.base = (const uint8_t *)a.A + (t.r0 + m_blk) * A.ld;
        A.k_bytes = K * 2;
        A.span = M - m_blk;
    } else {
        A.base = (const uint8_t *)a.A + t.r0 * A.ld + m_blk * 2;
        A.k_bytes = K;
        A.span = (M - m_blk) * 2;
    }
    constexpr int BE = S::BLAY == GL_Q8 ? 1 : 2;
    B.ld = a.ldb * BE;
    if constexpr (S::BLAY == GL_K) {
        B.base = (const uint8_t *)a.B + ((int64_t)t.g * a.N + n_blk) * B.ld;
        B.k_bytes = K * 2;
        B.span = a.N - n_blk;
    } else {
        B.base = (const uint8_t *)a.B + (S::W ? t.r0 : (int64_t)t.g * a.K) * B.ld + n_blk * BE;
        B.k_bytes = K;
        B.span = (a.N - n_blk) * BE;
    }
    if constexpr (S::BLAY == GL_Q8) {
        B.ld_sc = (a.N + 31) / 32;
        B.sc = a.bs + t.r0 * B.ld_sc + n_blk / 32;
    }
    A.init(lane, wave, wave / S::GN);
    B.init(lane, wave, wave % S::GN);
}

// Keeps a memory phase's steps in their order.
__device__ STG_AI inline void in_order()
{
    STG_COMPILER_FENCE();
    __builtin_amdgcn_sched_barrier(0);
}
// A workgroup barrier that nothing is moved across.
__device__ STG_AI inline void tile_barrier()
{
    in_order();
    __builtin_amdgcn_s_barrier();
    in_order();
}

// A wave's accumulators to the output, through 32-row slabs in `lds`; in as
// many pieces as its rows and columns lie in.
template <class OP, class S>
__device__ STG_AI inline void store_tile(const GroupedArgs &a, const GroupRows &t, int64_t m_blk,
                                         int64_t n_blk, int64_t M,
                                         typename OP::acc_t (&acc)[S::FM][S::FN], int lane,
                                         int wave, uint32_t *lds)
{
    typedef typename S::OpA OpA;
    typedef typename S::OpB OpB;
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    EpiArgs e = group_epilogue(a, t.g, t.r0, M);
    e.vec = a.vec;
    constexpr int PA = S::PA, PB = S::PB;
    auto store = [&](auto p, auto q, auto cpol) STG_AI {
        constexpr int C = decltype(cpol)::value;
        constexpr int FM = S::FM / PA, FN = S::FN / PB;
        constexpr int I = decltype(p)::value * FM, J = decltype(q)::value * FN;
        const int64_t m0 = m_blk + OpA::at(decltype(p)::value, (wave / S::GN) * OpA::ROWS);
        const int64_t n0 = n_blk + OpB::at(decltype(q)::value, (wave % S::GN) * OpB::ROWS);
        typename OP::acc_t part[FM][FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                part[i][j] = acc[I + i][J + j];
        if (a.d_kind == OUT_F32)
            epilogue_slabs<OP, FM, FN, OUT_F32, C>(e, part, m0, n0, lane, lds);
        else if (a.d_kind == OUT_F16)
            epilogue_slabs<OP, FM, FN, OUT_F16, C>(e, part, m0, n0, lane, lds);
        else
            epilogue_slabs<OP, FM, FN, OUT_BF16, C>(e, part, m0, n0, lane, lds);
    };
    auto pieces = [&](auto cpol) STG_AI {
        store(I0{}, I0{}, cpol);
        if constexpr (PB == 2)
            store(I0{}, I1{}, cpol);
        if constexpr (PA == 2)
            store(I1{}, I0{}, cpol);
        if constexpr (PA == 2 && PB == 2)
            store(I1{}, I1{}, cpol);
    };
    // Whole cache lines go past the caches (2-8 % faster where the operands
    // want them), parts of lines have to meet there: with rows of 60.25 lines
    // non-temporal stores took 163 us, plain ones 67 (12 groups of 2944 x
    // 1928).
    if (a.whole_lines)
        pieces(std::integral_constant<int, EPI_CPOL>{});
    else
        pieces(std::integral_constant<int, 0>{});
}

// One BM x BN tile of group t at (m_blk, n_blk); M, K: its group's rows (of
// the output) and sum.
template <class OP, bool W, int ALAY, int BLAY, int BM, int BN>
__device__ STG_AI inline void tile_body(const GroupedArgs &a, const GroupRows &t, int64_t m_blk,
                                        int64_t n_blk, int64_t M, int64_t K, int lane, int wave,
                                        const Regions &L)
{
    typedef TileShape<OP, W, ALAY, BLAY, BM, BN> S;
    constexpr int FA = S::FA, FB = S::FB;
    typedef typename S::OpA OpA;
    typedef typename S::OpB OpB;
    auto reg_a = [&](auto half, auto buf) STG_AI -> uint8_t * {
        if constexpr (decltype(buf)::value == 0)
            return decltype(half)::value == 0 ? L.a00 : L.a10;
        else
            return decltype(half)::value == 0 ? L.a01 : L.a11;
    };
    auto reg_b = [&](auto half, auto buf) STG_AI -> uint8_t * {
        if constexpr (decltype(buf)::value == 0)
            return decltype(half)::value == 0 ? L.b00 : L.b10;
        else
            return decltype(half)::value == 0 ? L.b01 : L.b11;
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    OpA A;
    OpB B;
    set_operands<S>(A, B, a, t, m_blk, n_blk, M, K, lane, wave);

    typename OP::acc_t acc[2 * FA][2 * FB];
#pragma unroll
    for (int i = 0; i < 2 * FA; ++i)
#pragma unroll
        for (int j = 0; j < 2 * FB; ++j)
            acc[i][j] = typename OP::acc_t{};

    const int KT = (int)((K + 63) / 64);
    if (KT > 0) {
        u4_t fa[FA][2], fb[2][FB][2];
        auto read_a = [&](auto half, auto buf) STG_AI {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < FA; ++r)
                    fa[r][s] = A.read(reg_a(half, buf), r, s);
        };
        auto read_b = [&](auto half, auto buf) STG_AI {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < FB; ++r)
                    fb[decltype(half)::value][r][s] = B.read(reg_b(half, buf), r, s);
        };
        auto mfma = [&](auto ha, auto hb) STG_AI {
            constexpr int P = decltype(ha)::value, Q = decltype(hb)::value;
            tile_barrier();
            __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt(0)
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < FA; ++i)
#pragma unroll
                    for (int j = 0; j < FB; ++j)
                        acc[P * FA + i][Q * FB + j] =
                            OP::mma((const uint32_t *)&fa[i][s], (const uint32_t *)&fb[Q][j][s],
                                    acc[P * FA + i][Q * FB + j]);
            __builtin_amdgcn_s_setprio(0);
            tile_barrier();
        };
        // vector-memory instructions of the five clusters up to and with one
        // that copies A (B): what may be in flight when the copies of the
        // cluster before them have to be complete
        constexpr int VA = OpA::VM, VB = OpB::VM;
        constexpr int AFTER_B = 3 * VA + 2 * VB, AFTER_A = 2 * VA + 3 * VB;
        constexpr bool Q8 = BLAY == GL_Q8;
        // copies of B: tile t's half h; 8-bit: the registers loaded four
        // clusters before go to LDS first (tile ts, buffer of that tile)
        auto put_b = [&](auto half, auto buf) STG_AI {
            if constexpr (Q8)
                B.store(reg_b(half, buf), half, lane, wave);
        };

        // One K tile t in buffer P.  Cluster c copies, into the place that
        // was read two clusters before: c = 0 A1 of t + 1 (buffer 1 - P), 1
        // B0, 2 A0, 3 B1 of t + 2 (buffer P).  8-bit: cluster 1 first stores
        // B0 of t + 1, loaded in cluster 1 of t - 1, cluster 3 B1 of t + 1.
        auto tile = [&](auto pc, int kt) STG_AI {
            using P = decltype(pc);
            using N = std::integral_constant<int, 1 - P::value>;
            read_a(I0{}, P{});
            in_order();
            A.copy(reg_a(I1{}, N{}), I1{}, kt + 1, wave);
            in_order();
            STG_WAIT_VMCNT(AFTER_B);
            mfma(I0{}, I0{});
            read_b(I1{}, P{});
            put_b(I0{}, N{});
            in_order();
            B.copy(reg_b(I0{}, P{}), I0{}, kt + 2, wave);
            in_order();
            STG_WAIT_VMCNT(AFTER_A);
            mfma(I0{}, I1{});
            read_a(I1{}, P{});
            in_order();
            A.copy(reg_a(I0{}, P{}), I0{}, kt + 2, wave);
            in_order();
            STG_WAIT_VMCNT(AFTER_B);
            mfma(I1{}, I0{});
            read_b(I0{}, N{});
            put_b(I1{}, N{});
            in_order();
            B.copy(reg_b(I1{}, P{}), I1{}, kt + 2, wave);
            in_order();
            STG_WAIT_VMCNT(AFTER_A);
            mfma(I1{}, I1{});
        };

        // the copies of the clusters before cluster 0, in their order
        B.copy(reg_b(I0{}, I0{}), I0{}, 0, wave);
        A.copy(reg_a(I0{}, I0{}), I0{}, 0, wave);
        B.copy(reg_b(I1{}, I0{}), I1{}, 0, wave);
        A.copy(reg_a(I1{}, I0{}), I1{}, 0, wave);
        put_b(I0{}, I0{});
        B.copy(reg_b(I0{}, I1{}), I0{}, 1, wave);
        A.copy(reg_a(I0{}, I1{}), I0{}, 1, wave);
        put_b(I1{}, I0{});
        B.copy(reg_b(I1{}, I1{}), I1{}, 1, wave);
        STG_WAIT_VMCNT(3 * VB + 2 * VA);
        __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt(0): 8-bit B's stores
        tile_barrier();
        read_b(I0{}, I0{});
        __builtin_amdgcn_s_waitcnt(0xC07F); // (read before anyone copies over it)
        if (wave >= 4)
            tile_barrier(); // the trailing half starts one phase later
        int kt = 0;
        for (; kt + 1 < KT; kt += 2) {
            tile(I0{}, kt);
            tile(I1{}, kt + 1);
        }
        if (kt < KT)
            tile(I0{}, kt);
        if (wave < 4)
            tile_barrier();
        STG_WAIT_VMCNT(0); // copies past the last tile, before LDS is reused
        tile_barrier();
    }

    // a wave's slab of 32 rows lies in the region of its number
    uint8_t *slab = wave == 0   ? L.a00
                    : wave == 1 ? L.a10
                    : wave == 2 ? L.a01
                    : wave == 3 ? L.a11
                    : wave == 4 ? L.b00
                    : wave == 5 ? L.b10
                    : wave == 6 ? L.b01
                                : L.b11;
    store_tile<OP, S>(a, t, m_blk, n_blk, M, acc, lane, wave, (uint32_t *)slab);
}

// A 64 x 64 tile, for products of few tiles: there the time is a workgroup's
// way through K at the rate one compute unit's copies reach (measured about
// 60 GB/s), and four times the workgroups each copy half as much.  Four
// waves, four buffers s[0..3], the copies of three K tiles in flight, one
// barrier per K tile: before it every wave has waited for its copies of tile
// t and has tile t - 1 in registers (lgkmcnt(0) before its MFMAs); after it
// the copies of t + 3 go where t - 1 was.  An 8-bit B of tile t + 1 (loaded two
// tiles before) is stored after the reads of t.
template <class OP, bool W, int ALAY, int BLAY>
__device__ STG_AI inline void small_body(const GroupedArgs &a, const GroupRows &t, int64_t m_blk,
                                         int64_t n_blk, int64_t M, int64_t K, int lane, int wave,
                                         uint8_t *s0, uint8_t *s1, uint8_t *s2, uint8_t *s3)
{
    typedef SmallShape<OP, W, ALAY, BLAY> S;
    constexpr int RB = 64 * 128; // bytes of a region: A, B in a buffer
    typename S::OpA A;
    typename S::OpB B;
    set_operands<S>(A, B, a, t, m_blk, n_blk, M, K, lane, wave);
    typename OP::acc_t acc[2][2] = {};
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    auto buf = [&](auto b) STG_AI {
        constexpr int P = decltype(b)::value;
        return P == 0 ? s0 : P == 1 ? s1 : P == 2 ? s2 : s3;
    };
    // K tile kt: buffer and register set by its last bits, b
    auto copy = [&](auto b, int kt) STG_AI {
        A.copy(buf(b), I0{}, kt, wave);
        B.template copy<decltype(b)::value & 1>(buf(b) + RB, I0{}, kt, wave);
    };
    auto put_b = [&](auto b) STG_AI {
        if constexpr (BLAY == GL_Q8)
            B.template store<decltype(b)::value & 1>(buf(b) + RB, I0{}, lane, wave);
    };
    constexpr int PER = S::OpA::VM + S::OpB::VM; // vector-memory instructions of copy()
    const int KT = (int)((K + 63) / 64);
    auto tile = [&](auto b, int kt) STG_AI {
        constexpr int P = decltype(b)::value;
        in_order();
        STG_WAIT_VMCNT(2 * PER);
        tile_barrier();
        u4_t fa[2][2], fb[2][2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                fa[r][s] = A.read(buf(b), r, s);
                fb[r][s] = B.read(buf(b) + RB, r, s);
            }
        put_b(std::integral_constant<int, (P + 1) & 3>{});
        in_order();
        copy(std::integral_constant<int, (P + 3) & 3>{}, kt + 3);
        in_order();
        __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt(0)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = OP::mma((const uint32_t *)&fa[i][s], (const uint32_t *)&fb[j][s],
                                        acc[i][j]);
    };
    if (KT > 0) {
        copy(I0{}, 0);
        copy(I1{}, 1);
        put_b(I0{});
        copy(I2{}, 2);
        __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt(0): 8-bit B's stores
        int kt = 0;
        for (; kt + 3 < KT; kt += 4) {
            tile(I0{}, kt);
            tile(I1{}, kt + 1);
            tile(I2{}, kt + 2);
            tile(I3{}, kt + 3);
        }
        if (kt < KT)
            tile(I0{}, kt);
        if (kt + 1 < KT)
            tile(I1{}, kt + 1);
        if (kt + 2 < KT)
            tile(I2{}, kt + 2);
        STG_WAIT_VMCNT(0); // copies past the last tile, before LDS is reused
        tile_barrier();
    }
    uint8_t *slab = wave == 0 ? s0 : wave == 1 ? s1 : wave == 2 ? s2 : s3;
    store_tile<OP, S>(a, t, m_blk, n_blk, M, acc, lane, wave, (uint32_t *)slab);
}

// The kernel.  The rows' product with 256-row tiles (SHORT) cuts a group's
// last rows, if they are at most 128, as a 128 x 256 tile (0.69 of the time
// of a 256 x 256 one), and lets these come last, so that the compute units
// that finish their long tiles first take them.  If the long tiles past the
// last full round of the compute units and the short ones then fit one round
// as short tiles, these long ones are cut in two as well.
template <class OP, bool W, int ALAY, int BLAY, int BM, int BN, bool SHORT>
__global__ __launch_bounds__(512, BM * BN >= 256 * 128 ? 2 : 4) void k_grouped_tiled(GroupedArgs a,
                                                                                    int tiles_m,
                                                                                    int tiles_n)
{
    constexpr int AB = region_bytes<BM / 2, BN / 4>(), BB = region_bytes<BN / 2, BN / 4>();
    __shared__ __attribute__((aligned(1024))) uint8_t a00[AB], a10[AB], a01[AB], a11[AB], b00[BB],
        b10[BB], b01[BB], b11[BB];
    const Regions L = {a00, a10, a01, a11, b00, b10, b01, b11};
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    GroupRows t;
    if constexpr (W) {
        // every XCD takes an eighth of each group's tiles: groups differ in
        // length, and whole groups would leave some XCDs idle at the end
        const int per = (tiles_m * tiles_n + 7) >> 3, slot = blockIdx.x >> 3;
        const int tile = (blockIdx.x & 7) * per + slot % per;
        if (tile >= tiles_m * tiles_n)
            return;
        int tm, tn, b, e;
        t.g = slot / per;
        tile_of(tile, tiles_m, tiles_n, tm, tn);
        group_bounds(a, t.g, b, e);
        t.r0 = __builtin_amdgcn_readfirstlane(b);
        t.r1 = __builtin_amdgcn_readfirstlane(e);
        tile_body<OP, W, ALAY, BLAY, BM, BN>(a, t, wave_uniform((int64_t)tm * BM),
                                             wave_uniform((int64_t)tn * BN), a.K, t.r1 - t.r0, lane,
                                             wave, L);
    } else {
        int n_long, n_short;
        count_tiles<BM, SHORT>(a, lane, n_long, n_short);
        const int total = n_long * tiles_n, shorts = n_short * tiles_n;
        int tm, tn, part = -1; // part: half of a long tile
        if constexpr (SHORT) {
            int id = blockIdx.x, whole = total;
            const int rest = total % a.num_cu;
            if (2 * rest + shorts <= a.num_cu && (total - rest) % 8 == 0)
                whole -= rest;
            if (id >= (whole + 7) / 8 * 8) {
                id -= (whole + 7) / 8 * 8;
                if (id < 2 * (total - whole)) {
                    part = id & 1;
                    tile_of(whole + (id >> 1), n_long, tiles_n, tm, tn);
                } else {
                    id -= 2 * (total - whole);
                    if (id >= shorts)
                        return;
                    tm = n_long + id / tiles_n;
                    tn = id % tiles_n;
                }
            } else {
                id = xcd_tile(id, whole);
                if (id < 0)
                    return;
                tile_of(id, n_long, tiles_n, tm, tn);
            }
        } else {
            const int id = xcd_tile(blockIdx.x, total);
            if (id < 0)
                return;
            tile_of(id, n_long, tiles_n, tm, tn);
        }
        if (!find_tile<BM, SHORT>(a, __builtin_amdgcn_readfirstlane(tm), n_long, lane, t))
            return;
        const int64_t m = wave_uniform((int64_t)t.tm * BM), n = wave_uniform((int64_t)tn * BN);
        const int64_t M = t.r1 - t.r0;
        if constexpr (SHORT) {
            if (part >= 0 || M - m <= BM / 2) {
                const int64_t mh = m + (part > 0 ? BM / 2 : 0);
                if (mh < M)
                    tile_body<OP, W, ALAY, BLAY, BM / 2, BN>(a, t, mh, n, M, a.K, lane, wave, L);
                return;
            }
        }
        tile_body<OP, W, ALAY, BLAY, BM, BN>(a, t, m, n, M, a.K, lane, wave, L);
    }
}

// The kernel of 64 x 64 tiles, two workgroups per compute unit.
template <class OP, bool W, int ALAY, int BLAY>
__global__ __launch_bounds__(256, 2) void k_grouped_small(GroupedArgs a, int tiles_m, int tiles_n)
{
    __shared__ __attribute__((aligned(1024))) uint8_t s0[16384], s1[16384], s2[16384], s3[16384];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    GroupRows t;
    int tm, tn;
    if constexpr (W) {
        const int per = (tiles_m * tiles_n + 7) >> 3, slot = blockIdx.x >> 3;
        const int tile = (blockIdx.x & 7) * per + slot % per;
        if (tile >= tiles_m * tiles_n)
            return;
        int b, e;
        t.g = slot / per;
        tile_of(tile, tiles_m, tiles_n, tm, tn);
        group_bounds(a, t.g, b, e);
        t.r0 = __builtin_amdgcn_readfirstlane(b);
        t.r1 = __builtin_amdgcn_readfirstlane(e);
    } else {
        int n_long, n_short;
        count_tiles<64, false>(a, lane, n_long, n_short);
        const int id = xcd_tile(blockIdx.x, n_long * tiles_n);
        if (id < 0)
            return;
        tile_of(id, n_long, tiles_n, tm, tn);
        if (!find_tile<64, false>(a, __builtin_amdgcn_readfirstlane(tm), n_long, lane, t))
            return;
        tm = t.tm;
    }
    const int64_t M = W ? a.K : t.r1 - t.r0, K = W ? t.r1 - t.r0 : a.K;
    small_body<OP, W, ALAY, BLAY>(a, t, wave_uniform((int64_t)tm * 64), wave_uniform((int64_t)tn * 64),
                                 M, K, lane, wave, s0, s1, s2, s3);
}

} // namespace stg

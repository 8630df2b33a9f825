// The rows' grouped product for groups of few rows (a decoder's tokens over
// its experts), bound by streaming the groups' B once.
//
// A workgroup owns CW columns of one group and up to 64 of its rows; its
// eight waves split K (chunk c of KCH values goes to wave c % 8) and add
// their partial sums through LDS.  B goes straight from global memory into
// LDS, 1 KB per instruction in runs of 256 bytes (K-contiguous B, 4 columns)
// or 2 CW bytes (row-major B), into two buffers per wave that no other wave
// touches, so the loop has no barrier; the chunk after the one being
// multiplied is in flight.  A (few rows, read by every workgroup) comes from
// L2 straight into the MFMA's layout.
//
// K-contiguous B: column r's 16-byte chunk q of a 256-byte run at slot q ^
// (r & 15); lane group g takes chunks 4 g .. 4 g + 3 one per MFMA, and the
// same 64 bytes of A's rows.  Row-major B: K rows of CW values, read with
// the transposing loads; 32-byte piece p of K row k at p ^ swz(k), so that
// the eight K rows half a wave touches lie on all pieces of 256 bytes.
//
// Measured on MI355X: 4 rows in 4 of 32 groups, 1024 x 2048, 5.7 us (a 128 x
// 128 tile 19); 128 rows, 32 groups, 4096 x 2048, 109 us, 4.9 TB/s.
#include "grouped_common.hpp"

namespace stg {

constexpr int SK_BM = 64; // rows of a workgroup

template <bool BROW, int CW>
struct SkinnyGeom {
    static constexpr int KCH = BROW ? 64 : 128;      // K values per chunk
    static constexpr int BYTES = CW * KCH * 2;       // B bytes per chunk
    static constexpr int ND = BYTES / 1024;          // copies per chunk
    static constexpr int STEPS = KCH / 32;           // MFMA K steps per chunk
    static constexpr int FC = CW / 16;               // column fragments
};

template <class OP, bool BROW, int CW, int NRB>
__device__ STG_AI inline void skinny_body(const GroupedArgs &a, const GroupRows &t, int64_t m0,
                                          int64_t n0, int lane, int wave, uint8_t *buf0,
                                          uint8_t *buf1, float *red)
{
    typedef SkinnyGeom<BROW, CW> S;
    const int64_t M = t.r1 - t.r0;
    const int64_t lda = a.lda * 2, ldb = a.ldb * 2, kb = a.K * 2;
    const uint8_t *A = (const uint8_t *)a.A + (t.r0 + m0) * lda;
    const __amdgpu_buffer_rsrc_t ra = tile_rsrc(A, (M - m0 - 1) * lda + kb);
    const int l16 = lane & 15, q = lane >> 4;
    const int NC = (int)((a.K + S::KCH - 1) / S::KCH);
    const uint8_t *B =
        (const uint8_t *)a.B + (BROW ? (int64_t)t.g * a.K * ldb + n0 * 2
                                     : ((int64_t)t.g * a.N + n0) * ldb);
    const __amdgpu_buffer_rsrc_t rbc = tile_rsrc(B, BROW ? 0 : (a.N - n0 - 1) * ldb + kb);

    // A: byte in a row of step s of a chunk
    auto a_byte = [&](int s) STG_AI { return BROW ? 64 * s + 16 * q : 64 * q + 16 * s; };
    u4_t pa[2][NRB][S::STEPS];
    auto load = [&](auto set, uint8_t *buf, int c) STG_AI {
        constexpr int P = decltype(set)::value;
        if constexpr (!BROW) {
            const int r4 = lane >> 4;
#pragma unroll
            for (int d = 0; d < S::ND; ++d) {
                const int r = 4 * d + r4, ch = ((lane & 15) ^ (r & 15)) * 16;
                // (past K: an offset outside every resource, which reads zeros)
                const bool in = (int64_t)c * 256 + ch < kb;
                dma16(rbc, buf + d * 1024, in ? r * (int)ldb + ch : (int)0x80000000, c * 256);
            }
        } else {
            const int64_t left = a.K - (int64_t)c * S::KCH;
            const __amdgpu_buffer_rsrc_t rb = epi_rsrc(
                B + (int64_t)c * S::KCH * ldb, left > 0 ? (left - 1) * ldb + (a.N - n0) * 2 : 0);
            constexpr int CPR = CW / 8; // 16-byte chunks per K row
#pragma unroll
            for (int d = 0; d < S::ND; ++d) {
                const int i = d * 64 + lane, k = i / CPR;
                const int f = CPR == 8 ? ((k >> 1) & 1) | (((k >> 3) & 1) << 1) : (k >> 3) & 1;
                dma16(rb, buf + d * 1024, k * (int)ldb + ((i % CPR) ^ (f << 1)) * 16, 0);
            }
        }
#pragma unroll
        for (int b = 0; b < NRB; ++b)
#pragma unroll
            for (int s = 0; s < S::STEPS; ++s) {
                const bool in = (int64_t)c * (S::KCH * 2) + a_byte(s) < kb;
                pa[P][b][s] = buf_load16(
                    ra, in ? (16 * b + l16) * (int)lda + a_byte(s) : (int)0x80000000, c * S::KCH * 2);
            }
    };
    typename OP::acc_t acc[NRB][S::FC];
#pragma unroll
    for (int b = 0; b < NRB; ++b)
#pragma unroll
        for (int f = 0; f < S::FC; ++f)
            acc[b][f] = typename OP::acc_t{};
    auto compute = [&](auto set, const uint8_t *buf) STG_AI {
        constexpr int P = decltype(set)::value;
        // everything older than the next chunk's loads has arrived
        STG_COMPILER_FENCE();
        STG_WAIT_VMCNT(S::ND + NRB * S::STEPS);
        STG_COMPILER_FENCE();
        u4_t fb[S::FC][S::STEPS];
#pragma unroll
        for (int f = 0; f < S::FC; ++f)
#pragma unroll
            for (int s = 0; s < S::STEPS; ++s) {
                if constexpr (!BROW) {
                    fb[f][s] = *(const u4_t *)(buf + (16 * f + l16) * 256 +
                                               (((4 * q + s) ^ l16) << 4));
                } else {
                    constexpr int PITCH = CW * 2;
                    const int k = 8 * q + (l16 >> 2);
                    const int w = CW == 64 ? ((k >> 1) & 1) | (((k >> 3) & 1) << 1) : (k >> 3) & 1;
                    const uint8_t *p = buf + k * PITCH + ((f ^ w) << 5) + (l16 & 3) * 8;
                    lds_read_tr<2>(p + 32 * s * PITCH, (uint32_t *)&fb[f][s]);
                    lds_read_tr<2>(p + (32 * s + 4) * PITCH, (uint32_t *)&fb[f][s] + 2);
                }
            }
        wave_lds_sync(); // read before the buffer is copied into again
#pragma unroll
        for (int s = 0; s < S::STEPS; ++s)
#pragma unroll
            for (int b = 0; b < NRB; ++b)
#pragma unroll
                for (int f = 0; f < S::FC; ++f)
                    acc[b][f] = OP::mma((const uint32_t *)&pa[P][b][s],
                                        (const uint32_t *)&fb[f][s], acc[b][f]);
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    // (chunks past the last one read zeros without touching memory)
    load(I0{}, buf0, wave);
    for (int c = wave; c < NC; c += 16) {
        load(I1{}, buf1, c + 8);
        compute(I0{}, buf0);
        load(I0{}, buf0, c + 16);
        compute(I1{}, buf1);
    }
    STG_WAIT_VMCNT(0); // copies past the last chunk, before LDS is reused
    __syncthreads();

    // sixteen rows at a time: fragment f of wave w at red[(f * 8 + w) * 256 +
    // 4 lane], then wave f adds fragment f's eight parts in order
    const EpiArgs e = group_epilogue(a, t.g, t.r0, M);
#pragma unroll
    for (int b = 0; b < NRB; ++b) {
        if (b)
            __syncthreads();
#pragma unroll
        for (int f = 0; f < S::FC; ++f)
            *(typename OP::acc_t *)(red + (f * 8 + wave) * 256 + 4 * lane) = acc[b][f];
        __syncthreads();
        if (wave < S::FC) {
            typename OP::acc_t x = *(const typename OP::acc_t *)(red + wave * 8 * 256 + 4 * lane);
#pragma unroll
            for (int w = 1; w < 8; ++w)
                x += *(const typename OP::acc_t *)(red + (wave * 8 + w) * 256 + 4 * lane);
            const int64_t col = n0 + 16 * wave + l16;
            if (col < e.N)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int64_t row = m0 + 16 * b + 4 * q + r;
                    const float y = x[r];
                    if (row < M)
                        store_kind(e, row * e.ldd + col, y);
                }
        }
    }
}

template <class OP, bool BROW, int CW>
__global__ __launch_bounds__(512, 2) void k_grouped_skinny(GroupedArgs a, int strips)
{
    typedef SkinnyGeom<BROW, CW> S;
    // two buffers per wave; afterwards the first hold the partial sums of FC
    // fragments of 8 waves (1 KB each)
    constexpr int BUF = 8 * S::BYTES;
    static_assert(S::FC * 1024 <= S::BYTES, "partial sums");
    __shared__ __attribute__((aligned(1024))) uint8_t b0[BUF], b1[BUF];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    GroupRows t;
    // strips of one group go round robin over the XCDs
    if (!find_tile<SK_BM>(a, blockIdx.x / strips, 0, lane, t))
        return;
    const int64_t n0 = wave_uniform((int64_t)(blockIdx.x % strips) * CW);
    const int64_t m0 = wave_uniform((int64_t)t.tm * SK_BM);
    const int64_t rows = t.r1 - t.r0 - m0;
    uint8_t *w0 = b0 + wave * S::BYTES, *w1 = b1 + wave * S::BYTES;
    if (rows <= 16)
        skinny_body<OP, BROW, CW, 1>(a, t, m0, n0, lane, wave, w0, w1, (float *)b0);
    else if (rows <= 32)
        skinny_body<OP, BROW, CW, 2>(a, t, m0, n0, lane, wave, w0, w1, (float *)b0);
    else
        skinny_body<OP, BROW, CW, 4>(a, t, m0, n0, lane, wave, w0, w1, (float *)b0);
}

template <class OP, bool BROW, int CW>
static hipError_t launch_t(const GroupedArgs &a, hipStream_t s)
{
    const int strips = (int)((a.N + CW - 1) / CW);
    const dim3 grid((unsigned)(max_row_tiles<SK_BM>(a) * strips));
    hipLaunchKernelGGL((k_grouped_skinny<OP, BROW, CW>), grid, dim3(512), 0, s, a, strips);
    return hipGetLastError();
}

template <class OP>
static hipError_t launch_op(const GroupedArgs &a, hipStream_t s)
{
    // narrow strips where wide ones would leave compute units idle
    const int64_t tiles = max_row_tiles<SK_BM>(a);
    if (a.b_row)
        return tiles * ((a.N + 63) / 64) < 1024 ? launch_t<OP, true, 32>(a, s)
                                                : launch_t<OP, true, 64>(a, s);
    return tiles * ((a.N + 31) / 32) < 1024 ? launch_t<OP, false, 16>(a, s)
                                            : launch_t<OP, false, 32>(a, s);
}

hipError_t launch_grouped_skinny(const GroupedArgs &a, hipStream_t s)
{
    return a.bf16 ? launch_op<Op16BF16>(a, s) : launch_op<Op16F16>(a, s);
}

} // namespace stg

// Activation checkpoints in 8 bits (E4M3 codes, one E8M0 scale per 32
// columns of a row) and the gated activation H = silu(G) * U that keeps and
// uses them.
//
// All kernels are bound by memory: each lane handles 8 consecutive columns
// (16 bytes of the 16-bit tensor, 8 bytes of codes), four neighbouring lanes
// one block of 32, whose largest magnitude they exchange within the quad.
// Rows need no alignment beyond their elements'.  Measured on MI355X, calls in
// a row on the same buffers: 16384 rows of 2 x 2048 columns, bf16: the activation with its checkpoint 52 us (5.2
// TB/s), without one 35 (5.7), the checkpoint alone 32 (6.3) and back to 16
// bits 31 (6.6), the gradient 60 (5.6); 9001 rows of 2 x 1416, fp16, the gradient
// 23 us (5.6).
#include "device_common.hpp"
#include "moe_args.hpp"
#include "q8.hpp"
#include "vec16.hpp"

namespace stg {

typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
struct __attribute__((packed, aligned(1))) u2_any_t {
    u2_t v;
};

// The first n (1..8) of eight codes at p; zeros after them.
__device__ STG_AI inline u2_t load_codes(const uint8_t *p, int n)
{
    if (n >= 8)
        return ((const u2_any_t *)p)->v;
    u2_t v{};
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n)
            v[e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
    return v;
}

__device__ STG_AI inline void store_codes(uint8_t *p, u2_t v, int n)
{
    if (n >= 8) {
        ((u2_any_t *)p)->v = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n)
            p[e] = (uint8_t)(v[e >> 2] >> (8 * (e & 3)));
}

// The smallest e >= -127 with amax <= 448 * 2^e (0 for amax = 0): with amax
// = m 2^x, 1 <= m < 2, it is x - 8 for m <= 1.75 and x - 7 above.  amax is
// finite; 16-bit subnormals are normal in fp32 except bfloat16's, whose x is
// below the clamp.
__device__ STG_AI inline int block_exponent(float amax)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, amax);
    const int x = (int)(b >> 23) - 127;
    const int e = x - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return b == 0 ? 0 : e < -127 ? -127 : e;
}

// Largest finite |x| of eight values (0 if none is finite).
__device__ STG_AI inline float amax8(const float (&f)[8])
{
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float a = __builtin_fabsf(f[e]);
        m = a < __builtin_inff() && a > m ? a : m;
    }
    return m;
}

// The largest of a quad's values in each of its four lanes.
__device__ STG_AI inline float quad_max(float m)
{
    m = fmaxf(m, __shfl_xor(m, 1));
    return fmaxf(m, __shfl_xor(m, 2));
}

// Codes of eight values under the block exponent e: x 2^-e is exact in fp32
// or far below E4M3's smallest value, so the conversion's is the only
// rounding; |x| 2^-e <= 448 except for infinities, which become NaN first.
__device__ STG_AI inline u2_t encode8(const float (&f)[8], int e)
{
    // 2^-e: e from -127 to 120
    const float s = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = __builtin_fabsf(f[i]) < __builtin_inff() ? f[i] * s : __builtin_nanf("");
    u2_t v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], w, true);
        v[i] = (uint32_t)w;
    }
    return v;
}

// The values of eight codes, element i scaled by s0 (i < split) or s1.
__device__ STG_AI inline void decode8(u2_t v, float s0, float s1, int split, float (&f)[8])
{
    typedef float f2_t __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], false);
        const f2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], true);
        f[4 * i] = lo.x, f[4 * i + 1] = lo.y, f[4 * i + 2] = hi.x, f[4 * i + 3] = hi.y;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] *= i < split ? s0 : s1;
}

// s = 1 / (1 + exp(-g)) from exp(-|g|), which never leaves 0 .. 1.  The
// exponential is the square of exp(-|g| / 2): the exponential instruction
// flushes results below 2^-126 to zero, the multiplication does not, and
// g * s is still a normal bfloat16 there.
__device__ STG_AI inline float sigmoid(float g)
{
    const float r = __builtin_amdgcn_exp2f(__builtin_fabsf(g) * -0.72134752f); // log2(e) / 2
    const float t = r * r;
    const float d = __builtin_amdgcn_rcpf(1.0f + t);
    return g < 0.0f ? t * d : d;
}

// Lanes of a workgroup over (row, piece of 8 columns): `per` lanes per row
// (a power of two, at least 4 so that a block's quad stays in one wave).
struct Lanes {
    int64_t row, step; // first row of this lane, rows per sweep of the grid
    int piece;         // first piece
};
template <int TPR>
__device__ STG_AI inline Lanes lanes()
{
    Lanes l;
    l.row = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    l.step = (int64_t)gridDim.x * (256 / TPR);
    l.piece = threadIdx.x % TPR;
    return l;
}

// ---------------------------------------------------------------- store, swiglu

// Codes and scales of a rows x cols tensor; ACT: and H = silu(G) * U, G its
// first half and U its second.  A lane quantises the piece it loads; lanes
// of the second half also load G's values beside theirs (from L2: another
// lane of the workgroup has read them), so that any width runs one code.
template <bool BF, bool ACT, int TPR>
__global__ __launch_bounds__(256) void k_q8_store(Q8Args a)
{
    const Lanes l = lanes<TPR>();
    const int64_t nb = (a.cols + 31) / 32, half = a.cols / 2;
    for (int64_t r = l.row; r < a.rows; r += l.step) {
        const uint16_t *x = (const uint16_t *)a.x + r * a.ldx;
        // (whole quads together: the block's last lanes may hold no column)
        for (int64_t c = l.piece * 8; c - (c & 31) < a.cols; c += TPR * 8) {
            const int n = (int)min((int64_t)8, max((int64_t)0, a.cols - c));
            float f[8] = {};
            if (n > 0)
                widen8<BF>(load8(x + c, n), f);
            if (a.codes) {
                const int e = block_exponent(quad_max(amax8(f)));
                if (n > 0)
                    store_codes(a.codes + r * a.cols + c, encode8(f, e), n);
                if ((c & 31) == 0)
                    a.scales[r * nb + c / 32] = (uint8_t)(e + 127);
            }
            if constexpr (ACT) {
                uint16_t *h = (uint16_t *)a.out + r * a.ldo;
                // columns of U: those from `half` on
                const int skip = (int)min((int64_t)8, max((int64_t)0, half - c));
                if (skip == 0 && n > 0) {
                    float g[8], y[8];
                    widen8<BF>(load8(x + (c - half), n), g);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = g[e] * sigmoid(g[e]) * f[e];
                    store8(h + (c - half), narrow8<BF>(y), n);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e >= skip && e < n) {
                            const float g = widen<BF>(x[c + e - half]);
                            const float y = g * sigmoid(g) * f[e];
                            h[c + e - half] = BF ? f32_to_bf16_bits(y) : f32_to_f16_bits(y);
                        }
                }
            }
        }
    }
}

// ---------------------------------------------------------------- load

template <bool BF, int TPR>
__global__ __launch_bounds__(256) void k_q8_load(Q8Args a)
{
    const Lanes l = lanes<TPR>();
    const int64_t nb = (a.cols + 31) / 32;
    for (int64_t r = l.row; r < a.rows; r += l.step)
        for (int64_t c = l.piece * 8; c < a.cols; c += TPR * 8) {
            const int n = (int)min((int64_t)8, a.cols - c);
            const float s = e8m0(a.scales[r * nb + c / 32]);
            float f[8];
            decode8(load_codes(a.codes + r * a.cols + c, n), s, s, 8, f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = clamp16<BF>(f[e]);
            store8((uint16_t *)a.out + r * a.ldo + c, narrow8<BF>(f), n);
        }
}

// ---------------------------------------------------------------- backward

// Values are clamped to the type's range, as in k_q8_load: the block that ends
// at bfloat16's largest value has codes of 256 * 2^120, infinity in fp32.  Both
// this and a dH * u past fp32's range are looked for once per eight columns:
// a clamp and a choice for each cost 2.7 of 22.1 us (9001 rows of 1416).
template <bool BF, int TPR>
__global__ __launch_bounds__(256) void k_swiglu_backward(Q8Args a)
{
    const Lanes l = lanes<TPR>();
    const int64_t nb = (a.cols + 31) / 32, half = a.cols / 2;
    for (int64_t r = l.row; r < a.rows; r += l.step) {
        const uint8_t *q = a.codes + r * a.cols, *sc = a.scales + r * nb;
        for (int64_t c = l.piece * 8; c < half; c += TPR * 8) {
            const int n = (int)min((int64_t)8, half - c);
            const int64_t cu = half + c;
            float g[8], u[8], d[8], dg[8], du[8], h[8];
            const u2_t qg = load_codes(q + c, n), qu = load_codes(q + cu, n);
            const u4_t dv = load8((const uint16_t *)a.x + r * a.ldx + c, n);
            // U's piece may reach into the next block
            const uint32_t bg = sc[c / 32], bu0 = sc[cu / 32], bu1 = sc[min((cu + 7) / 32, nb - 1)];
            decode8(qg, e8m0(bg), e8m0(bg), 8, g);
            decode8(qu, e8m0(bu0), e8m0(bu1), 32 - (int)(cu & 31), u);
            if (max(max(bg, bu0), bu1) > MAX_SCALE<BF>)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    g[e] = clamp16<BF>(g[e]);
                    u[e] = clamp16<BF>(u[e]);
                }
            widen8<BF>(dv, d);
            float far = 0.0f; // largest |dH * u|
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float s = sigmoid(g[e]), gs = g[e] * s, p = d[e] * u[e];
                far = BF ? fmaxf(far, __builtin_fabsf(p)) : far; // (fp16: below 2^32)
                dg[e] = p * s * (1.0f + g[e] * (1.0f - s));
                du[e] = d[e] * gs;
                h[e] = gs * u[e];
            }
            // dH * u may leave fp32's range where s brings it back: both are
            // above 1 then, and the gate's derivative goes first
            if (far == __builtin_inff())
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!(__builtin_fabsf(d[e] * u[e]) < __builtin_inff())) {
                        const float s = sigmoid(g[e]);
                        dg[e] = d[e] * (s * (1.0f + g[e] * (1.0f - s))) * u[e];
                    }
            uint16_t *o = (uint16_t *)a.out + r * a.ldo;
            store8(o + c, narrow8<BF>(dg), n);
            store8(o + cu, narrow8<BF>(du), n);
            if (a.out2)
                store8((uint16_t *)a.out2 + r * a.ldo2 + c, narrow8<BF>(h), n);
        }
    }
}

// ---------------------------------------------------------------- launch

// Lanes per row for `cols` columns, and the grid.
template <class F>
static void with_lanes(int64_t rows, int64_t cols, F &&f)
{
    const int tpr = cols <= 128 ? 16 : cols <= 512 ? 64 : 256;
    const int64_t nb = (rows + 256 / tpr - 1) / (256 / tpr);
    const dim3 grid((unsigned)(nb < (1 << 20) ? nb : (1 << 20)));
    if (tpr == 16)
        f(std::integral_constant<int, 16>{}, grid);
    else if (tpr == 64)
        f(std::integral_constant<int, 64>{}, grid);
    else
        f(std::integral_constant<int, 256>{}, grid);
}

hipError_t launch_q8_store(const Q8Args &a, hipStream_t s)
{
    with_lanes(a.rows, a.cols, [&](auto t, dim3 grid) {
        constexpr int T = decltype(t)::value;
        if (a.bf16)
            hipLaunchKernelGGL((k_q8_store<true, false, T>), grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_q8_store<false, false, T>), grid, dim3(256), 0, s, a);
    });
    return hipGetLastError();
}

hipError_t launch_swiglu(const Q8Args &a, hipStream_t s)
{
    with_lanes(a.rows, a.cols, [&](auto t, dim3 grid) {
        constexpr int T = decltype(t)::value;
        if (a.bf16)
            hipLaunchKernelGGL((k_q8_store<true, true, T>), grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_q8_store<false, true, T>), grid, dim3(256), 0, s, a);
    });
    return hipGetLastError();
}

hipError_t launch_q8_load(const Q8Args &a, hipStream_t s)
{
    with_lanes(a.rows, a.cols, [&](auto t, dim3 grid) {
        constexpr int T = decltype(t)::value;
        if (a.bf16)
            hipLaunchKernelGGL((k_q8_load<true, T>), grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_q8_load<false, T>), grid, dim3(256), 0, s, a);
    });
    return hipGetLastError();
}

hipError_t launch_swiglu_backward(const Q8Args &a, hipStream_t s)
{
    with_lanes(a.rows, a.cols / 2, [&](auto t, dim3 grid) {
        constexpr int T = decltype(t)::value;
        if (a.bf16)
            hipLaunchKernelGGL((k_swiglu_backward<true, T>), grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_swiglu_backward<false, T>), grid, dim3(256), 0, s, a);
    });
    return hipGetLastError();
}

} // namespace stg

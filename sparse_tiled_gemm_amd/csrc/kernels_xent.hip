// Linear cross entropy: the launches around its products.  Rows are the tokens
// that have a target, in their order: the products then skip the others, and
// read X in whole aligned 16-byte chunks whatever its strides.
#include "vec16.hpp"
#include "xent_common.hpp"

namespace stg {

// |x|, 0 for an infinity or NaN
__device__ STG_AI inline float finite_abs(float x)
{
    x = __builtin_fabsf(x);
    return x <= 3.402823466e38f ? x : 0.0f;
}

// Rows, targets and coefficients of a.prep tokens, and 512 columns
// (blockIdx.y) of their rows of X.  A workgroup counts the targets before its
// tokens by itself, so that one launch does; what it needs of its own tokens
// is loaded before that.
template <bool BACKWARD>
__global__ __launch_bounds__(256) void k_xent_prepare(XentArgs a)
{
    constexpr int R = XENT_STEP / 4; // rows of a wave
    __shared__ int part[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t first = (int64_t)blockIdx.x * a.prep;
    const bool lists = blockIdx.y == 0;
    const int64_t c = ((int64_t)blockIdx.y * 64 + lane) * 8, at = c < a.hp ? c : 0;
    const int nc = (int)min((int64_t)8, a.hidden - c);
    const bool full = a.hidden >= 8 && __all(nc >= 8 || c >= a.hp);
    int before = -1;
    float g = 0.0f;
    for (int64_t t0 = first; t0 < min(first + a.prep, a.tokens); t0 += XENT_STEP) {
        // the first 32 lanes of every wave hold the step's tokens
        const int64_t t = min(t0 + (lane & (XENT_STEP - 1)), a.tokens - 1);
        const bool in = lane < XENT_STEP && t0 + lane < a.tokens;
        const int target = xent_target(a, t);
        float cb = 0.0f, cd = 0.0f, cl = 0.0f;
        if constexpr (BACKWARD) {
            cb = a.dloss[t];
            cl = a.lse_in[t];
            cd = a.dlse ? a.dlse[t] : 0.0f;
        }
        u4_t x[R];
        if (full)
#pragma unroll
            for (int i = 0; i < R; ++i)
                x[i] = ((const u4_any_t *)((const uint16_t *)a.X +
                                           min(t0 + wave * R + i, a.tokens - 1) * a.ldx + at))->v;
        if (before < 0) {
            int b = 0;
            for (int64_t s = tid; s < first; s += 1024) { // (four in flight)
                int v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[q] = xent_target(a, min(s + 256 * q, first - 1));
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    b += s + 256 * q < first && v[q] >= 0;
            }
#pragma unroll
            for (int d = 32; d; d >>= 1)
                b += __shfl_xor(b, d);
            if (lane == 0)
                part[wave] = b;
            __syncthreads();
            before = part[0] + part[1] + part[2] + part[3];
        }
        const int y = in ? target : -1;
        const uint64_t m = __ballot(y >= 0);
        const int row = y >= 0 ? before + __popcll(m & (((uint64_t)1 << lane) - 1)) : -1;
        before += __popcll(m);
        if (wave == 0 && lists) {
            if (in)
                a.pos[t] = row;
            if (row >= 0) {
                a.map[row] = (int)t;
                a.tgt[row] = y;
                if constexpr (BACKWARD) {
                    const float ca = a.dlse ? cb + cd : cb;
                    a.ca[row] = ca;
                    a.cb[row] = cb;
                    a.cl[row] = cl * LOG2E;
                    g = __builtin_fmaxf(g, __builtin_fmaxf(finite_abs(ca), finite_abs(cb)));
                }
            } else if (in && !BACKWARD) {
                a.lse[t] = 0.0f;
                if (a.loss)
                    a.loss[t] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t to = __shfl(row, wave * R + i);
            if (to < 0 || c >= a.hp)
                continue;
            *(u4_t *)(a.Xc + to * a.ldc + c) =
                full ? x[i] : load8((const uint16_t *)a.X + (t0 + wave * R + i) * a.ldx + c, nc);
        }
    }
    if (wave == 0 && lists) {
        if constexpr (BACKWARD) {
#pragma unroll
            for (int d = 32; d; d >>= 1)
                g = __builtin_fmaxf(g, __shfl_xor(g, d));
            if (lane == 0)
                a.gmax[blockIdx.x] = g;
        }
        if (lane == 0 && blockIdx.x == gridDim.x - 1) {
            before = max(before, 0); // (no tokens)
            a.count[0] = before;
            if constexpr (BACKWARD)
                a.count[1] = xent_splits(before, a.dx.edge, a.dx.tiles_n, a.dx.cols, a.dx.slots,
                                         a.dx.most);
        }
    }
}

// Rows of W in whole aligned 16-byte chunks.
__global__ __launch_bounds__(256) void k_xent_copy(XentCopy c)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int pieces = (int)(c.hp / 8);
    for (int64_t r = (int64_t)blockIdx.x * 4 + wave; r < c.n; r += (int64_t)gridDim.x * 4)
        for (int i = lane; i < pieces; i += 64) {
            const int n = (int)min((int64_t)8, c.hidden - i * 8);
            *(u4_t *)(c.out + r * c.ldo + i * 8) = load8(c.W + r * c.ldw + i * 8, n);
        }
}

// lse and loss of `rows` rows (a power of two up to 64) per workgroup from
// the tiles' maxima and sums: 256 / rows threads per row, joined in order.
__global__ __launch_bounds__(256) void k_xent_loss(XentArgs a, int rows)
{
    __shared__ float sm[256], ss[256];
    const int tid = threadIdx.x, slices = 256 / rows;
    const int n = xent_rows(a);
    const int64_t row = (int64_t)blockIdx.x * rows + (tid & (rows - 1));
    float m = -INFINITY, s = 0.0f;
    auto join = [&](float m2, float s2) STG_AI {
        const float mx = __builtin_fmaxf(m, m2), ref = sum_ref(mx);
        s = s * __builtin_amdgcn_exp2f((m - ref) * LOG2E) +
            s2 * __builtin_amdgcn_exp2f((m2 - ref) * LOG2E);
        m = mx;
    };
    typedef float f2_t __attribute__((ext_vector_type(2)));
    const f2_t *part = (const f2_t *)a.part + row;
    if (row < n)
        for (int64_t i = tid / rows; i < a.part_tiles; i += 4 * slices) {
            f2_t p[4]; // (in flight together)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                p[q] = part[min(i + q * slices, a.part_tiles - 1) * a.tokens];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i + q * slices < a.part_tiles)
                    join(p[q].x, p[q].y);
        }
    sm[tid] = m;
    ss[tid] = s;
    __syncthreads();
    for (int d = 128; d >= rows; d >>= 1) {
        if (tid < d) {
            join(sm[tid + d], ss[tid + d]);
            sm[tid] = m;
            ss[tid] = s;
        }
        __syncthreads();
    }
    if (tid < rows && row < n) {
        const int64_t t = a.direct ? row : a.map[row];
        const bool in = !a.direct || xent_target(a, t) >= 0;
        // (in 64 bits: a loss far below lse keeps its bits)
        const double lse = (double)m + log((double)s);
        a.lse[t] = in ? (float)lse : 0.0f;
        if (a.loss)
            a.loss[t] = in ? (float)(lse - (double)a.zt[row]) : 0.0f;
    }
}

// dX by token: the splits' sums, scaled and rounded once; zeros for tokens
// without a target.  A wave per token and 512 columns, or (JOIN, where there may
// be many splits) a workgroup whose waves take a quarter of the splits each.
template <int DK, bool JOIN>
__global__ __launch_bounds__(256) void k_xent_out(XentArgs a, XentOut o)
{
    __shared__ f4_t red[JOIN ? 3 : 1][2][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = ((int64_t)blockIdx.y * 64 + lane) * 8, at = c < a.hp ? c : 0;
    const Gmax first = load_gmax(a, lane);
    const int64_t slab = (int64_t)a.count[0] * a.hp;
    const int splits = a.count[1], per = JOIN ? (splits + 3) / 4 : splits;
    const int s0 = JOIN ? wave * per : 0, s1 = min(splits, s0 + per);
    const int n = (int)min((int64_t)8, a.hidden - c);
    constexpr int W = JOIN ? 1 : 4;
    for (int64_t t = (int64_t)blockIdx.x * W + (JOIN ? 0 : wave); t < a.tokens;
         t += (int64_t)gridDim.x * W) {
        const int row = a.pos[t];
        f4_t x{}, y{};
        if (row >= 0) {
            const float *p = o.acc + (int64_t)row * a.hp + at;
            constexpr int B = JOIN ? 8 : 4; // in flight
            for (int s = s0; s < s1; s += B) {
                f4_t u[B], v[B];
#pragma unroll
                for (int q = 0; q < B; ++q) {
                    const f4_t *z = (const f4_t *)(p + min(s + q, s1 - 1) * slab);
                    u[q] = z[0];
                    v[q] = z[1];
                }
#pragma unroll
                for (int q = 0; q < B; ++q)
                    if (s + q < s1) {
                        x += u[q];
                        y += v[q];
                    }
            }
        }
        if constexpr (JOIN) {
            if (wave) {
                red[wave - 1][0][lane] = x;
                red[wave - 1][1][lane] = y;
            }
            __syncthreads();
            if (wave == 0)
#pragma unroll
                for (int w = 0; w < 3; ++w) {
                    x += red[w][0][lane];
                    y += red[w][1][lane];
                }
            __syncthreads();
        }
        const float f = xent_factor(a, first, lane); // (by all lanes)
        if ((JOIN && wave) || c >= a.hidden)
            continue;
        x *= f;
        y *= f;
        const float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        if constexpr (DK == OUT_F32) {
            float *d = (float *)o.dX + t * o.ldd + c;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n)
                    d[e] = row >= 0 ? v[e] : 0.0f;
        } else {
            store8((uint16_t *)o.dX + t * o.ldd + c, row >= 0 ? narrow8<DK == OUT_BF16>(v) : u4_t{}, n);
        }
    }
}

// ---------------------------------------------------------------- launch

hipError_t launch_xent_prepare(const XentArgs &a, bool backward, hipStream_t s)
{
    // (no tokens: the count is still written)
    const dim3 grid((unsigned)(a.tokens > 0 ? (a.tokens + a.prep - 1) / a.prep : 1),
                    (unsigned)((a.hp + 511) / 512));
    if (backward)
        hipLaunchKernelGGL(k_xent_prepare<true>, grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL(k_xent_prepare<false>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_xent_copy(const XentCopy &c, hipStream_t s)
{
    const int64_t b = (c.n + 3) / 4;
    hipLaunchKernelGGL(k_xent_copy, dim3((unsigned)(b < (1 << 16) ? b : (1 << 16))), dim3(256), 0, s, c);
    return hipGetLastError();
}

hipError_t launch_xent_loss(const XentArgs &a, hipStream_t s)
{
    int rows = 1; // up to 512 workgroups
    while (rows < 64 && rows * 512 < a.tokens)
        rows *= 2;
    hipLaunchKernelGGL(k_xent_loss, dim3((unsigned)((a.tokens + rows - 1) / rows)), dim3(256), 0, s, a,
                       rows);
    return hipGetLastError();
}

template <int DK>
static void launch_out(const XentArgs &a, const XentOut &o, hipStream_t s)
{
    // (at most 2^16 workgroups for the tokens; they take several then)
    auto grid = [&](int per) {
        const int64_t b = (a.tokens + per - 1) / per;
        return dim3((unsigned)(b < (1 << 16) ? b : 1 << 16), (unsigned)((a.hidden + 511) / 512));
    };
    const XentSplits &x = a.dx;
    if (xent_splits((int)a.tokens, x.edge, x.tiles_n, x.cols, x.slots, x.most) >= 8)
        hipLaunchKernelGGL((k_xent_out<DK, true>), grid(1), dim3(256), 0, s, a, o);
    else
        hipLaunchKernelGGL((k_xent_out<DK, false>), grid(4), dim3(256), 0, s, a, o);
}

hipError_t launch_xent_out(const XentArgs &a, const XentOut &o, hipStream_t s)
{
    if (o.d_kind == OUT_F32)
        launch_out<OUT_F32>(a, o, s);
    else if (o.d_kind == OUT_F16)
        launch_out<OUT_F16>(a, o, s);
    else
        launch_out<OUT_BF16>(a, o, s);
    return hipGetLastError();
}

} // namespace stg

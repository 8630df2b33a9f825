// Linear cross entropy: the launches around its products.  Rows are the tokens
// that have a target, in their order: the products then skip the others, and
// read X in whole aligned 16-byte chunks whatever its strides.
#include "vec16.hpp"
#include "xent_common.hpp"

namespace stg {

// Rows, targets and coefficients of XENT_PREP tokens, and their rows of X.  A
// workgroup counts the targets before its tokens by itself, so that one launch
// does (8192 tokens: 256 workgroups, 32 KB of targets each on average).
template <bool BACKWARD>
__global__ __launch_bounds__(256) void k_xent_prepare(XentArgs a)
{
    __shared__ int part[4], row_of[XENT_PREP];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t0 = (int64_t)blockIdx.x * XENT_PREP;
    int before = 0;
    for (int64_t t = tid; t < t0; t += 256)
        before += xent_target(a, t) >= 0;
#pragma unroll
    for (int d = 32; d; d >>= 1)
        before += __shfl_xor(before, d);
    if (lane == 0)
        part[wave] = before;
    __syncthreads();
    before = part[0] + part[1] + part[2] + part[3];
    if (wave == 0) {
        const int64_t t = t0 + lane;
        const bool in = lane < XENT_PREP && t < a.tokens;
        const int y = in ? xent_target(a, t) : -1;
        const uint64_t m = __ballot(y >= 0);
        const int row = y >= 0 ? before + __popcll(m & (((uint64_t)1 << lane) - 1)) : -1;
        if (lane < XENT_PREP)
            row_of[lane] = row;
        if (in)
            a.pos[t] = row;
        float g = 0.0f;
        if (row >= 0) {
            a.map[row] = (int)t;
            a.tgt[row] = y;
            if constexpr (BACKWARD) {
                const float cb = a.dloss[t], ca = a.dlse ? cb + a.dlse[t] : cb;
                a.ca[row] = ca;
                a.cb[row] = cb;
                a.cl[row] = a.lse_in[t] * LOG2E;
                g = __builtin_fmaxf(__builtin_fabsf(ca), __builtin_fabsf(cb));
            }
        } else if (in && !BACKWARD) {
            a.lse[t] = 0.0f;
            if (a.loss)
                a.loss[t] = 0.0f;
        }
        if constexpr (BACKWARD) {
#pragma unroll
            for (int d = 32; d; d >>= 1)
                g = __builtin_fmaxf(g, __shfl_xor(g, d));
            if (lane == 0)
                a.gmax[blockIdx.x] = g;
        }
        if (lane == 0 && blockIdx.x == gridDim.x - 1)
            *a.count = before + __popcll(m);
    }
    __syncthreads();
    const int pieces = (int)(a.hp / 8);
    for (int i = wave; i < XENT_PREP; i += 4) {
        const int row = row_of[i];
        if (row < 0)
            continue;
        const uint16_t *x = (const uint16_t *)a.X + (t0 + i) * a.ldx;
        for (int c = lane; c < pieces; c += 64) {
            const int n = (int)min((int64_t)8, a.hidden - c * 8);
            *(u4_t *)(a.Xc + row * a.hp + c * 8) = load8(x + c * 8, n);
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
            *(u4_t *)(c.out + r * c.hp + i * 8) = load8(c.W + r * c.ldw + i * 8, n);
        }
}

// lse and loss of `rows` rows (a power of two up to 64) per workgroup from
// the tiles' maxima and sums: 256 / rows threads per row, joined in order.
__global__ __launch_bounds__(256) void k_xent_loss(XentArgs a, int rows)
{
    __shared__ float sm[256], ss[256];
    const int tid = threadIdx.x, slices = 256 / rows;
    const int n = *a.count;
    const int64_t row = (int64_t)blockIdx.x * rows + (tid & (rows - 1));
    float m = -INFINITY, s = 0.0f;
    auto join = [&](float m2, float s2) STG_AI {
        const float mx = __builtin_fmaxf(m, m2), ref = mx == -INFINITY ? 0.0f : mx;
        s = s * __builtin_amdgcn_exp2f((m - ref) * LOG2E) +
            s2 * __builtin_amdgcn_exp2f((m2 - ref) * LOG2E);
        m = mx;
    };
    if (row < n)
        for (int64_t i = tid / rows; i < a.part_tiles; i += slices) {
            const float *p = a.part + (i * a.tokens + row) * 2;
            join(p[0], p[1]);
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
        const int t = a.map[row];
        // (in 64 bits: a loss far below lse keeps its bits)
        const double lse = (double)m + log((double)s);
        a.lse[t] = (float)lse;
        if (a.loss)
            a.loss[t] = (float)(lse - (double)a.zt[row]);
    }
}

// dX by token: the splits' sums in order, scaled and rounded once; zeros for
// tokens without a target.
template <int DK>
__global__ __launch_bounds__(256) void k_xent_out(XentArgs a, XentOut o)
{
    const int lane = threadIdx.x & 63;
    const int64_t c = ((int64_t)blockIdx.y * 64 + lane) * 8;
    const float f = xent_factor(a, lane);
    if (c >= a.hidden)
        return;
    const int n = (int)min((int64_t)8, a.hidden - c);
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.tokens;
         t += (int64_t)gridDim.x * 4) {
        const int row = a.pos[t];
        f4_t x{}, y{};
        if (row >= 0) {
            for (int s = 0; s < o.splits; ++s) {
                const f4_t *p = (const f4_t *)(o.acc + ((int64_t)s * a.tokens + row) * a.hp + c);
                x += p[0];
                y += p[1];
            }
            x *= f;
            y *= f;
        }
        const float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        if constexpr (DK == OUT_F32) {
            float *d = (float *)o.dX + t * o.ldd + c;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n)
                    d[e] = v[e];
        } else {
            store8((uint16_t *)o.dX + t * o.ldd + c, narrow8<DK == OUT_BF16>(v), n);
        }
    }
}

// ---------------------------------------------------------------- launch

hipError_t launch_xent_prepare(const XentArgs &a, bool backward, hipStream_t s)
{
    // (no tokens: the count is still written)
    const dim3 grid((unsigned)(a.tokens > 0 ? (a.tokens + XENT_PREP - 1) / XENT_PREP : 1));
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
    int rows = 1;
    while (rows < 64 && rows < a.tokens)
        rows *= 2;
    hipLaunchKernelGGL(k_xent_loss, dim3((unsigned)((a.tokens + rows - 1) / rows)), dim3(256), 0, s, a,
                       rows);
    return hipGetLastError();
}

hipError_t launch_xent_out(const XentArgs &a, const XentOut &o, hipStream_t s)
{
    const int64_t b = (a.tokens + 3) / 4;
    const dim3 grid((unsigned)(b < (1 << 16) ? b : (1 << 16)), (unsigned)((a.hidden + 511) / 512));
    if (o.d_kind == OUT_F32)
        hipLaunchKernelGGL(k_xent_out<OUT_F32>, grid, dim3(256), 0, s, a, o);
    else if (o.d_kind == OUT_F16)
        hipLaunchKernelGGL(k_xent_out<OUT_F16>, grid, dim3(256), 0, s, a, o);
    else
        hipLaunchKernelGGL(k_xent_out<OUT_BF16>, grid, dim3(256), 0, s, a, o);
    return hipGetLastError();
}

} // namespace stg

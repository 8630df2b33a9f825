// Routing for a mixture-of-experts MLP: slots (token, choice) sorted by
// expert, rows copied to the sorted order, combined back with weights, and
// the combination's gradient.
//
// The sort (32768 slots, 64 groups: 4.7 us for the counts, 5.8 for the places,
// both a chain of latencies) is a counting sort: a slot's place is the number of slots of
// lower experts plus the number of earlier slots of its own expert, so the
// result depends on the ids alone.  Within 64 slots the earlier ones of the
// same expert are counted with one ballot per bit of the expert's number.
//
// All row kernels move 8 elements (16 bytes) per lane and piece; rows need no
// alignment beyond their elements' (gfx950 loads and stores 16 bytes at any
// 2-byte address), so odd widths run the same code.
#include "device_common.hpp"
#include "moe_args.hpp"
#include "sort_util.hpp"
#include "vec16.hpp"

namespace stg {

constexpr int SORT_NT = 512, SORT_W = SORT_NT / 64;

__device__ STG_AI inline int route_id(const RouteArgs &a, int64_t s)
{
    // -1 for every id without a group
    if (a.id8) {
        const int64_t v = ((const int64_t *)a.ids)[s];
        return v >= 0 && v < a.groups ? (int)v : -1;
    }
    const int32_t v = ((const int32_t *)a.ids)[s];
    return v >= 0 && v < a.groups ? v : -1;
}

// ---------------------------------------------------------------- sort

// Slots per group of each chunk of a.chunk slots.
__global__ __launch_bounds__(SORT_NT) void k_route_count(RouteArgs a)
{
    __shared__ int hist[ROUTE_MAX_GROUPS];
    const int tid = threadIdx.x;
    for (int g = tid; g < a.groups; g += SORT_NT)
        hist[g] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * a.chunk;
    for (int i = tid; i < a.chunk; i += SORT_NT) {
        if (s0 + i < a.slots) {
            const int g = route_id(a, s0 + i);
            if (g >= 0)
                atomicAdd(&hist[g], 1);
        }
    }
    __syncthreads();
    for (int g = tid; g < a.groups; g += SORT_NT)
        a.counts[(int64_t)blockIdx.x * a.groups + g] = hist[g];
}

// Places of one chunk's slots from the counts of all chunks.  Wave w takes
// the chunk's w-th eighth, 64 slots a step.
__global__ __launch_bounds__(SORT_NT) void k_route_place(RouteArgs a)
{
    __shared__ int tot[ROUTE_MAX_GROUPS + 1], bef[ROUTE_MAX_GROUPS];
    __shared__ int whist[SORT_W][ROUTE_MAX_GROUPS];
    __shared__ int tmp[SORT_W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int G = a.groups, me = blockIdx.x;
    for (int g = tid; g < G; g += SORT_NT) {
        tot[g] = bef[g] = 0;
#pragma unroll
        for (int w = 0; w < SORT_W; ++w)
            whist[w][g] = 0;
    }
    __syncthreads();
    // this wave's slots by group
    const int per = a.chunk / SORT_W; // a multiple of 64
    const int64_t c0 = (int64_t)me * a.chunk, w0 = c0 + (int64_t)wave * per;
    for (int i = 0; i < per; i += 64) {
        const int64_t s = w0 + i + lane;
        const int g = s < a.slots ? route_id(a, s) : -1;
        if (g >= 0)
            atomicAdd(&whist[wave][g], 1);
    }
    // all chunks' counts: a power of two of threads beside each other take
    // neighbouring groups, the others further chunks
    int gp = 64;
    while (gp < G && gp < SORT_NT)
        gp *= 2;
    const int parts = SORT_NT / gp;
    for (int g = tid % gp; g < G; g += gp) {
        int t = 0, b = 0;
        for (int c = tid / gp; c < a.chunks; c += parts) {
            const int v = a.counts[(int64_t)c * G + g];
            t += v;
            b += c < me ? v : 0;
        }
        atomicAdd(&tot[g], t);
        atomicAdd(&bef[g], b);
    }
    __syncthreads();
    scan_lds<SORT_NT>(tot, G, tmp, tid);
    if (me == 0)
        for (int g = tid; g <= G; g += SORT_NT)
            a.offsets[g] = tot[g];
    for (int g = tid; g < G; g += SORT_NT) {
        int at = tot[g] + bef[g];
#pragma unroll
        for (int w = 0; w < SORT_W; ++w) {
            const int n = whist[w][g];
            whist[w][g] = at;
            at += n;
        }
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz(G);
    for (int i = 0; i < per; i += 64) {
        const int64_t s = w0 + i + lane;
        const int g = s < a.slots ? route_id(a, s) : -1;
        const uint64_t same = same_group(g, bits);
        const int rank = lanes_below(same);
        int p = -1;
        if (g >= 0)
            p = whist[wave][g] + rank;
        wave_lds_sync();
        if (g >= 0 && rank == 0)
            whist[wave][g] = p + __popcll(same);
        wave_lds_sync();
        if (s < a.slots)
            a.pos[s] = p;
        if (p >= 0)
            a.order[p] = (int)s;
    }
    // order past the last place
    for (int64_t i = c0 + tid; i < c0 + a.chunk && i < a.slots; i += SORT_NT)
        if (i >= tot[G])
            a.order[i] = -1;
}

// ---------------------------------------------------------------- rows

// Up to ROUTE_SMALL slots, one launch: a workgroup counts all slots by group
// for itself (those before its own apart), ranks its own ROUTE_CHUNK slots
// and, with COPY (dispatch), moves their rows.  blockIdx.y cuts the columns, so
// that a decoder's few tokens still spread over the chip; workgroups of y = 0
// write the lists.  With gemm_moe_combine behind it, against the three
// launches of the chunked sort and copy: 680 tokens of 3 choices, 13 groups,
// 1027 columns 11.4 and 17.8 us, 1360 tokens 17.8 and 18.2 us, 1999 tokens
// 24.8 and 20.0 us.
constexpr int ROUTE_CHUNK = 32;
template <bool COPY>
__global__ __launch_bounds__(SORT_NT) void k_route_small(RouteArgs a, RowsArgs r, int pieces)
{
    __shared__ int tot[ROUTE_MAX_GROUPS + 1], bef[ROUTE_MAX_GROUPS];
    __shared__ int place[ROUTE_CHUNK];
    __shared__ int tmp[SORT_W];
    constexpr int PER = ROUTE_SMALL / SORT_NT; // slots per thread at most
    const int tid = threadIdx.x;
    const int G = a.groups, n = (int)a.slots, c0 = blockIdx.x * ROUTE_CHUNK;
    int gid[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        gid[i] = i * SORT_NT + tid < n ? route_id(a, i * SORT_NT + tid) : -1;
    // the first wave's lanes hold this workgroup's slots
    const int own = c0 + tid;
    const int g = tid < ROUTE_CHUNK && own < n ? route_id(a, own) : -1;
    for (int i = tid; i < G; i += SORT_NT)
        tot[i] = bef[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (gid[i] >= 0) {
            atomicAdd(&tot[gid[i]], 1);
            if (i * SORT_NT + tid < c0)
                atomicAdd(&bef[gid[i]], 1);
        }
    __syncthreads();
    scan_lds<SORT_NT>(tot, G, tmp, tid);
    if (tid < 64) {
        const int rank = lanes_below(same_group(g, 32 - __builtin_clz(G)));
        const int p = g >= 0 ? tot[g] + bef[g] + rank : -1;
        if (tid < ROUTE_CHUNK && own < n) {
            place[tid] = p;
            if (blockIdx.y == 0) {
                a.pos[own] = p;
                if (p >= 0)
                    a.order[p] = own;
                if (own >= tot[G])
                    a.order[own] = -1;
            }
        }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = tid; i <= G; i += SORT_NT)
            a.offsets[i] = tot[i];
    if constexpr (COPY) {
        __syncthreads();
        // this workgroup's pieces of 8 columns of its slots
        const int per = (pieces + gridDim.y - 1) / gridDim.y, p0 = blockIdx.y * per;
        const int np = min(per, pieces - p0), total = np > 0 ? min(ROUTE_CHUNK, n - c0) * np : 0;
        for (int i = tid; i < total; i += SORT_NT) {
            const int s = i / np;
            const int64_t c = (int64_t)(p0 + i - s * np) * 8;
            const int p = place[s];
            if (p >= 0) {
                const int64_t t = (c0 + s) / (int)r.topk;
                const int nc = (int)min((int64_t)8, r.cols - c);
                store8((uint16_t *)r.out + p * r.ld_out + c,
                       load8((const uint16_t *)r.in + t * r.ld_in + c, nc), nc);
            }
        }
    }
}

// Rows of X to their places: each piece of a row is read once and written
// topk times.  TPR lanes per token.  Bound by the writes: 8192 tokens of 4
// choices, 4096 columns, 56 us, 5.9 TB/s.
template <int TPR>
__global__ __launch_bounds__(256) void k_route_copy(RowsArgs r)
{
    int64_t t = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    for (; t < r.tokens; t += (int64_t)gridDim.x * (256 / TPR)) {
        const uint16_t *x = (const uint16_t *)r.in + t * r.ld_in;
        const int32_t *pos = r.pos + t * r.topk;
        for (int64_t c = (threadIdx.x % TPR) * 8; c < r.cols; c += TPR * 8) {
            const int n = (int)min((int64_t)8, r.cols - c);
            const u4_t v = load8(x + c, n);
            for (int64_t k = 0; k < r.topk; ++k) {
                const int32_t p = pos[k];
                if (p >= 0)
                    store8((uint16_t *)r.out + p * r.ld_out + c, v, n);
            }
        }
    }
}

// Y[t] = sum over k of w[t,k] Ys[pos[t,k]].  TPR lanes per token and
// blockIdx.y's part of the columns, one piece per lane; KB rows are in flight
// per lane.  Bound by memory: 8192 tokens of 4 choices, 4096 columns, 81 us
// (4.1 TB/s), 93 right after the rows were written; two tokens per lane
// measured no faster.
template <bool BF, int TPR, int KB>
__global__ __launch_bounds__(256) void k_combine(RowsArgs r)
{
    const int64_t c = ((int64_t)blockIdx.y * TPR + threadIdx.x % TPR) * 8;
    if (c >= r.cols)
        return;
    const int n = (int)min((int64_t)8, r.cols - c);
    int64_t t = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    for (; t < r.tokens; t += (int64_t)gridDim.x * (256 / TPR)) {
        const int32_t *pos = r.pos + t * r.topk;
        const float *wt = r.weights ? r.weights + t * r.topk : nullptr;
        float acc[8] = {};
        for (int64_t k0 = 0; k0 < r.topk; k0 += KB) {
            int64_t p[KB];
            u4_t v[KB];
            float w[KB];
            // (a slot without a place adds nothing, whatever its weight)
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                p[q] = k0 + q < r.topk ? pos[k0 + q] : -1;
                p[q] = p[q] < r.rows ? p[q] : -1;
                w[q] = wt && k0 + q < r.topk ? wt[k0 + q] : 1.0f;
            }
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                v[q] = u4_t{};
                if (p[q] >= 0)
                    v[q] = load8((const uint16_t *)r.in + p[q] * r.ld_in + c, n);
            }
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                float f[8];
                widen8<BF>(v[q], f);
                const float x = p[q] >= 0 ? w[q] : 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[e] = __builtin_fmaf(x, f[e], acc[e]);
            }
        }
        store8((uint16_t *)r.out + t * r.ld_out + c, narrow8<BF>(acc), n);
    }
}

// The gradient of k_combine: per token, each choice's row of dYs and the dot
// product of its row of Ys with dY.  TPT lanes per token: a part of a wave for
// narrow rows, a wave, or a workgroup of four where there are few tokens; KB
// choices share one pass over dY.  Bound by memory: 8192 tokens of 4 choices,
// 4096 columns, 112 us, 5.4 TB/s; 6457 tokens of 6 choices, 157 columns, 28 us
// with 16 lanes per token and 40 with 64.
template <bool BF, int TPT, int KB>
__global__ __launch_bounds__(256) void k_combine_backward(RowsArgs r)
{
    __shared__ float part[256 / 64][KB];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // (t is uniform over the lanes of a token, and over the workgroup where
    // it meets at barriers)
    int64_t t = (int64_t)blockIdx.x * (256 / TPT) + threadIdx.x / TPT;
    for (; t < r.tokens; t += (int64_t)gridDim.x * (256 / TPT)) {
        const uint16_t *dy = (const uint16_t *)r.in + t * r.ld_in;
        for (int64_t k0 = 0; k0 < r.topk; k0 += KB) {
            float acc[KB] = {}, w[KB];
            int64_t p[KB];
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                const int64_t s = t * r.topk + k0 + q;
                const bool in = k0 + q < r.topk;
                p[q] = in ? r.pos[s] : -1;
                p[q] = p[q] < r.rows ? p[q] : -1;
                w[q] = in ? r.weights[s] : 0.0f;
            }
            for (int64_t c = (threadIdx.x % TPT) * 8; c < r.cols; c += TPT * 8) {
                const int n = (int)min((int64_t)8, r.cols - c);
                u4_t y[KB];
                float d[8];
                const u4_t dv = load8(dy + c, n);
#pragma unroll
                for (int q = 0; q < KB; ++q)
                    if (p[q] >= 0)
                        y[q] = load8((const uint16_t *)r.in2 + p[q] * r.ld_in2 + c, n);
                widen8<BF>(dv, d);
#pragma unroll
                for (int q = 0; q < KB; ++q)
                    if (p[q] >= 0) {
                        float f[8], g[8];
                        widen8<BF>(y[q], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            acc[q] = __builtin_fmaf(f[e], d[e], acc[q]);
                            g[e] = w[q] * d[e];
                        }
                        store8((uint16_t *)r.out + p[q] * r.ld_out + c, narrow8<BF>(g), n);
                    }
            }
#pragma unroll
            for (int q = 0; q < KB; ++q) {
#pragma unroll
                for (int d = (TPT < 64 ? TPT : 64) / 2; d; d >>= 1)
                    acc[q] += __shfl_xor(acc[q], d);
            }
            if constexpr (TPT <= 64) {
                if (lane % TPT == 0)
#pragma unroll
                    for (int q = 0; q < KB; ++q)
                        if (k0 + q < r.topk)
                            r.dw[t * r.topk + k0 + q] = acc[q];
            } else {
                if (lane == 0)
#pragma unroll
                    for (int q = 0; q < KB; ++q)
                        part[wave][q] = acc[q];
                __syncthreads();
                if (threadIdx.x < KB && k0 + threadIdx.x < r.topk) {
                    float x = 0.0f;
#pragma unroll
                    for (int w2 = 0; w2 < 256 / 64; ++w2)
                        x += part[w2][threadIdx.x];
                    r.dw[t * r.topk + k0 + threadIdx.x] = x;
                }
                __syncthreads();
            }
        }
    }
}

// ---------------------------------------------------------------- launch

// Workgroups for n tokens, `per` of them each; past 2^18 they take several.
static unsigned blocks(int64_t n, int per)
{
    const int64_t b = (n + per - 1) / per;
    return (unsigned)(b < (1 << 18) ? b : (1 << 18));
}

// Lanes per row of 8-column pieces: enough for one pass over a narrow row,
// at most a workgroup.
static int lanes_per_row(int64_t cols)
{
    return cols <= 128 ? 16 : cols <= 512 ? 64 : 256;
}

hipError_t launch_route(const RouteArgs &a, const RowsArgs *r, hipStream_t s)
{
    if (a.slots <= ROUTE_SMALL) {
        const unsigned chunks = (unsigned)(a.slots > 0 ? (a.slots + ROUTE_CHUNK - 1) / ROUTE_CHUNK : 1);
        if (!r) {
            hipLaunchKernelGGL(k_route_small<false>, dim3(chunks), dim3(SORT_NT), 0, s, a, RowsArgs{},
                               0);
        } else {
            // about two workgroups per compute unit, each with work for its lanes
            const int64_t pieces = (r->cols + 7) / 8, slots = a.slots < ROUTE_CHUNK ? a.slots : ROUTE_CHUNK;
            int64_t y = (slots * pieces + SORT_NT - 1) / SORT_NT;
            if (y > 512 / (int64_t)chunks)
                y = 512 / (int64_t)chunks;
            hipLaunchKernelGGL(k_route_small<true>, dim3(chunks, (unsigned)(y < 1 ? 1 : y)),
                               dim3(SORT_NT), 0, s, a, *r, (int)pieces);
        }
        return hipGetLastError();
    }
    hipLaunchKernelGGL(k_route_count, dim3((unsigned)a.chunks), dim3(SORT_NT), 0, s, a);
    hipLaunchKernelGGL(k_route_place, dim3((unsigned)a.chunks), dim3(SORT_NT), 0, s, a);
    if (r && r->cols > 0) {
        switch (lanes_per_row(r->cols)) {
        case 16:
            hipLaunchKernelGGL(k_route_copy<16>, dim3(blocks(r->tokens, 16)), dim3(256), 0, s, *r);
            break;
        case 64:
            hipLaunchKernelGGL(k_route_copy<64>, dim3(blocks(r->tokens, 4)), dim3(256), 0, s, *r);
            break;
        default:
            hipLaunchKernelGGL(k_route_copy<256>, dim3(blocks(r->tokens, 1)), dim3(256), 0, s, *r);
        }
    }
    return hipGetLastError();
}

template <bool BF, int TPR>
static void combine_t(const RowsArgs &a, hipStream_t s)
{
    // (cols <= 2^23: at most 2^12 column parts of 256 lanes x 8)
    const dim3 grid(blocks(a.tokens, 256 / TPR), (unsigned)((a.cols + 8 * TPR - 1) / (8 * TPR)));
    if (a.topk <= 4)
        hipLaunchKernelGGL((k_combine<BF, TPR, 4>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_combine<BF, TPR, 8>), grid, dim3(256), 0, s, a);
}

template <bool BF>
static void combine_lanes(const RowsArgs &a, hipStream_t s)
{
    switch (lanes_per_row(a.cols)) {
    case 16: combine_t<BF, 16>(a, s); break;
    case 64: combine_t<BF, 64>(a, s); break;
    default: combine_t<BF, 256>(a, s);
    }
}

hipError_t launch_combine(const RowsArgs &a, hipStream_t s)
{
    a.bf16 ? combine_lanes<true>(a, s) : combine_lanes<false>(a, s);
    return hipGetLastError();
}

template <bool BF, int TPT>
static void combine_backward_t(const RowsArgs &a, hipStream_t s)
{
    const dim3 grid(blocks(a.tokens, 256 / TPT));
    if (a.topk <= 4)
        hipLaunchKernelGGL((k_combine_backward<BF, TPT, 4>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_combine_backward<BF, TPT, 8>), grid, dim3(256), 0, s, a);
}

template <bool BF>
static void combine_backward_lanes(const RowsArgs &a, hipStream_t s)
{
    if (a.cols <= 256)
        combine_backward_t<BF, 16>(a, s);
    else if (a.tokens >= 2048)
        combine_backward_t<BF, 64>(a, s);
    else
        combine_backward_t<BF, 256>(a, s);
}

hipError_t launch_combine_backward(const RowsArgs &a, hipStream_t s)
{
    a.bf16 ? combine_backward_lanes<true>(a, s) : combine_backward_lanes<false>(a, s);
    return hipGetLastError();
}

} // namespace stg

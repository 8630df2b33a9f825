// Rows of an embedding table looked up by token, and their gradient.
//
// The lookup Y[t] = s E[id_t] is one pass of 16-byte pieces; bound by memory.
//
// The gradient dE[v] = s sum of dY[t] over the tokens t of row v needs the
// tokens grouped by row.  Up to EMBED_SMALL tokens one launch does it without
// a sort: a workgroup per token looks through all ids, leaves if an earlier
// token has its id, and sums the rows of the later ones otherwise.  More
// tokens are sorted in two stable passes, by the low bits of the id (counts
// and places of chunks, as the routing's sort) and, a workgroup per bin, by
// the high bits.  A wave then sums the rows of EMBED_RUN sorted positions; sums
// of a row that reach over several runs (a frequent token) are left in the
// workspace and joined by a last launch.  Every sum's order is a function of
// the ids alone.
//
// Where the whole gradient is written, zeros go to all of dE beside the
// sort's three launches, which leave most of the chip idle, and the rows that
// have tokens are written after them.
#include "device_common.hpp"
#include "sort_util.hpp"
#include "vec16.hpp"
#include "vocab_args.hpp"

namespace stg {

// ---------------------------------------------------------------- eight values

struct __attribute__((packed, aligned(4))) f4_any_t {
    f4_t v;
};

constexpr int elem_bytes(int kind) { return kind == OUT_F32 ? 4 : 2; }

// Elements off .. off + n - 1 (n in 1 .. 8, zeros after them) of an array of
// kind K.
template <int K>
__device__ STG_AI inline void load8f(const void *base, int64_t off, int n, float (&f)[8])
{
    if constexpr (K == OUT_F32) {
        const float *p = (const float *)base + off;
        if (n >= 8) {
            const f4_t a = ((const f4_any_t *)p)->v, b = ((const f4_any_t *)(p + 4))->v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[e] = a[e];
                f[4 + e] = b[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = e < n ? p[e] : 0.0f;
        }
    } else {
        widen8<K == OUT_BF16>(load8((const uint16_t *)base + off, n), f);
    }
}

template <int K>
__device__ STG_AI inline void store8f(void *base, int64_t off, int n, const float (&f)[8])
{
    if constexpr (K == OUT_F32) {
        float *p = (float *)base + off;
        if (n >= 8) {
            ((f4_any_t *)p)->v = f4_t{f[0], f[1], f[2], f[3]};
            ((f4_any_t *)(p + 4))->v = f4_t{f[4], f[5], f[6], f[7]};
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n)
                    p[e] = f[e];
        }
    } else {
        store8((uint16_t *)base + off, narrow8<K == OUT_BF16>(f), n);
    }
}

// Token t's row of the table, -1 for an id that names none.
__device__ STG_AI inline int embed_id(const EmbedArgs &a, int64_t t)
{
    if (a.id8) {
        const int64_t v = ((const int64_t *)a.ids)[t];
        return v >= 0 && v < a.vocab ? (int)v : -1;
    }
    const int32_t v = ((const int32_t *)a.ids)[t];
    return v >= 0 && v < a.vocab ? v : -1;
}

// ---------------------------------------------------------------- lookup

// TPR lanes per token and blockIdx.y's part of the columns, eight columns per
// lane.
template <int EK, int YK, int TPR>
__global__ __launch_bounds__(256) void k_embed(EmbedArgs a)
{
    const int64_t c = ((int64_t)blockIdx.y * TPR + threadIdx.x % TPR) * 8;
    if (c >= a.cols)
        return;
    const int n = (int)min((int64_t)8, a.cols - c);
    int64_t t = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    for (; t < a.tokens; t += (int64_t)gridDim.x * (256 / TPR)) {
        const int id = embed_id(a, t);
        float f[8] = {};
        if (id >= 0) {
            load8f<EK>(a.in, id * a.ld_in + c, n, f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] *= a.scale;
        }
        store8f<YK>(a.out, t * a.ld_out + c, n, f);
    }
}

// ---------------------------------------------------------------- gradient: rows

// dE's row v, columns c .. c + n - 1, from the sum of its tokens' rows.
template <int DK>
__device__ STG_AI inline void put_row(const EmbedArgs &a, int64_t v, int64_t c, int n, float (&f)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] *= a.scale;
    if (a.accumulate) {
        float d[8];
        load8f<DK>(a.out, v * a.ld_out + c, n, d);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] += d[e];
    }
    store8f<DK>(a.out, v * a.ld_out + c, n, f);
}

// Zeros to rows [r0, r1) of dE by `parts` workgroups of NT threads, this one
// being part `part`.
template <int NT>
__device__ STG_AI inline void zero_rows(const EmbedArgs &a, int64_t r0, int64_t r1, int64_t part,
                                        int64_t parts)
{
    const int64_t eb = elem_bytes(a.e_kind);
    const bool flat = a.ld_out == a.cols;
    const int64_t row = (flat ? (r1 - r0) * a.cols : a.cols) * eb, rows = flat ? 1 : r1 - r0;
    // rows by their 16-byte pieces and a tail of 2-byte ones; many short rows
    // go to the workgroups in turn, a long one is cut among them
    const bool cut = flat || rows < parts;
    for (int64_t r = cut ? 0 : part; r < rows; r += cut ? 1 : parts) {
        uint8_t *p = (uint8_t *)a.out + (r0 + r) * a.ld_out * eb;
        const int64_t pieces = row >> 4;
        int64_t i = (cut ? part * NT : 0) + threadIdx.x;
        for (; i < pieces; i += cut ? parts * NT : NT)
            ((u4_any_t *)(p + i * 16))->v = u4_t{};
        if (!cut || part == 0)
            for (int64_t o = pieces * 16 + threadIdx.x * 2; o < row; o += NT * 2)
                *(uint16_t *)(p + o) = 0;
    }
}

// ---------------------------------------------------------------- gradient: few tokens

// Workgroups 0 .. tokens-1: the row of token blockIdx.x, if it is the first of
// its id.  The others: zeros to EMBED_ZR rows of dE each that have no token.
// blockIdx.y cuts the columns, 512 (a wave's 64 x 8) each.
constexpr int EMBED_ZR = 32;
template <int YK, int DK>
__global__ __launch_bounds__(256) void k_embed_grad_small(EmbedArgs a)
{
    constexpr int PER = EMBED_SMALL / 256;
    __shared__ int found[PER * 4 + 1];
    __shared__ int list[EMBED_SMALL];
    __shared__ float red[4][64][9]; // (9: the lanes' eight values on all banks)
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int T = (int)a.tokens;
    int id[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        id[i] = i * 256 + tid < T ? embed_id(a, i * 256 + tid) : -1;
    const int64_t c = ((int64_t)blockIdx.y * 64 + lane) * 8;
    const int nc = (int)min((int64_t)8, a.cols - c); // (may be negative)
    if (blockIdx.x >= T) {
        const int64_t r0 = (int64_t)(blockIdx.x - T) * EMBED_ZR;
        if (tid < EMBED_ZR)
            list[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t r = id[i] - r0;
            if (id[i] >= 0 && r >= 0 && r < EMBED_ZR)
                list[r] = 1;
        }
        __syncthreads();
        const float z[8] = {};
        for (int r = wave; r < EMBED_ZR; r += 4)
            if (r0 + r < a.vocab && !list[r] && nc > 0)
                store8f<DK>(a.out, (r0 + r) * a.ld_out + c, nc, z);
        return;
    }
    const int me = blockIdx.x, mine = embed_id(a, me);
    if (mine < 0)
        return;
    // tokens of this id by their numbers; an earlier one has the row
    bool early = false;
    uint64_t m[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool same = id[i] == mine;
        early |= same && i * 256 + tid < me;
        m[i] = __ballot(same);
        if (lane == 0)
            found[i * 4 + wave] = __popcll(m[i]);
    }
    if (__syncthreads_or(early))
        return;
    int n = 0;
    for (int k = 0; k < PER * 4; ++k) {
        const int x = found[k];
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (k == i * 4 + wave && (m[i] >> lane & 1))
                list[n + lanes_below(m[i])] = i * 256 + tid;
        n += x;
    }
    __syncthreads();
    // a quarter of the rows per wave, eight in flight; joined in order
    const int per = n >= 16 ? (n + 3) / 4 : n;
    float acc[8] = {};
    if (nc > 0)
        for (int k0 = wave * per; k0 < min(n, (wave + 1) * per); k0 += 8) {
            float f[8][8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (k0 + q < min(n, (wave + 1) * per))
                    load8f<YK>(a.in, list[k0 + q] * a.ld_in + c, nc, f[q]);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (k0 + q < min(n, (wave + 1) * per))
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[e] += f[q][e];
        }
    if (n >= 16) {
        if (wave)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                red[wave][lane][e] = acc[e];
        __syncthreads();
        if (wave == 0)
#pragma unroll
            for (int w = 1; w < 4; ++w)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[e] += red[w][lane][e];
    }
    if (wave == 0 && nc > 0)
        put_row<DK>(a, mine, c, nc, acc);
}

// ---------------------------------------------------------------- gradient: sort

constexpr int ES_NT = 512, ES_W = ES_NT / 64;

// Part `third` (0 .. 2) of dE's zeros, by the workgroups behind the sort's
// `sorters`.
__device__ STG_AI inline void zero_third(const EmbedArgs &a, int third, int sorters)
{
    zero_rows<ES_NT>(a, a.vocab * third / 3, a.vocab * (third + 1) / 3, blockIdx.x - sorters,
                     gridDim.x - sorters);
}

// Tokens per low-bits bin of each chunk.
__global__ __launch_bounds__(ES_NT) void k_embed_count(EmbedArgs a)
{
    __shared__ int hist[EMBED_MAX_BINS];
    if ((int)blockIdx.x >= a.chunks) {
        zero_third(a, 0, a.chunks);
        return;
    }
    const int tid = threadIdx.x, bins = 1 << a.lo_bits;
    for (int g = tid; g < bins; g += ES_NT)
        hist[g] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * a.chunk;
    for (int i = tid; i < a.chunk; i += ES_NT)
        if (s0 + i < a.tokens) {
            const int v = embed_id(a, s0 + i);
            if (v >= 0)
                atomicAdd(&hist[v & (bins - 1)], 1);
        }
    __syncthreads();
    for (int g = tid; g < bins; g += ES_NT)
        a.counts[(int64_t)blockIdx.x * bins + g] = hist[g];
}

// This wave's items [i0, i1) of `get(i)` (a bin, -1: none) to the places
// whist[bin] counts up from, in order; put(i, place).
template <class Get, class Put>
__device__ STG_AI inline void place_items(int64_t i0, int64_t i1, int lane, int bits, int *whist,
                                          Get &&get, Put &&put)
{
    for (int64_t i = i0; i < i1; i += 64) {
        const int g = i + lane < i1 ? get(i + lane) : -1;
        const uint64_t same = same_group(g, bits);
        const int rank = lanes_below(same);
        int p = -1;
        if (g >= 0)
            p = whist[g] + rank;
        wave_lds_sync();
        if (g >= 0 && rank == 0)
            whist[g] = p + __popcll(same);
        wave_lds_sync();
        if (p >= 0)
            put(i + lane, p);
    }
}

// The tokens by the low bits of their ids.  Wave w takes its chunk's w-th
// eighth.
__global__ __launch_bounds__(ES_NT) void k_embed_place(EmbedArgs a)
{
    __shared__ int tot[EMBED_MAX_BINS + 1], bef[EMBED_MAX_BINS];
    __shared__ int whist[ES_W][EMBED_MAX_BINS];
    __shared__ int tmp[ES_W];
    if ((int)blockIdx.x >= a.chunks) {
        zero_third(a, 1, a.chunks);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int bins = 1 << a.lo_bits, me = blockIdx.x;
    for (int g = tid; g < bins; g += ES_NT) {
        tot[g] = bef[g] = 0;
#pragma unroll
        for (int w = 0; w < ES_W; ++w)
            whist[w][g] = 0;
    }
    __syncthreads();
    const int per = a.chunk / ES_W; // a multiple of 64
    const int64_t w0 = (int64_t)me * a.chunk + (int64_t)wave * per;
    const int64_t w1 = min(w0 + per, a.tokens);
    auto bin = [&](int64_t t) STG_AI {
        const int v = embed_id(a, t);
        return v >= 0 ? v & (bins - 1) : -1;
    };
    for (int64_t t = w0 + lane; t < w1; t += 64) {
        const int g = bin(t);
        if (g >= 0)
            atomicAdd(&whist[wave][g], 1);
    }
    // all chunks' counts: neighbouring threads take neighbouring bins, the
    // others further chunks
    int gp = 64;
    while (gp < bins && gp < ES_NT)
        gp *= 2;
    const int parts = ES_NT / gp;
    for (int g = tid % gp; g < bins; g += gp) {
        int t = 0, b = 0;
        for (int c = tid / gp; c < a.chunks; c += parts) {
            const int v = a.counts[(int64_t)c * bins + g];
            t += v;
            b += c < me ? v : 0;
        }
        atomicAdd(&tot[g], t);
        atomicAdd(&bef[g], b);
    }
    __syncthreads();
    scan_lds<ES_NT>(tot, bins, tmp, tid);
    if (me == 0)
        for (int g = tid; g <= bins; g += ES_NT)
            a.bounds[g] = tot[g];
    for (int g = tid; g < bins; g += ES_NT) {
        int at = tot[g] + bef[g];
#pragma unroll
        for (int w = 0; w < ES_W; ++w) {
            const int n = whist[w][g];
            whist[w][g] = at;
            at += n;
        }
    }
    __syncthreads();
    place_items(w0, w1, lane, a.lo_bits, whist[wave], bin,
                [&](int64_t t, int p) STG_AI { a.binned[p] = (int)t; });
}

// One bin's tokens by the high bits of their ids.  Wave w takes the bin's w-th
// eighth.
__global__ __launch_bounds__(ES_NT) void k_embed_group(EmbedArgs a)
{
    __shared__ int tot[EMBED_MAX_BINS + 1];
    __shared__ int whist[ES_W][EMBED_MAX_BINS];
    __shared__ int tmp[ES_W];
    const int lows = 1 << a.lo_bits;
    if ((int)blockIdx.x >= lows) {
        zero_third(a, 2, lows);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int bins = 1 << a.hi_bits;
    const int b0 = a.bounds[blockIdx.x], n = a.bounds[blockIdx.x + 1] - b0;
    if (n <= 0)
        return;
    for (int g = tid; g < bins; g += ES_NT)
#pragma unroll
        for (int w = 0; w < ES_W; ++w)
            whist[w][g] = 0;
    __syncthreads();
    const int per = ((n + ES_W - 1) / ES_W + 63) / 64 * 64;
    const int w0 = min(n, wave * per), w1 = min(n, w0 + per);
    auto bin = [&](int64_t i) STG_AI { return embed_id(a, a.binned[b0 + i]) >> a.lo_bits; };
    for (int i = w0 + lane; i < w1; i += 64)
        atomicAdd(&whist[wave][bin(i)], 1);
    __syncthreads();
    for (int g = tid; g < bins; g += ES_NT) {
        int t = 0;
#pragma unroll
        for (int w = 0; w < ES_W; ++w)
            t += whist[w][g];
        tot[g] = t;
    }
    __syncthreads();
    scan_lds<ES_NT>(tot, bins, tmp, tid);
    for (int g = tid; g < bins; g += ES_NT) {
        int at = b0 + tot[g];
#pragma unroll
        for (int w = 0; w < ES_W; ++w) {
            const int x = whist[w][g];
            whist[w][g] = at;
            at += x;
        }
    }
    __syncthreads();
    place_items(w0, w1, lane, a.hi_bits, whist[wave], bin, [&](int64_t i, int p) STG_AI {
        const int t = a.binned[b0 + i];
        a.order[p] = t;
        a.key[p] = embed_id(a, t);
    });
}

// ---------------------------------------------------------------- gradient: sums

// A wave's run of EMBED_RUN sorted positions, 512 columns (blockIdx.y).  Sums
// of ids that begin or end outside the run go to part[run][0] (from the run's
// first position) or [1].
template <int YK, int DK>
__global__ __launch_bounds__(256) void k_embed_runs(EmbedArgs a)
{
    const int lane = threadIdx.x & 63;
    const int n = a.bounds[1 << a.lo_bits];
    const int64_t run = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t p0 = run * EMBED_RUN;
    if (p0 >= n)
        return;
    const int cnt = (int)min((int64_t)EMBED_RUN, n - p0);
    // lane i: position p0 + i - 1
    const int64_t at = p0 + lane - 1;
    const int key = at >= 0 && at < n && lane < cnt + 2 ? a.key[at] : -1;
    const int tok = lane >= 1 && lane <= cnt ? a.order[at] : 0;
    const int64_t c = ((int64_t)blockIdx.y * 64 + lane) * 8;
    const int nc = (int)min((int64_t)8, a.cols - c); // (may be negative)
    float acc[8] = {};
    int first = 1; // of the id's positions in this run, as a lane
    constexpr int B = 8;
    for (int i0 = 1; i0 <= cnt; i0 += B) {
        float f[B][8];
#pragma unroll
        for (int q = 0; q < B; ++q)
            if (i0 + q <= cnt && nc > 0)
                load8f<YK>(a.in, (int64_t)__builtin_amdgcn_readlane(tok, i0 + q) * a.ld_in + c, nc,
                           f[q]);
#pragma unroll
        for (int q = 0; q < B; ++q) {
            const int i = i0 + q;
            if (i > cnt)
                break;
            const int k = __builtin_amdgcn_readlane(key, i);
            const int next = __builtin_amdgcn_readlane(key, i + 1);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[e] += f[q][e];
            if (i < cnt && next == k)
                continue;
            if (nc > 0) {
                const bool before = first == 1 && __builtin_amdgcn_readlane(key, 0) == k;
                if (before || next == k)
                    store8f<OUT_F32>(a.part, (run * 2 + (first > 1)) * a.cols + c, nc, acc);
                else
                    put_row<DK>(a, k, c, nc, acc);
            }
            first = i + 1;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[e] = 0.0f;
        }
    }
}

// The rows whose sums reach over several runs: a workgroup per run that such
// a row begins in, eight waves each taking an eighth of the runs it goes on in.
template <int DK>
__global__ __launch_bounds__(512) void k_embed_join(EmbedArgs a)
{
    __shared__ float red[8][64][9];
    __shared__ int more;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = a.bounds[1 << a.lo_bits];
    const int64_t run = blockIdx.x, p0 = run * EMBED_RUN, p1 = p0 + EMBED_RUN;
    if (p1 >= n)
        return;
    const int k = a.key[p1];
    if (a.key[p1 - 1] != k)
        return;
    // it begins here: some position of the run has another id, or the one
    // before the run
    const int64_t at = p0 - 1 + lane;
    const uint64_t other = __ballot(lane <= EMBED_RUN && (at < 0 || a.key[at] != k));
    if (!other)
        return;
    const int slot = (other >> 1) != 0; // (a position of the run itself)
    // the runs after it that begin with the id
    int runs = 0;
    for (;;) {
        const int64_t p = p1 + (int64_t)(runs + tid) * EMBED_RUN;
        const bool same = p < n && a.key[p] == k;
        if (tid == 0)
            more = 0;
        __syncthreads();
        const uint64_t m = __ballot(same);
        if (lane == 0 && m)
            atomicAdd(&more, __popcll(m));
        __syncthreads();
        const int x = more;
        __syncthreads();
        runs += x;
        if (x < 512)
            break;
    }
    const int64_t c = ((int64_t)blockIdx.y * 64 + lane) * 8;
    const int nc = (int)min((int64_t)8, a.cols - c);
    // part 0 is this run's, part i run + i's
    const int total = runs + 1, per = (total + 7) / 8;
    const int e1 = min(total, (wave + 1) * per);
    float acc[8] = {};
    if (nc > 0)
        for (int i0 = wave * per; i0 < e1; i0 += 4) {
            float f[4][8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + q;
                if (i < e1)
                    load8f<OUT_F32>(a.part, ((run + i) * 2 + (i == 0 ? slot : 0)) * a.cols + c, nc,
                                    f[q]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i0 + q < e1)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[e] += f[q][e];
        }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        red[wave][lane][e] = acc[e];
    __syncthreads();
    if (wave == 0 && nc > 0) {
#pragma unroll
        for (int w = 1; w < 8; ++w)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[e] += red[w][lane][e];
        put_row<DK>(a, k, c, nc, acc);
    }
}

// ---------------------------------------------------------------- launch

// f(kind) with the kind as a constant.
template <class F>
static void with_kind(int kind, F &&f)
{
    if (kind == OUT_F32)
        f(std::integral_constant<int, OUT_F32>{});
    else if (kind == OUT_F16)
        f(std::integral_constant<int, OUT_F16>{});
    else
        f(std::integral_constant<int, OUT_BF16>{});
}

// Workgroups for n tokens, `per` of them each; past 2^18 they take several.
static unsigned blocks(int64_t n, int per)
{
    const int64_t b = (n + per - 1) / per;
    return (unsigned)(b < (1 << 18) ? b : (1 << 18));
}

hipError_t launch_embed(const EmbedArgs &a, hipStream_t s)
{
    with_kind(a.e_kind, [&](auto ek) {
        with_kind(a.y_kind, [&](auto yk) {
            constexpr int EK = decltype(ek)::value, YK = decltype(yk)::value;
            // (cols <= 2^23: at most 2^14 column parts)
            auto go = [&](auto tpr) {
                constexpr int TPR = decltype(tpr)::value;
                const dim3 grid(blocks(a.tokens, 256 / TPR),
                                (unsigned)((a.cols + 8 * TPR - 1) / (8 * TPR)));
                hipLaunchKernelGGL((k_embed<EK, YK, TPR>), grid, dim3(256), 0, s, a);
            };
            if (a.cols <= 128)
                go(std::integral_constant<int, 16>{});
            else
                go(std::integral_constant<int, 64>{});
        });
    });
    return hipGetLastError();
}

hipError_t launch_embed_backward(const EmbedArgs &a, hipStream_t s)
{
    const unsigned parts = (unsigned)((a.cols + 511) / 512);
    if (a.tokens <= EMBED_SMALL) {
        const int64_t zero = a.accumulate ? 0 : (a.vocab + EMBED_ZR - 1) / EMBED_ZR;
        if (a.tokens + zero == 0)
            return hipSuccess;
        with_kind(a.y_kind, [&](auto yk) {
            with_kind(a.e_kind, [&](auto dk) {
                hipLaunchKernelGGL((k_embed_grad_small<decltype(yk)::value, decltype(dk)::value>),
                                   dim3((unsigned)(a.tokens + zero), parts), dim3(256), 0, s, a);
            });
        });
        return hipGetLastError();
    }
    // zeros: about four workgroups per compute unit in each of three launches
    const unsigned zero = a.accumulate ? 0 : 1024;
    hipLaunchKernelGGL(k_embed_count, dim3(a.chunks + zero), dim3(ES_NT), 0, s, a);
    hipLaunchKernelGGL(k_embed_place, dim3(a.chunks + zero), dim3(ES_NT), 0, s, a);
    hipLaunchKernelGGL(k_embed_group, dim3((1u << a.lo_bits) + zero), dim3(ES_NT), 0, s, a);
    const int64_t runs = (a.tokens + EMBED_RUN - 1) / EMBED_RUN;
    with_kind(a.e_kind, [&](auto dk) {
        constexpr int DK = decltype(dk)::value;
        with_kind(a.y_kind, [&](auto yk) {
            hipLaunchKernelGGL((k_embed_runs<decltype(yk)::value, DK>),
                               dim3((unsigned)((runs + 3) / 4), parts), dim3(256), 0, s, a);
        });
        hipLaunchKernelGGL((k_embed_join<DK>), dim3((unsigned)runs, parts), dim3(512), 0, s, a);
    });
    return hipGetLastError();
}

} // namespace stg

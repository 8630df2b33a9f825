// Rows of an embedding table looked up by token, and their gradient.
//
// The lookup Y[t] = s E[id_t] is one pass of 16-byte pieces; bound by memory.
//
// The gradient dE[v] = s sum of dY[t] over the tokens t of row v needs the
// tokens grouped by row.  For few tokens (embed_small) one launch does it without
// a sort, behind one that writes the zeros if the whole gradient is written: a
// workgroup per token looks through all ids, leaves if an earlier token has its
// id, and sums the rows of the later ones otherwise.  More tokens are sorted in
// two stable passes, by the low bits of the id (counts and places of chunks, as
// the routing's sort) and, a workgroup per bin, by the high bits.  (One launch,
// in which a workgroup per bin picked its tokens from all ids, took 64 us for
// 50000 tokens, the three 40.)  A wave then sums the rows of EMBED_RUN sorted
// positions; sums of a row that reach over several runs (a frequent token) are
// left in the workspace and joined by a last launch.  Every sum's order is a
// function of the ids alone.
//
// Where the whole gradient is written, zeros go to all of dE beside the
// sort's launches, which leave most of the chip idle, and the rows that have
// tokens are written after them.
#include <climits>

#include "device_common.hpp"
#include "sort_util.hpp"
#include "vec16.hpp"
#include "vocab_id.hpp"

namespace stg {

typedef EmbedArgs::Binned Binned;

// ---------------------------------------------------------------- eight values

struct __attribute__((packed, aligned(4))) f4_any_t {
    f4_t v;
};

constexpr int elem_bytes(int kind) { return kind == OUT_F32 ? 4 : 2; }

// Elements off .. off + 7 of an array of kind K, as they lie in memory.  Loads
// are kept apart from what becomes of them, and free of branches, so that
// several are in flight: a branch per load made the gradient's sums six times
// as long.
template <int K>
struct Raw8 {
    u4_t v[elem_bytes(K) / 2];
};

// FULL: all eight exist; else the first n (0 .. 7), zeros after them.
template <int K, bool FULL>
__device__ STG_AI inline Raw8<K> load_raw(const void *base, int64_t off, int n)
{
    Raw8<K> r;
    if constexpr (FULL) {
        const uint8_t *p = (const uint8_t *)base + off * elem_bytes(K);
#pragma unroll
        for (int i = 0; i < elem_bytes(K) / 2; ++i)
            r.v[i] = ((const u4_any_t *)(p + 16 * i))->v;
    } else if constexpr (K == OUT_F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r.v[e >> 2][e & 3] = e < n ? ((const uint32_t *)base)[off + e] : 0;
    } else {
        r.v[0] = u4_t{};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n)
                r.v[0][e >> 1] |= (uint32_t)((const uint16_t *)base)[off + e] << (16 * (e & 1));
    }
    return r;
}

template <int K>
__device__ STG_AI inline void widen_raw(const Raw8<K> &r, float (&f)[8])
{
    if constexpr (K == OUT_F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t w = r.v[e >> 2][e & 3];
            f[e] = __builtin_bit_cast(float, w);
        }
    } else {
        widen8<K == OUT_BF16>(r.v[0], f);
    }
}

// The columns of a lane: elements e0 .. 7 of the eight from column c on (e0 8:
// none).  A row's last lane takes the row's last eight columns, of which the
// first e0 belong to the lane before it, so that every lane loads whole pieces;
// rows of less than eight columns (FULL false) have one lane with n of them.
struct Cols {
    int64_t c;
    int e0, n;
};
__device__ STG_AI inline Cols lane_cols(const EmbedArgs &a, int64_t c)
{
    if (a.cols < 8)
        return {0, c == 0 ? 0 : 8, c == 0 ? (int)a.cols : 0};
    const int64_t left = a.cols - c;
    return {min(c, a.cols - 8), left >= 8 ? 0 : left > 0 ? 8 - (int)left : 8, 8};
}
template <class F>
__device__ STG_AI inline void with_full(const EmbedArgs &a, F &&f)
{
    if (a.cols >= 8)
        f(std::true_type{});
    else
        f(std::false_type{});
}

// A lane's columns of the row at element `row`.
template <int K, bool FULL>
__device__ STG_AI inline Raw8<K> load_cols(const void *base, int64_t row, const Cols &k)
{
    return load_raw<K, FULL>(base, row + k.c, k.n);
}
// NT: past the caches.
template <int K, bool FULL, bool NT = false>
__device__ STG_AI inline void store_cols(void *base, int64_t row, const Cols &k, const float (&f)[8])
{
    uint8_t *const p = (uint8_t *)base + (row + k.c) * elem_bytes(K);
    auto put = [](void *q, u4_t v) STG_AI {
        if constexpr (NT)
            __builtin_nontemporal_store(v, &((u4_any_t *)q)->v);
        else
            ((u4_any_t *)q)->v = v;
    };
    u4_t v[elem_bytes(K) / 2];
    if constexpr (K == OUT_F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            v[i] = __builtin_bit_cast(u4_t, f4_t{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]});
    } else {
        v[0] = narrow8<K == OUT_BF16>(f);
    }
    if (FULL && k.e0 == 0) {
#pragma unroll
        for (int i = 0; i < elem_bytes(K) / 2; ++i)
            put(p + 16 * i, v[i]);
    } else if (k.e0 < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= k.e0 && (FULL || e < k.n)) {
                if constexpr (K == OUT_F32)
                    ((float *)p)[e] = f[e];
                else
                    ((uint16_t *)p)[e] = (uint16_t)(v[0][e >> 1] >> (16 * (e & 1)));
            }
    }
}

// Token t's row of the table, -1 for an id that names none.
__device__ STG_AI inline int embed_id(const EmbedArgs &a, int64_t t)
{
    return vocab_id(a.ids, a.id8, a.vocab, t);
}

// ---------------------------------------------------------------- lookup

// TPR lanes per token and blockIdx.y's part of the columns, eight columns and
// U tokens per lane.  Y goes past the caches (NT) where it is larger than all
// L2 together: 16384 tokens of 4096 columns 58 -> 41 us; rows that do not begin on
// cache lines too: 53055 of 4791 266 -> 241, 29397 of 7898 237 -> 220.
template <int EK, int YK, int TPR, int U, bool NT>
__global__ __launch_bounds__(256) void k_embed(EmbedArgs a)
{
    const Cols k = lane_cols(a, ((int64_t)blockIdx.y * TPR + threadIdx.x % TPR) * 8);
    const int64_t first = ((int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR) * U;
    with_full(a, [&](auto full) STG_AI {
        constexpr bool FULL = decltype(full)::value;
        for (int64_t t = first; t < a.tokens; t += (int64_t)gridDim.x * (256 / TPR) * U) {
            int id[U];
            Raw8<EK> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                id[u] = t + u < a.tokens ? embed_id(a, t + u) : -1;
            // (a table without rows has no ids; an id without a row reads row 0)
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (a.vocab > 0)
                    r[u] = load_cols<EK, FULL>(a.in, (id[u] < 0 ? 0 : id[u]) * a.ld_in, k);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[8] = {};
                if (id[u] >= 0) {
                    widen_raw<EK>(r[u], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] *= a.scale;
                }
                if (t + u < a.tokens)
                    store_cols<YK, FULL, NT>(a.out, (t + u) * a.ld_out, k, f);
            }
        }
    });
}

// ---------------------------------------------------------------- gradient: rows

// dE's row v, this lane's columns, from the sum of its tokens' rows; d: what
// it held, if added to.
template <int DK, bool FULL>
__device__ STG_AI inline void put_row(const EmbedArgs &a, int64_t v, const Cols &k, float (&f)[8],
                                      const Raw8<DK> &d)
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] *= a.scale;
    if (a.accumulate) {
        float x[8];
        widen_raw<DK>(d, x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] += x[e];
    }
    store_cols<DK, FULL>(a.out, v * a.ld_out, k, f);
}
template <int DK, bool FULL>
__device__ STG_AI inline Raw8<DK> get_row(const EmbedArgs &a, int64_t v, const Cols &k)
{
    Raw8<DK> d{};
    if (a.accumulate)
        d = load_cols<DK, FULL>(a.out, v * a.ld_out, k);
    return d;
}

// Zeros to rows of dE, by the workgroups of a launch from number `first` (a
// multiple of 8) on.  Packed rows are one stretch: every XCD (workgroups go to
// the eight in turn) fills an eighth, whole cache lines of it, 16 bytes per
// thread and a workgroup for each 16 bytes of NT threads.  1 GB in three
// launches takes 165 us so; 203 by 512 workgroups that loop; 259 with eighths
// that begin off the lines; 276 where each workgroup finds its bounds from the
// sizes by itself.  Non-temporal: the rows that are summed next keep the caches
// (131072 x 2048 fp32 of 16384 tokens 228 -> 222 us, 50021 x 776 fp16 of 50000
// tokens 88 -> 76).
struct ZeroArgs {
    int first;        // INT_MAX: nothing to fill
    uint8_t *at;      // the line that the stretch begins in; rows: the first
    uint8_t *lo, *hi; // the stretch
    int64_t per;      // bytes of an eighth, whole lines; rows: rows of an eighth
    int64_t rows, row, pitch; // rows that are not packed: how many, bytes, bytes apart (else rows 0)
};
template <int NT>
__device__ STG_AI inline void fill_zeros(const ZeroArgs &z)
{
    const int64_t xcd = blockIdx.x & 7, me = (blockIdx.x - z.first) >> 3;
    const int64_t all = (gridDim.x - z.first) >> 3;
    // 16 aligned bytes at p, as far as they lie in [lo, hi)
    auto zero = [&](uint8_t *p, uint8_t *lo, uint8_t *hi) STG_AI {
        if (p >= lo && p + 16 <= hi)
            __builtin_nontemporal_store(u4_t{}, (u4_t *)p);
        else
            for (int i = 0; i < 16; i += 2)
                if (p + i >= lo && p + i < hi)
                    *(uint16_t *)(p + i) = 0;
    };
    if (z.rows == 0) {
        uint8_t *const e = z.at + (xcd + 1) * z.per, *const hi = e < z.hi ? e : z.hi;
        for (uint8_t *p = z.at + xcd * z.per + (me * NT + threadIdx.x) * 16; p < hi; p += all * NT * 16)
            zero(p, z.lo, hi);
    } else {
        const int64_t e = min(z.rows, (xcd + 1) * z.per);
        for (int64_t r = xcd * z.per + me * (NT / 64) + (threadIdx.x >> 6); r < e; r += all * (NT / 64)) {
            uint8_t *const lo = z.at + r * z.pitch, *const hi = lo + z.row; // a wave per row
            for (uint8_t *p = (uint8_t *)((uintptr_t)lo & ~(uintptr_t)15) + (threadIdx.x & 63) * 16; p < hi;
                 p += 64 * 16)
                zero(p, lo, hi);
        }
    }
}

// ---------------------------------------------------------------- gradient: few tokens

// dE's zeros, alone.
__global__ __launch_bounds__(512) void k_embed_zero(ZeroArgs z) { fill_zeros<512>(z); }

// The row of token blockIdx.x, if it is the first of its id: P parts of 512
// columns (a wave's 64 x 8), four waves each.  Bound by its chain of latencies (the
// token's own row, and dE's, are loaded beside the search), and by the search
// where there are many: a workgroup per part took 8.9 us for 512 tokens of 2048
// columns, one for the four 6.8, and 56 and 26 for 2048 of 1104.  MAX: tokens.
template <int YK, int DK, int P, int MAX>
__global__ __launch_bounds__(256 * P) void k_embed_grad_small(EmbedArgs a)
{
    constexpr int NT = 256 * P, NW = 4 * P, PER = MAX / NT;
    __shared__ int found[PER * NW];
    __shared__ int list[MAX];
    __shared__ float red[NW][64][9]; // (9: the lanes' eight values on all banks)
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int part = wave % P, quarter = wave / P;
    const int T = (int)a.tokens, me = blockIdx.x;
    int id[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        id[i] = i * NT + tid < T ? embed_id(a, i * NT + tid) : -1;
    const Cols k = lane_cols(a, (((int64_t)blockIdx.y * P + part) * 64 + lane) * 8);
    const int mine = embed_id(a, me);
    if (mine < 0)
        return;
    with_full(a, [&](auto full) STG_AI {
        constexpr bool FULL = decltype(full)::value;
        const Raw8<YK> own = load_cols<YK, FULL>(a.in, me * a.ld_in, k);
        const Raw8<DK> old = get_row<DK, FULL>(a, mine, k);
        // tokens of this id by their numbers; an earlier one has the row
        bool early = false;
        uint64_t m[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool same = id[i] == mine;
            early |= same && i * NT + tid < me;
            m[i] = __ballot(same);
            if (lane == 0)
                found[i * NW + wave] = __popcll(m[i]);
        }
        if (__syncthreads_or(early))
            return;
        int n = 0;
        for (int j = 0; j < PER * NW; ++j) {
            const int x = found[j];
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (j == i * NW + wave && (m[i] >> lane & 1))
                    list[n + lanes_below(m[i])] = i * NT + tid;
            n += x;
        }
        float acc[8];
        if (n == 1) {
            if (quarter == 0) {
                widen_raw<YK>(own, acc);
                put_row<DK, FULL>(a, mine, k, acc, old);
            }
            return;
        }
        __syncthreads();
        // a quarter of the rows per wave of a part, eight in flight; joined in order
        const int per = n >= 16 ? (n + 3) / 4 : n, end = min(n, (quarter + 1) * per);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc[e] = 0.0f;
        for (int k0 = quarter * per; k0 < end; k0 += 8) {
            Raw8<YK> r[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) // (past the end: the last one again)
                r[q] = load_cols<YK, FULL>(a.in, list[min(k0 + q, end - 1)] * a.ld_in, k);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (k0 + q < end) {
                    float f[8];
                    widen_raw<YK>(r[q], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[e] += f[e];
                }
        }
        if (n >= 16) {
            if (quarter)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    red[wave][lane][e] = acc[e];
            __syncthreads();
            if (quarter == 0)
#pragma unroll
                for (int w = 1; w < 4; ++w)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[e] += red[w * P + part][lane][e];
        }
        if (quarter == 0)
            put_row<DK, FULL>(a, mine, k, acc, old);
    });
}

// ---------------------------------------------------------------- gradient: sort

constexpr int ES_NT = 512, ES_W = ES_NT / 64;   // first pass
constexpr int EG_NT = 1024, EG_W = EG_NT / 64; // second

// Tokens per low-bits bin of each chunk.
__global__ __launch_bounds__(ES_NT) void k_embed_count(EmbedArgs a, ZeroArgs z)
{
    __shared__ int hist[EMBED_MAX_BINS];
    if ((int)blockIdx.x >= z.first) {
        fill_zeros<ES_NT>(z);
        return;
    }
    if ((int)blockIdx.x >= a.chunks)
        return;
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

// same_group where most lanes may hold one id (a frequent token's bin): that
// one first, and the others one by one if they are few.
__device__ STG_AI inline uint64_t same_bin(int g, int bits)
{
    uint64_t left = __ballot(g >= 0), same = 0;
    if (!left)
        return 0;
    int lead = __builtin_amdgcn_readlane(g, __builtin_ctzll(left));
    uint64_t m = __ballot(g == lead);
    if (__popcll(left & ~m) > 8)
        return same_group(g, bits);
    for (;;) {
        same = g == lead ? m : same;
        left &= ~m;
        if (!left)
            return same;
        lead = __builtin_amdgcn_readlane(g, __builtin_ctzll(left));
        m = __ballot(g == lead);
    }
}

// One step of 64 items in order: those of bin g (-1: none) to the places
// whist[g] counts up from; the place, or -1.
__device__ STG_AI inline int place_step(int g, int bits, int *whist)
{
    const uint64_t same = same_bin(g, bits);
    const int rank = lanes_below(same);
    int p = -1;
    if (g >= 0)
        p = whist[g] + rank;
    wave_lds_sync();
    if (g >= 0 && rank == 0)
        whist[g] = p + __popcll(same);
    wave_lds_sync();
    return p;
}

// The tokens by the low bits of their ids.  Wave w takes its chunk's w-th
// eighth.
__global__ __launch_bounds__(ES_NT) void k_embed_place(EmbedArgs a, ZeroArgs z)
{
    // (no more LDS than the bins need: the zeros' workgroups reserve it too)
    extern __shared__ int lds[];
    if ((int)blockIdx.x >= z.first) {
        fill_zeros<ES_NT>(z);
        return;
    }
    if ((int)blockIdx.x >= a.chunks)
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int bins = 1 << a.lo_bits, me = blockIdx.x;
    int *const tmp = lds, *const tot = tmp + ES_W, *const bef = tot + bins + 1;
    auto whist = [&](int w) STG_AI { return bef + bins + w * bins; };
    for (int g = tid; g < bins; g += ES_NT) {
        tot[g] = bef[g] = 0;
#pragma unroll
        for (int w = 0; w < ES_W; ++w)
            whist(w)[g] = 0;
    }
    __syncthreads();
    const int per = a.chunk / ES_W; // a multiple of 64
    const int64_t w0 = (int64_t)me * a.chunk + (int64_t)wave * per;
    const int64_t w1 = min(w0 + per, a.tokens);
    auto bin = [&](int64_t t) STG_AI {
        const int v = t < w1 ? embed_id(a, t) : -1;
        return v >= 0 ? v & (bins - 1) : -1;
    };
    for (int64_t t = w0 + lane; t - lane < w1; t += 64) {
        const int g = bin(t);
        if (g >= 0)
            atomicAdd(&whist(wave)[g], 1);
    }
    // all chunks' counts: neighbouring threads take neighbouring bins, the
    // others further chunks
    int gp = 64;
    while (gp < bins && gp < ES_NT)
        gp *= 2;
    const int parts = ES_NT / gp;
    for (int g = tid % gp; g < bins; g += gp) {
        int t = 0, b = 0;
        for (int c0 = tid / gp; c0 < a.chunks; c0 += 8 * parts) {
            int v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) { // (eight loads in flight)
                const int c = c0 + q * parts;
                v[q] = a.counts[(int64_t)min(c, a.chunks - 1) * bins + g];
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int c = c0 + q * parts;
                t += c < a.chunks ? v[q] : 0;
                b += c < me ? v[q] : 0;
            }
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
            const int n = whist(w)[g];
            whist(w)[g] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int64_t t = w0 + lane; t - lane < w1; t += 64) {
        const int p = place_step(bin(t), a.lo_bits, whist(wave));
        if (p >= 0)
            a.binned[p] = Binned{embed_id(a, t), (int)t};
    }
}

// One bin's tokens by the high bits of their ids.  Wave w takes the bin's w-th
// sixteenth, up to EG_STEPS steps of 64 from registers (the bin of a token
// that is a third of 50000: 14 us instead of 30 with a load per step).  Sixteen steps
// are 32 of the 128 registers that a thread of 1024 may have; a bin of more than
// 16384 tokens loads at each step (the whole gradient of 160 columns with 16000
// tokens in one bin 54 us, with 17000 64, with 48000 120).
constexpr int EG_STEPS = 16;
__global__ __launch_bounds__(EG_NT) void k_embed_group(EmbedArgs a, ZeroArgs z)
{
    extern __shared__ int lds[];
    const int lows = 1 << a.lo_bits;
    if ((int)blockIdx.x >= z.first) {
        fill_zeros<EG_NT>(z);
        return;
    }
    if ((int)blockIdx.x >= lows)
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int bins = 1 << a.hi_bits;
    int *const tmp = lds, *const tot = tmp + EG_W;
    auto whist = [&](int w) STG_AI { return tot + bins + 1 + w * bins; };
    const int b0 = a.bounds[blockIdx.x], n = a.bounds[blockIdx.x + 1] - b0;
    if (n <= 0)
        return;
    const int per = ((n + EG_W - 1) / EG_W + 63) / 64 * 64;
    const int w0 = min(n, wave * per), w1 = min(n, w0 + per);
    const bool held = per <= 64 * EG_STEPS;
    Binned x[EG_STEPS];
    if (held)
#pragma unroll
        for (int q = 0; q < EG_STEPS; ++q)
            x[q] = a.binned[b0 + min(w0 + 64 * q + lane, n - 1)];
    // f(item, whether it exists) for the wave's items, 64 a step
    auto each = [&](auto &&f) STG_AI {
        if (held) {
#pragma unroll
            for (int q = 0; q < EG_STEPS; ++q)
                if (w0 + 64 * q < w1)
                    f(x[q], w0 + 64 * q + lane < w1);
        } else {
            for (int i = w0 + lane; i - lane < w1; i += 64)
                f(a.binned[b0 + min(i, n - 1)], i < w1);
        }
    };
    for (int g = tid; g < bins; g += EG_NT)
#pragma unroll
        for (int w = 0; w < EG_W; ++w)
            whist(w)[g] = 0;
    __syncthreads();
    each([&](const Binned &y, bool in) STG_AI {
        // (one addition per id: 64 to one address take a turn each)
        const int g = in ? y.id >> a.lo_bits : -1;
        const uint64_t same = same_bin(g, a.hi_bits);
        if (g >= 0 && lanes_below(same) == 0)
            whist(wave)[g] += __popcll(same);
        wave_lds_sync();
    });
    __syncthreads();
    for (int g = tid; g < bins; g += EG_NT) {
        int t = 0;
#pragma unroll
        for (int w = 0; w < EG_W; ++w)
            t += whist(w)[g];
        tot[g] = t;
    }
    __syncthreads();
    scan_lds<EG_NT>(tot, bins, tmp, tid);
    for (int g = tid; g < bins; g += EG_NT) {
        int at = b0 + tot[g];
#pragma unroll
        for (int w = 0; w < EG_W; ++w) {
            const int n1 = whist(w)[g];
            whist(w)[g] = at;
            at += n1;
        }
    }
    __syncthreads();
    each([&](const Binned &y, bool in) STG_AI {
        const int p = place_step(in ? y.id >> a.lo_bits : -1, a.hi_bits, whist(wave));
        if (p >= 0) {
            a.order[p] = y.token;
            a.key[p] = y.id;
        }
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
    const int64_t run = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t p0 = run * EMBED_RUN;
    // lane i: position p0 + i - 1 (loaded beside n; past it there is nothing)
    const int64_t at = min(max(p0 + lane - 1, (int64_t)0), a.tokens - 1);
    int key = a.key[at], tok = a.order[at];
    const int n = a.bounds[1 << a.lo_bits];
    if (p0 >= n)
        return;
    const int cnt = (int)min((int64_t)EMBED_RUN, n - p0);
    key = p0 + lane >= 1 && p0 + lane <= n && lane < cnt + 2 ? key : -1;
    tok = lane >= 1 && lane <= cnt ? tok : 0;
    const Cols k = lane_cols(a, ((int64_t)blockIdx.y * 64 + lane) * 8);
    with_full(a, [&](auto full) STG_AI {
        constexpr bool FULL = decltype(full)::value;
        // (32 rows of 16 bits at once: a load behind a store waits for it)
        constexpr int B = YK == OUT_F32 ? 8 : 16;
        auto load = [&](Raw8<YK>(&r)[B], int i0) STG_AI {
#pragma unroll
            for (int q = 0; q < B; ++q) { // (past the end: the last one again)
                const int t = __builtin_amdgcn_readlane(tok, min(i0 + q, cnt));
                r[q] = load_cols<YK, FULL>(a.in, t * a.ld_in, k);
            }
        };
        float acc[8] = {};
        int first = 1; // of the id's positions in this run, as a lane
        auto add = [&](const Raw8<YK>(&r)[B], int i0) STG_AI {
#pragma unroll
            for (int q = 0; q < B; ++q) {
                const int i = i0 + q;
                if (i <= cnt) {
                    const int id = __builtin_amdgcn_readlane(key, i);
                    const int next = __builtin_amdgcn_readlane(key, i + 1);
                    float f[8];
                    widen_raw<YK>(r[q], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[e] += f[e];
                    if (i == cnt || next != id) {
                        const bool before = first == 1 && __builtin_amdgcn_readlane(key, 0) == id;
                        if (before || next == id) {
                            store_cols<OUT_F32, FULL>(a.part, (run * 2 + (first > 1)) * a.cols, k,
                                                      acc);
                        } else {
                            put_row<DK, FULL>(a, id, k, acc, get_row<DK, FULL>(a, id, k));
                        }
                        first = i + 1;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            acc[e] = 0.0f;
                    }
                }
            }
        };
        Raw8<YK> r0[B], r1[B];
        load(r0, 1);
        for (int i0 = 1; i0 <= cnt; i0 += 2 * B) {
            if (i0 + B <= cnt)
                load(r1, i0 + B);
            add(r0, i0);
            if (i0 + 2 * B <= cnt)
                load(r0, i0 + 2 * B);
            if (i0 + B <= cnt)
                add(r1, i0 + B);
        }
    });
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
    // lane i: position p0 + i - 1, up to p1
    const int64_t at = p0 - 1 + lane;
    const int key = at >= 0 && lane <= EMBED_RUN + 1 ? a.key[at] : -1;
    const int id = __builtin_amdgcn_readlane(key, EMBED_RUN + 1);
    if (__builtin_amdgcn_readlane(key, EMBED_RUN) != id)
        return;
    // it begins here: some position of the run has another id, or the one
    // before the run
    const uint64_t other = __ballot(lane <= EMBED_RUN && key != id);
    if (!other)
        return;
    const int slot = (other >> 1) != 0; // (a position of the run itself)
    // the runs after it that begin with the id
    int runs = 0;
    for (;;) {
        const int64_t p = p1 + (int64_t)(runs + tid) * EMBED_RUN;
        const bool same = p < n && a.key[p] == id;
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
    const Cols k = lane_cols(a, ((int64_t)blockIdx.y * 64 + lane) * 8);
    with_full(a, [&](auto full) STG_AI {
        constexpr bool FULL = decltype(full)::value;
        const Raw8<DK> old = get_row<DK, FULL>(a, id, k);
        // part 0 is this run's, part i run + i's
        const int total = runs + 1, per = (total + 7) / 8;
        const int i1 = min(total, (wave + 1) * per);
        float acc[8] = {};
        constexpr int B = 8;
        for (int i0 = wave * per; i0 < i1; i0 += B) {
            Raw8<OUT_F32> r[B];
#pragma unroll
            for (int q = 0; q < B; ++q) {
                const int i = min(i0 + q, i1 - 1);
                r[q] = load_cols<OUT_F32, FULL>(a.part,
                                                ((run + i) * 2 + (i == 0 ? slot : 0)) * a.cols, k);
            }
#pragma unroll
            for (int q = 0; q < B; ++q)
                if (i0 + q < i1) {
                    float f[8];
                    widen_raw<OUT_F32>(r[q], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[e] += f[e];
                }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            red[wave][lane][e] = acc[e];
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int w = 1; w < 8; ++w)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[e] += red[w][lane][e];
            put_row<DK, FULL>(a, id, k, acc, old);
        }
    });
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
            auto go = [&](auto tpr, auto uc, auto nt) {
                constexpr int TPR = decltype(tpr)::value, U = decltype(uc)::value;
                constexpr bool NT = decltype(nt)::value;
                const dim3 grid(blocks(a.tokens, 256 / TPR * U),
                                (unsigned)((a.cols + 8 * TPR - 1) / (8 * TPR)));
                hipLaunchKernelGGL((k_embed<EK, YK, TPR, U, NT>), grid, dim3(256), 0, s, a);
            };
            using I = std::integral_constant<int, 1>;
            using I4 = std::integral_constant<int, 4>;
            using I16 = std::integral_constant<int, 16>;
            using I64 = std::integral_constant<int, 64>;
            const int64_t n = a.tokens * a.cols;
            const bool many = n >= (int64_t)1 << 22, nt = n * elem_bytes(YK) >= (int64_t)32 << 20;
            if (nt)
                a.cols <= 128 ? go(I16{}, I4{}, std::true_type{}) : go(I64{}, I4{}, std::true_type{});
            else if (many)
                a.cols <= 128 ? go(I16{}, I4{}, std::false_type{}) : go(I64{}, I4{}, std::false_type{});
            else
                a.cols <= 128 ? go(I16{}, I{}, std::false_type{}) : go(I64{}, I{}, std::false_type{});
        });
    });
    return hipGetLastError();
}

hipError_t launch_embed_backward(const EmbedArgs &a, hipStream_t s)
{
    const unsigned parts = (unsigned)((a.cols + 511) / 512);
    // rows [r0, r1) of dE's zeros by workgroups of nt threads behind `sorters`
    auto zeros = [&](int64_t r0, int64_t r1, int sorters, int nt, ZeroArgs &z) {
        const int64_t eb = elem_bytes(a.e_kind), rows = r1 - r0;
        z.first = (sorters + 7) / 8 * 8;
        z.lo = z.at = (uint8_t *)a.out + r0 * a.ld_out * eb;
        int64_t wgs;
        if (a.ld_out == a.cols) {
            z.hi = z.lo + rows * a.cols * eb;
            z.at = (uint8_t *)((uintptr_t)z.lo & ~(uintptr_t)127);
            z.per = ((z.hi - z.at + 7) / 8 + 127) / 128 * 128;
            wgs = (z.per + nt * 16 - 1) / (nt * 16);
        } else {
            z.rows = rows;
            z.row = a.cols * eb;
            z.pitch = a.ld_out * eb;
            z.per = (rows + 7) / 8;
            wgs = (z.per + nt / 64 - 1) / (nt / 64);
        }
        return z.first - sorters + 8 * (unsigned)(wgs < (1 << 16) ? wgs : 1 << 16);
    };
    if (embed_small(a.tokens, a.cols)) {
        if (!a.accumulate) {
            ZeroArgs z{};
            const unsigned n = zeros(0, a.vocab, 0, 512, z);
            hipLaunchKernelGGL(k_embed_zero, dim3(n), dim3(512), 0, s, z);
        }
        if (a.tokens > 0)
            with_kind(a.y_kind, [&](auto yk) {
                with_kind(a.e_kind, [&](auto dk) {
                    constexpr int YK = decltype(yk)::value, DK = decltype(dk)::value;
                    auto go = [&](auto pc) {
                        constexpr int P = decltype(pc)::value;
                        const dim3 grid((unsigned)a.tokens, (parts + P - 1) / P), block(256 * P);
                        if (a.tokens <= 1024)
                            hipLaunchKernelGGL((k_embed_grad_small<YK, DK, P, 1024>), grid, block, 0, s, a);
                        else
                            hipLaunchKernelGGL((k_embed_grad_small<YK, DK, P, 2048>), grid, block, 0, s, a);
                    };
                    if (parts == 1)
                        go(std::integral_constant<int, 1>{});
                    else if (parts == 2)
                        go(std::integral_constant<int, 2>{});
                    else
                        go(std::integral_constant<int, 4>{});
                });
            });
        return hipGetLastError();
    }
    // a third of dE's zeros beside each of the sort's launches
    auto go = [&](auto kernel, int sorters, int third, int nt, unsigned lds) {
        ZeroArgs z{};
        unsigned n = 0;
        z.first = INT_MAX;
        if (!a.accumulate)
            n = zeros(a.vocab * third / 3, a.vocab * (third + 1) / 3, sorters, nt, z);
        hipLaunchKernelGGL(kernel, dim3(sorters + n), dim3(nt), lds, s, a, z);
    };
    const int lows = 1 << a.lo_bits, highs = 1 << a.hi_bits;
    go(k_embed_count, a.chunks, 0, ES_NT, 0);
    go(k_embed_place, a.chunks, 1, ES_NT, (ES_W + lows + 1 + lows + ES_W * lows) * sizeof(int));
    go(k_embed_group, lows, 2, EG_NT, (EG_W + highs + 1 + EG_W * highs) * sizeof(int));
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

/*
 * gemm_moe.h - C ABI of the operators around a mixture-of-experts MLP
 * (libstgemm.so): routing of tokens to experts and back, the experts'
 * products over ragged groups of rows, and activation checkpoints in 8 bits
 * with their use in the backward pass.
 *
 * The conventions of gemm.h hold: sizes and leading dimensions are in
 * elements, data pointers are device pointers, the caller owns every buffer
 * (these functions allocate nothing and synchronise nothing, so all of them
 * may be captured into a HIP graph), `stream` is a hipStream_t, every
 * function returns a status, and gemm_last_error() explains the last
 * failure.  A leading dimension of 0 means packed.  Pointers need the
 * alignment of their elements only.  An output must not share bytes with an
 * input or with another output (GEMM_ERR_UNSUPPORTED) except where a
 * function says so.  Device data that steers a kernel (expert ids, places,
 * group bounds) is checked by the kernel: values out of range are treated
 * as stated below and never reach memory outside the buffers.
 *
 * The forward pass of one MLP with experts W1_e (K x 2F), W2_e (F x K):
 *     dispatch:  Xs = rows of X sorted by expert            gemm_moe_dispatch
 *     GU = Xs W1 (by group)                          gemm_grouped_run (ROWS)
 *     H = silu(G) * U, checkpoint of GU in 8 bits               gemm_swiglu
 *     Ys = H W2 (by group)                           gemm_grouped_run (ROWS)
 *     Y[t] = sum_k w[t,k] Ys[place of (t,k)]                gemm_moe_combine
 * and its backward pass:
 *     dYs, dw from dY                              gemm_moe_combine_backward
 *     dH = dYs W2^T                    gemm_grouped_run (ROWS, W2 as stored)
 *     dGU, H from the checkpoint                       gemm_swiglu_backward
 *     dW2 = H^T dYs, dW1 = Xs^T dGU               gemm_grouped_run (WEIGHTS)
 *     dXs = dGU W1^T                                 gemm_grouped_run (ROWS)
 *     dX[t] = sum_k dXs[place of (t,k)]     gemm_moe_combine without weights
 */
#ifndef STGEMM_GEMM_MOE_H
#define STGEMM_GEMM_MOE_H

#include <stddef.h>
#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ routing
 *
 * A slot s = t * topk + k is choice k of token t; ids[s] is its expert.  A
 * slot whose id is not in 0 .. groups-1 (dropped by a capacity, padding) has
 * no place.  The other slots are sorted by expert, slots of one expert in
 * ascending order:
 *   offsets[g] (groups + 1 int32): the first sorted row of group g;
 *              offsets[groups] is the number of slots with a place;
 *   order[p]   (tokens * topk int32): the slot at sorted row p, -1 past
 *              offsets[groups];
 *   pos[s]     (tokens * topk int32): the sorted row of slot s, -1 without
 *              a place.
 * The result is a function of the ids alone (no order of arrival enters).
 * Limits: 1 <= groups <= 1024, tokens * topk < 2^31 (GEMM_ERR_UNSUPPORTED
 * above).  ids are int32 (id_bytes 4) or int64 (id_bytes 8). */

/* Bytes of workspace that gemm_moe_sort and gemm_moe_dispatch need for these
 * sizes (may be 0; the pointer may then be NULL).  Its contents need no
 * initialisation and nothing is kept in it from one call to the next; two
 * calls that may overlap in time need two workspaces. */
gemm_status_t gemm_moe_sort_workspace(int64_t tokens, int64_t topk, int64_t groups, size_t *bytes);

/* Enqueue the sort alone: offsets, order and pos from ids. */
gemm_status_t gemm_moe_sort(int64_t tokens, int64_t topk, int64_t groups, int32_t id_bytes,
                            const void *ids, int32_t *offsets, int32_t *order, int32_t *pos,
                            void *workspace, gemm_stream_t stream);

/* Enqueue the sort and Xs[pos[s]] = X[s / topk] for every slot with a place
 * (X: tokens x cols, Xs: tokens * topk rows; rows of Xs past offsets[groups]
 * are not written).  type: GEMM_F16 or GEMM_BF16 (the rows are copied bit by
 * bit). */
gemm_status_t gemm_moe_dispatch(int64_t tokens, int64_t topk, int64_t groups, int64_t cols,
                                int32_t type, int32_t id_bytes, const void *ids, const void *X,
                                int64_t ldx, int32_t *offsets, int32_t *order, int32_t *pos,
                                void *Xs, int64_t ldxs, void *workspace, gemm_stream_t stream);

/* Enqueue Y[t] = sum_k weights[t,k] * Ys[pos[t,k]], summed in fp32 with k
 * ascending and rounded once (weights: fp32, NULL = 1).  A slot whose pos is
 * not in 0 .. rows-1 adds nothing, whatever its weight; a token without any
 * place gets zeros.  Ys: rows x cols. */
gemm_status_t gemm_moe_combine(int64_t tokens, int64_t topk, int64_t cols, int32_t type,
                               const int32_t *pos, const float *weights, const void *Ys,
                               int64_t ldys, int64_t rows, void *Y, int64_t ldy,
                               gemm_stream_t stream);

/* Enqueue the gradient of gemm_moe_combine from dY (tokens x cols):
 *   dYs[pos[s]] = weights[s] * dY[s / topk]   (fp32 product, rounded once)
 *   dw[s] = sum_c Ys[pos[s], c] * dY[s / topk, c]   (fp32, fixed order)
 * A slot without a place gets dw = 0 and writes no row of dYs; rows of dYs
 * no slot points to keep what they held.  Two slots must not share a place
 * (those of gemm_moe_sort never do; the row then holds either's value). */
gemm_status_t gemm_moe_combine_backward(int64_t tokens, int64_t topk, int64_t cols, int32_t type,
                                        const int32_t *pos, const float *weights, const void *dY,
                                        int64_t lddy, const void *Ys, int64_t ldys, int64_t rows,
                                        void *dYs, int64_t lddys, float *dw, gemm_stream_t stream);

/* ------------------------------------------------------------ grouped products
 *
 * `offsets` (groups + 1 int32, device) cuts `rows` rows into groups: group g
 * holds rows offsets[g] .. offsets[g+1] - 1.  Bounds are clamped to 0 ..
 * rows, and a group whose end is before its start is empty.  Groups must not
 * share rows in ROWS mode (ascending bounds never do; rows of several groups
 * get an unspecified one's product, or none).
 *
 * GEMM_GROUPED_ROWS:    D[r] = cast(A[r] * B_g) for the rows r of each group:
 *     A rows x K, D rows x N row-major; B holds `groups` matrices one after
 *     the other, each N x K (b_layout COL_MAJOR, as B of gemm_run, ldb >= K)
 *     or K x N (ROW_MAJOR, ldb >= N).  Rows outside every group are not
 *     written.  b_type = a_type; no C.
 * GEMM_GROUPED_WEIGHTS: D_g = cast(A_g^T * B_g + C_g), the sum over the rows
 *     of group g: A rows x K, B rows x N, D and C hold `groups` K x N
 *     matrices one after the other (ldd; C has D's type and leading
 *     dimension and may be D itself).  A group without rows gives C_g, or 0.
 *     b_type = a_type, or GEMM_F8_E4M3 for a B kept by gemm_q8_store or
 *     gemm_swiglu: then B holds the codes (packed, ldb = N), `scales` their
 *     scales, and each value enters as the one gemm_q8_load of a_type gives.
 *     b_layout is ROW_MAJOR (rows contiguous along N).
 *
 * The fast kernels move 16-byte chunks: K, lda and ldb (and N where B is
 * row-major) in multiples of 8, leading dimensions below 2^21, A and B 16-byte
 * aligned.  Everything else runs a generic kernel, which takes some 30 (ROWS)
 * or 10 (WEIGHTS) times as long on large products (4 groups of 512 rows, 2048 x
 * 2048 bf16: 889 and 31 us, 297 and 28).  Alignment is known at the call only:
 * a plan of any family runs the generic kernel for A or B off 16 bytes, and
 * gemm_grouped_plan_describe names the kernel of aligned ones.
 *
 * a_type GEMM_F16 or GEMM_BF16; d_type GEMM_F32, GEMM_F16 or GEMM_BF16; fp32
 * accumulation, one rounding.  1 <= groups <= 65535; rows, N, K below 2^31;
 * matrices of at most 2^40 elements. */
typedef enum { GEMM_GROUPED_ROWS = 0, GEMM_GROUPED_WEIGHTS = 1 } gemm_grouped_mode_t;

typedef struct {
    int32_t mode;     /* gemm_grouped_mode_t */
    int32_t groups;
    int64_t rows, N, K;
    int32_t a_type, b_type, d_type; /* gemm_dtype_t */
    int32_t b_layout;               /* gemm_layout_t */
    int32_t has_c;                  /* WEIGHTS: add C */
    int32_t algo;                   /* gemm_algo_t: AUTO, or GENERIC, SKINNY (ROWS only),
                                       TILED, TILED_128, TILED_256 to force a family
                                       (GEMM_ERR_UNSUPPORTED if it cannot serve) */
    int64_t lda, ldb, ldd;          /* 0 = packed */
} gemm_grouped_desc_t;

typedef struct gemm_grouped_plan gemm_grouped_plan_t;

/* Validate a descriptor on the host (no device is touched). */
gemm_status_t gemm_grouped_validate_desc(const gemm_grouped_desc_t *desc);

/* Validate, check the device, choose the kernel; the plan (host memory) is
 * immutable, may be shared by threads, and is released with
 * gemm_grouped_plan_destroy.  The choice depends on the descriptor and, at
 * run time, on pointer alignment; never on the group bounds. */
gemm_status_t gemm_grouped_plan(const gemm_grouped_desc_t *desc, gemm_grouped_plan_t **out);
gemm_status_t gemm_grouped_plan_destroy(gemm_grouped_plan_t *plan);
gemm_status_t gemm_grouped_plan_describe(const gemm_grouped_plan_t *plan, char *buf, size_t len);

/* Enqueue the product.  scales: NULL unless b_type is GEMM_F8_E4M3; C: NULL
 * unless has_c. */
gemm_status_t gemm_grouped_run(const gemm_grouped_plan_t *plan, const void *A, const void *B,
                               const uint8_t *scales, const int32_t *offsets, const void *C,
                               void *D, gemm_stream_t stream);

/* ------------------------------------------------------------ 8-bit checkpoints
 *
 * A rows x cols tensor of 16-bit values x is kept as E4M3 codes (rows x cols
 * bytes, packed) and one E8M0 scale per 32 columns of a row (rows x
 * ceil(cols/32) bytes, packed; the last block of a row may be shorter):
 *   amax = the largest finite |x| of the block;
 *   e    = the smallest integer >= -127 with amax <= 448 * 2^e, 0 if amax = 0;
 *   code = E4M3(x * 2^-e), round to nearest even;  scale = e + 127.
 * A NaN or an infinity is kept as the NaN code, so that an overflow stays
 * visible; the other values of its block keep theirs.  The value of a code is
 * E4M3value * 2^(scale - 127); it is brought back to a 16-bit type clamped to
 * the type's finite range and rounded to nearest even (a scale of 255, which
 * is never written, gives NaN). */

/* Enqueue codes and scales of X. */
gemm_status_t gemm_q8_store(int64_t rows, int64_t cols, int32_t type, const void *X, int64_t ldx,
                            uint8_t *codes, uint8_t *scales, gemm_stream_t stream);

/* Enqueue X = the values of codes and scales in `type`. */
gemm_status_t gemm_q8_load(int64_t rows, int64_t cols, int32_t type, const uint8_t *codes,
                           const uint8_t *scales, void *X, int64_t ldx, gemm_stream_t stream);

/* Enqueue H = silu(G) * U, silu(g) = g / (1 + exp(-g)), from GU (rows x
 * 2 cols: G in columns 0 .. cols-1, U in the rest; fp32 arithmetic, one
 * rounding), and the checkpoint of GU (rows x 2 cols, both NULL to keep
 * none). */
gemm_status_t gemm_swiglu(int64_t rows, int64_t cols, int32_t type, const void *GU, int64_t ldgu,
                          void *H, int64_t ldh, uint8_t *codes, uint8_t *scales,
                          gemm_stream_t stream);

/* Enqueue the gradient from the checkpoint of GU and dH (rows x cols), with
 * s = 1 / (1 + exp(-g)):
 *   dG = dH * u * s * (1 + g (1 - s)),  dU = dH * g * s   (dGU: rows x 2 cols)
 * and H = silu(g) * u once more, which the gradient of the next weights
 * reads (NULL: not wanted).  g and u are the codes' values clamped to the
 * type's finite range. */
gemm_status_t gemm_swiglu_backward(int64_t rows, int64_t cols, int32_t type, const uint8_t *codes,
                                   const uint8_t *scales, const void *dH, int64_t lddh, void *dGU,
                                   int64_t lddgu, void *H, int64_t ldh, gemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif

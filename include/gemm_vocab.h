/*
 * gemm_vocab.h - C ABI of the operators over a vocabulary (libstgemm.so): the
 * rows of an embedding table looked up by token and their gradient, and the
 * softmax cross entropy of a linear layer over the vocabulary with its
 * gradients.
 *
 * The conventions of gemm.h hold: sizes and leading dimensions are in
 * elements, data pointers are device pointers, the caller owns every buffer
 * (these functions allocate nothing and synchronise nothing, so all of them
 * may be captured into a HIP graph), `stream` is a hipStream_t, every
 * function returns a status, and gemm_last_error() explains the last
 * failure.  A leading dimension of 0 means packed.  An output must not share
 * bytes with an input or with another output (GEMM_ERR_UNSUPPORTED).  A
 * workspace needs no initialisation and nothing is kept in it from one call
 * to the next; two calls that may overlap in time need two workspaces.
 *
 * Token ids and targets are int32 (id_bytes 4) or int64 (id_bytes 8) device
 * data.  They are checked by the kernels: one that is not in 0 .. vocab-1
 * (padding, a masked token) names no row and never reaches memory.
 *
 * One training step of a model whose table and output layer share a matrix E
 * (vocab x hidden):
 *     X0[t] = s E[id_t]                                        gemm_embed
 *     ... the layers ...
 *     loss, lse from X and E                            gemm_xent_forward
 *     dX, dE from dloss                                gemm_xent_backward
 *     ... the layers' gradients ...
 *     dE += what dX0 adds                    gemm_embed_backward, accumulate
 */
#ifndef STGEMM_GEMM_VOCAB_H
#define STGEMM_GEMM_VOCAB_H

#include <stddef.h>
#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ embedding
 *
 * E: vocab x cols, Y: tokens x cols; types GEMM_F16, GEMM_BF16 or GEMM_F32,
 * in any combination.  Pointers need the alignment of their elements only.
 * tokens at most 2^25, vocab at most 2^20, cols at most 2^23
 * (GEMM_ERR_UNSUPPORTED above). */

/* Enqueue Y[t] = cast(scale * E[ids[t]]) (fp32 product, rounded once), zeros
 * for a token whose id names no row. */
gemm_status_t gemm_embed(int64_t tokens, int64_t vocab, int64_t cols, int32_t e_type,
                         int32_t y_type, int32_t id_bytes, const void *ids, const void *E,
                         int64_t lde, void *Y, int64_t ldy, float scale, gemm_stream_t stream);

/* Bytes of workspace that gemm_embed_backward needs for these sizes (may be
 * 0; the pointer may then be NULL). */
gemm_status_t gemm_embed_workspace(int64_t tokens, int64_t vocab, int64_t cols, size_t *bytes);

/* Enqueue the gradient of gemm_embed from dY (tokens x cols, y_type):
 *     dE[v] = cast(scale * sum over t with ids[t] = v of dY[t])
 * for every row of the table (zeros where no token names it), or with
 * accumulate = 1 dE[v] = cast(dE[v] + that sum) for the rows that are named;
 * the others are then neither read nor written.  Sums are in fp32 in an
 * order that depends on the sizes and the ids alone, so equal calls give equal
 * bits. */
gemm_status_t gemm_embed_backward(int64_t tokens, int64_t vocab, int64_t cols, int32_t y_type,
                                  int32_t e_type, int32_t id_bytes, const void *ids,
                                  const void *dY, int64_t lddy, void *dE, int64_t ldde,
                                  int32_t accumulate, void *workspace, float scale,
                                  gemm_stream_t stream);

/* ------------------------------------------------------------ linear cross entropy
 *
 * With X (tokens x hidden) and W (vocab x hidden), both of x_type, the logits
 * are z[t,v] = scale * sum_h X[t,h] W[v,h], summed in fp32.  They are made in
 * tiles of the vocabulary and never kept:
 *     lse[t]  = log sum_v exp(z[t,v])
 *     loss[t] = lse[t] - z[t, targets[t]]
 * both fp32; a logit of +inf makes lse +inf, one of -inf adds nothing, a NaN makes
 * both NaN.  A token whose target is not in 0 .. vocab-1 gets loss = lse = 0;
 * neither its row of X nor its elements of the vectors below enter anything.
 * The gradient takes lse as the forward pass wrote it, dloss[t] and dlse[t]
 * (fp32; dlse may be NULL for zeros), and makes the logits again, piece by
 * piece of the vocabulary:
 *     p[t,v] = exp(z[t,v] - lse[t])
 *     G[t,v] = scale * ((dloss[t] + dlse[t]) p[t,v] - (v = targets[t] ? dloss[t] : 0))
 *     dX[t]  = sum_v G[t,v] W[v]       (zeros for tokens without a target)
 *     dW[v]  = sum_t G[t,v] X[t]       (accumulate = 1: added to dW)
 * G enters both products as a value of x_type relative to the largest |dloss|
 * and |dloss + dlse| of the call (fp16 with 14 more binades above the
 * smallest), so that gradients far below that type's range keep their bits;
 * the products are summed in fp32 and rounded once.  That rounding of G is what
 * fp32 outputs are off by (1.1e-3 of the result's norm for bf16, 1.5e-4 for fp16).
 * In fp16 a token whose coefficients lie more than 2^18 below the call's largest
 * loses bits (2^24 below, its row of dX is off by 2.5e-3); in bf16 none does.
 * An infinity or NaN among a token's values reaches its row of dX and dW.
 *
 * x_type GEMM_F16 or GEMM_BF16; dx_type and dw_type GEMM_F32, GEMM_F16 or
 * GEMM_BF16.  1 <= hidden <= 2^15, 1 <= vocab <= 2^24, tokens <= 2^20,
 * and at most 2^36 logits.
 * Where hidden or ldw is no multiple of 8, or W is not 16-byte aligned
 * (`unaligned` = 1 makes room for that; GEMM_ERR_MISALIGNED without it), W is
 * copied to the workspace piece by piece; the forward pass of up to 16 tokens
 * reads it where it lies. */
typedef struct {
    int64_t tokens, vocab, hidden;
    int32_t x_type, dx_type, dw_type; /* gemm_dtype_t */
    int32_t id_bytes;                 /* of the targets: 4 or 8 */
    int32_t accumulate;               /* 1: dW is added to */
    int32_t unaligned;                /* 1: W may lie off 16 bytes */
    int64_t ldx, ldw, lddx, lddw;     /* 0 = packed */
    int64_t piece;                    /* columns of the vocabulary whose G the workspace
                                         holds at a time (rounded up to 256); 0 = chosen */
    float scale;                      /* 1.0f = none */
} gemm_xent_desc_t;

typedef struct gemm_xent_plan gemm_xent_plan_t;

/* Validate a descriptor on the host (no device is touched). */
gemm_status_t gemm_xent_validate_desc(const gemm_xent_desc_t *desc);

/* Validate, check the device, choose the kernels; the plan (host memory) is
 * immutable, may be shared by threads, and is released with
 * gemm_xent_plan_destroy. */
gemm_status_t gemm_xent_plan(const gemm_xent_desc_t *desc, gemm_xent_plan_t **out);
gemm_status_t gemm_xent_plan_destroy(gemm_xent_plan_t *plan);
gemm_status_t gemm_xent_plan_describe(const gemm_xent_plan_t *plan, char *buf, size_t len);

/* Bytes of workspace (16-byte aligned) of the two calls; either pointer may
 * be NULL. */
gemm_status_t gemm_xent_workspace(const gemm_xent_plan_t *plan, size_t *forward, size_t *backward);

/* Enqueue loss and lse (tokens values each; loss may be NULL). */
gemm_status_t gemm_xent_forward(const gemm_xent_plan_t *plan, const void *X, const void *W,
                                const void *targets, float *loss, float *lse, void *workspace,
                                gemm_stream_t stream);

/* Enqueue dX and dW; either may be NULL (not wanted). */
gemm_status_t gemm_xent_backward(const gemm_xent_plan_t *plan, const void *X, const void *W,
                                 const void *targets, const float *lse, const float *dloss,
                                 const float *dlse, void *dX, void *dW, void *workspace,
                                 gemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif

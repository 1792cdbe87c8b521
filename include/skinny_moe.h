/*
 * skinny_moe.h -- C ABI of the routed half of a mixture-of-experts layer, in the same
 * library (libskinny_gemm_bf16.so): the choice of each token's experts from the router's
 * logits (skinny_gemm_bf16_f32out or skinny_linear_* make them), and the experts'
 * projections with their weighted sum for a few tokens.
 *
 * Conventions as in skinny_ops.h: device pointers, row-major matrices, row strides in
 * elements, arguments checked before anything is enqueued, nothing written on error nor
 * outside the named rows and columns, no allocation, no synchronisation, no state kept
 * between calls, legal under HIP graph capture, gfx950 only. M is any value from 0 up;
 * M == 0 is a no-op that returns SKINNY_OK. The same call gives the same bits.
 */
#ifndef SKINNY_MOE_H
#define SKINNY_MOE_H

#include <stddef.h>
#include <stdint.h>

#include "skinny_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Router ---------------------------------------------------------------------
 *   s[m, e] = softmax over e of logits[m, :], or sigmoid(logits[m, e])
 *   rank[m, e] = logits[m, e], or s[m, e] + bias[e] where there is a bias
 *   ids[m, :] = the k experts of the largest rank, largest first; equal ones by index
 *   weights[m, j] = scale * s[m, ids[m, j]], or with renormalize scale * s / (their sum)
 * With groups > 1 the experts are `groups` runs of E / groups, and only those of `kept`
 * groups are taken: the groups of the largest max of rank (no bias) or sum of their two
 * largest ranks (with a bias).
 * Ranks with a bias are compared in float64, so that they are in the order of the formula
 * wherever that has one. NaN ranks before everything. Weights are float32; renormalized, they are
 * the quotients of the scores however small these are, down to exp(-745), and 0 where all of them
 * are below that (logits of -infinity, or of the lowest finite value). A row of only -infinity
 * gives softmax weights 0; NaN or +infinity in a row makes softmax weights NaN.
 * One kernel. 1 <= E <= 1024, groups <= 64 divides E, 1 <= kept <= groups,
 * 1 <= k <= 64 and k <= kept * E / groups, scale finite.
 */
typedef enum skinny_score { SKINNY_SCORE_SOFTMAX = 0, SKINNY_SCORE_SIGMOID = 1 } skinny_score_t;

typedef struct skinny_route {
    const float *logits;      /* [M][E], row stride ldl >= E */
    const float *bias;        /* [E] or NULL */
    int32_t *ids;             /* [M][k] contiguous */
    float *weights;           /* [M][k] contiguous */
    int64_t ldl;
    int32_t M, E, k;
    int32_t score;            /* skinny_score_t */
    int32_t groups, kept;     /* 1, 1: no limit by groups */
    int32_t renormalize;      /* 0 or 1 */
    float scale;
} skinny_route_t;

int skinny_route(const skinny_route_t *args, hipStream_t stream);

/* ---- Experts --------------------------------------------------------------------
 *   h[m, j, :] = act(x[m] . Wg[e]^T) * (x[m] . Wu[e]^T),   e = ids[m, j]
 *   y[m, :] = sum_j weights[m, j] * (h[m, j, :] . Wd[e]^T) + residual[m, :]
 * An id outside 0 .. E - 1 names no expert: its term is left out (padding, or an expert
 * that another rank holds). A token may name an expert more than once. x, y and residual
 * are bfloat16; y may be the residual itself (same pointer and stride), no other overlap of
 * y or the workspace with another operand is accepted.
 * Weights are bfloat16, or 8-bit (e4m3 or integers) with float32 scales, each times x as it
 * is: 8-bit values are bfloat16 ones, exactly. Sums are held in float32 and y is rounded once.
 * Between the projections h is held as two bfloat16 values (16 bits) where experts are read for
 * 4 or 8 rows, and rounded to one, as skinny_linear_bf16 stores it, where for more: so a token's
 * outputs are as exact as y's type (0.0017 of their norm) among few tokens, and off by 0.0024 in a
 * batch that gives an expert more than 4.5 to 7 rows. Element-wise kernels hold h in float32.
 * Two kernels for every 128 rows, with h and the order of the pairs (m, j) by expert in the
 * workspace; each expert that a row names is read once for every 4 to 32 of its rows, most of them
 * from the caches after the first time. How many goes by the rows that an expert has on average, were
 * all M k ids spread over the E experts: those that name none count too. For up to some hundred
 * rows; a prompt of thousands reads every expert again for each 128 of them.
 * Fast path: x, ldx, weights and their strides multiples of 16 bytes, H and I multiples of 8
 * (bfloat16) or 16. Others run an element-wise kernel, which is right and slow.
 * 1 <= E <= 1024, 1 <= k <= 32; H, I >= 1.
 */
typedef enum skinny_weights {
    SKINNY_WEIGHTS_BF16 = 0,
    SKINNY_WEIGHTS_E4M3_ROW = 1,   /* scales [E][I], [E][H] */
    SKINNY_WEIGHTS_E4M3_BLOCK = 2, /* scales [E][ceil(I/128)][ceil(H/128)], [E][ceil(H/128)][ceil(I/128)] */
    SKINNY_WEIGHTS_INT8_ROW = 3    /* scales [E][I], [E][H] */
} skinny_weights_t;

typedef struct skinny_experts {
    const void *x;            /* [M][H] bfloat16, row stride ldx >= H */
    const int32_t *ids;       /* [M][k] contiguous */
    const float *weights;     /* [M][k] contiguous */
    const void *w_gate, *w_up; /* [E][I][H], expert e at e * up_stride elements, >= I * H */
    const void *w_down;       /* [E][H][I], expert e at e * down_stride elements, >= H * I */
    const float *gate_scale, *up_scale; /* expert e at e * up_scale_stride; NULL for bfloat16 */
    const float *down_scale;  /* expert e at e * down_scale_stride */
    const void *residual;     /* [M][H] bfloat16, row stride ldr >= H, or NULL */
    void *y;                  /* [M][H] bfloat16, row stride ldy >= H */
    void *workspace;          /* 16-byte aligned, skinny_experts_workspace_bytes() of it */
    size_t workspace_bytes;
    int64_t ldx, ldr, ldy;
    int64_t up_stride, down_stride, up_scale_stride, down_scale_stride;
    int32_t M, E, k, H, I;
    int32_t act;              /* skinny_act_t */
    int32_t type;             /* skinny_weights_t */
} skinny_experts_t;

/* Bytes of workspace that a call of these sizes needs (0: no call with them is accepted, or
 * M is 0). Its contents need no preparation and mean nothing after the call; calls that may
 * run at the same time need one each. */
size_t skinny_experts_workspace_bytes(int32_t M, int32_t k, int32_t E, int32_t I);

int skinny_experts(const skinny_experts_t *args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SKINNY_MOE_H */

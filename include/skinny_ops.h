/*
 * skinny_ops.h -- C ABI of the operators around the skinny GEMM, in the same library
 * (libskinny_gemm_bf16.so): the norm in front of a projection, and projections whose
 * bias, activation, gate and residual are applied before the result is stored, on
 * bfloat16, or on 8-bit floats or integers with scales.
 *
 * Conventions shared by every entry point below:
 *  - Pointers are DEVICE pointers. bfloat16 and e4m3 values (the OCP 8-bit float
 *    with 4 exponent and 3 fraction bits, largest value 448, no infinities) are
 *    raw bit patterns. Matrices are row-major; ld* is a row stride in elements.
 *  - M, the number of rows of x, is any value from 0 up: one decode token or a
 *    whole prompt. M == 0, N == 0 or D == 0 is a no-op that returns SKINNY_OK.
 *  - The caller owns every buffer. A call enqueues exactly one kernel on `stream`
 *    of the current device and returns: no allocation, no synchronisation, no
 *    workspace, no state kept between calls. Calls are legal under HIP graph
 *    capture, and calls on different streams may overlap.
 *  - Arguments are checked before anything is enqueued. Nothing is written on
 *    error, and nothing outside the named rows and columns ever is: the columns
 *    between the width and the row stride stay as they were.
 *  - Sums, norms and activations are held in float32, with one exception: the products
 *    of e4m3 x and W for more than 16 rows and bfloat16 outputs (see skinny_linear_fp8).
 *    Activations use the hardware's exponential and reciprocal: gelu is within
 *    (32 + 3 z^2) 2^-24 of its value, silu and gelu_tanh within 32 * 2^-24 of |z|. Each
 *    output value is rounded once. Results depend on the inputs and sizes alone: the same call gives the same
 *    bits, and no atomic is used. Calls of other sizes may take another kernel, whose sums
 *    have another order: a row of x need not give the same bits in a larger batch.
 *  - Only gfx950 devices are supported (others: SKINNY_ERR_UNSUPPORTED).
 */
#ifndef SKINNY_OPS_H
#define SKINNY_OPS_H

#include <stdint.h>

#include "skinny_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Root-mean-square norm -----------------------------------------------------
 *   h[m, d] = x[m, d] + residual[m, d]            (h = x without a residual)
 *   y[m, d] = h[m, d] * weight[d] / sqrt(mean_d(h[m, d]^2) + eps)
 * x, residual, weight: bfloat16. With a residual, h is also stored, rounded once to
 * bfloat16, in residual_out; the norm is taken of the unrounded h. Squares are summed
 * in float32, so they must stay finite (|h| below about 1e19 / sqrt(D)), as must
 * h * weight.
 * residual and residual_out are both given or both NULL. residual_out may be residual
 * or x itself (same pointer and stride), as may y be x in the bfloat16 form when
 * residual_out is not x; no other overlap of an output with an input or another
 * output is accepted. eps >= 0. Everything 2-byte aligned; any D and strides.
 * Rows of up to 32768 columns stay in registers; wider ones are read twice.
 */
typedef struct skinny_norm {
    const void *x;            /* [M][D] bfloat16, row stride ldx >= D */
    const void *residual;     /* [M][D] bfloat16, row stride ldr, or NULL */
    const void *weight;       /* [D] bfloat16 */
    void *residual_out;       /* [M][D] bfloat16, row stride ldro, or NULL */
    void *y;                  /* [M][D] bfloat16, or e4m3 for skinny_rms_norm_fp8, or int8; stride ldy */
    float *scale;             /* 8-bit outputs only: [M] or [M][ceil(D / group)] */
    int64_t ldx, ldr, ldro, ldy;
    int32_t M, D;
    int32_t group;            /* skinny_rms_norm_fp8: 0 = one scale per row, 128 = one per
                                 128 columns; the others: 0 */
    float eps;
} skinny_norm_t;

/* y as bfloat16. */
int skinny_rms_norm_bf16(const skinny_norm_t *args, hipStream_t stream);

/* y as e4m3 with float32 scales: scale = max(largest |y| of the row or group, 2^-100)
 * / 448 and q = e4m3(y / scale), nearest-even, so that q * scale stands for y. y is not
 * rounded to fewer bits before that; the quotient is y times the float32 reciprocal. Rows
 * and groups of zeros give zeros (with eps == 0 a row of zeros is 0 / 0: NaN). A NaN in a row makes the row's scales and values NaN. An infinity makes
 * the scale of its row or group NaN with all its values, and the row's other groups 0. */
int skinny_rms_norm_fp8(const skinny_norm_t *args, hipStream_t stream);

/* y as 8-bit integers with a float32 scale per row (group 0): scale = max(largest |y|, 2^-100)
 * / 127 and q = y / scale rounded to the nearest integer, ties to even, so -127 .. 127. The
 * quotient is that of a float32 division here, not the product with a reciprocal, so values half
 * way between two integers, up to the rounding of the scale, go where the division puts them
 * (for all rows of skinny_quantize_int8; here y may lie within 2^-22 of a step's last bit of a tie
 * of the division itself). Rows of zeros give zeros; a NaN or an infinity in a row makes its
 * scale NaN and its q 0, so that q * scale is NaN. */
int skinny_rms_norm_int8(const skinny_norm_t *args, hipStream_t stream);

/* The rows of x themselves as 8-bit integers: y = x in the formulas of skinny_rms_norm_int8.
 * weight, residual and residual_out are NULL, eps and group 0. An infinity makes the scale
 * of its row infinite and its q 0. */
int skinny_quantize_int8(const skinny_norm_t *args, hipStream_t stream);

/* ---- Projections with an epilogue ----------------------------------------------
 *   z[m, n] = sum_k x[m, k] * W0[n, k] + bias0[n]
 *   y[m, n] = act(z[m, n]) + residual[m, n]
 * and, with W1 given (the gated form; the residual is then NULL),
 *   y[m, n] = act(z[m, n]) * (sum_k x[m, k] * W1[n, k] + bias1[n]).
 * A merged gate/up weight [2N][K] is W0 = base, W1 = base + N * K elements.
 * W0, W1: contiguous [N][K]. Biases and the residual are bfloat16, each optional.
 * y may be the residual itself (bfloat16 output, same pointer and stride); no other
 * overlap of y with an input is accepted. K == 0 gives act(bias) + residual.
 * Fast path: x and W 16-byte aligned, row strides and K multiples of 16 bytes, both at
 * most 4194304 elements; anything else runs an element-wise kernel, which is right and
 * slow (bfloat16 1 x 4096 x 4100 151 us, 64 rows 205, 4096 rows 8.8 ms): pad K with zeros.
 */
typedef enum skinny_act {
    SKINNY_ACT_NONE = 0,
    SKINNY_ACT_RELU = 1,
    SKINNY_ACT_GELU = 2,      /* z * Phi(z), with the error function */
    SKINNY_ACT_GELU_TANH = 3, /* its tanh form: 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
    SKINNY_ACT_SILU = 4       /* z / (1 + exp(-z)) */
} skinny_act_t;

typedef enum skinny_scales {
    SKINNY_SCALES_ROW = 1,    /* x_scale [M], w_scale [N]: one per row of x and of W */
    SKINNY_SCALES_BLOCK = 2   /* x_scale [M][ceil(K/128)], w_scale [ceil(N/128)][ceil(K/128)] */
} skinny_scales_t;

typedef struct skinny_linear {
    const void *x;            /* [M][K], row stride ldx >= K */
    const void *W0, *W1;      /* [N][K] contiguous; W1 NULL: not gated */
    const float *x_scale;     /* 8-bit x and W only, contiguous float32 (see skinny_scales) */
    const float *w0_scale, *w1_scale;
    const void *bias0, *bias1; /* [N] bfloat16 or NULL; bias1 only with W1 */
    const void *residual;     /* [M][N] bfloat16, row stride ldr >= N, or NULL */
    void *y;                  /* [M][N] bfloat16, or float32 with out_f32; row stride ldy >= N */
    int64_t ldx, ldr, ldy;
    int32_t M, N, K;
    int32_t act;              /* skinny_act_t */
    int32_t out_f32;          /* 0 or 1 */
    int32_t scales;           /* skinny_linear_fp8, _int8: skinny_scales_t; skinny_linear_bf16: 0 */
} skinny_linear_t;

/* x and W bfloat16. */
int skinny_linear_bf16(const skinny_linear_t *args, hipStream_t stream);

/* x and W e4m3 with float32 scales: every product is multiplied by its x and W scale
 * (per row: after the sum; per block: each 128-column part of the sum before it is
 * added). The output of skinny_rms_norm_fp8 with group 0 or 128 is x with ROW or BLOCK
 * scales. Up to 16 rows, and for float32 outputs, the products are exact and summed in
 * float32. Otherwise the 8-bit matrix instruction takes them, which cuts those of each eight
 * columns off (towards zero) at 2^-13 of the largest before it adds them: about 2e-5 of a
 * result's norm, below bfloat16's rounding of 4e-3. */
int skinny_linear_fp8(const skinny_linear_t *args, hipStream_t stream);

/* x and W 8-bit integers (two's complement) with one float32 scale per row of x and per row of
 * W (scales: SKINNY_SCALES_ROW): what skinny_rms_norm_int8 and skinny_quantize_int8 make, and
 * weights with a scale for each output. The products are added up in 32-bit integers, which is
 * exact whatever kernel a call takes, so K is at most 131071; the sum is rounded to float32
 * once and multiplied by the scales. */
int skinny_linear_int8(const skinny_linear_t *args, hipStream_t stream);

/* The kernel that a projection call takes. Calls with the same element type, scales, gate,
 * output type and class of rows (up to 8, up to 16, more) choose among the same `count`
 * kernels, numbered by `index`. */
typedef enum skinny_linear_kind {
    SKINNY_LINEAR_ELEMENTS = 0, /* one output per thread: what is not 16-byte aligned */
    SKINNY_LINEAR_STREAM = 1,   /* K split over the waves of a block */
    SKINNY_LINEAR_TILE = 2      /* LDS tiles shared by the waves of a block */
} skinny_linear_kind_t;

typedef struct skinny_linear_plan {
    int32_t kind;               /* skinny_linear_kind_t */
    int32_t features, rows;     /* outputs of a block */
    int32_t waves;              /* of a block */
    int32_t ring;               /* stages of K that a wave holds (SKINNY_LINEAR_STREAM) */
    int32_t index, count;       /* -1 and 0 for SKINNY_LINEAR_ELEMENTS */
} skinny_linear_plan_t;

/* The plan of skinny_linear_bf16(args) (scales 0) or skinny_linear_fp8(args) (else) on a
 * device with that many compute units (256: a whole MI355X). Checks args as the call does,
 * touches no device and follows no pointer. SKINNY_ERR_INVALID_ARG for a call without
 * outputs. */
int skinny_linear_default_plan(const skinny_linear_t *args, int32_t compute_units, skinny_linear_plan_t *out);

/* The same of skinny_linear_int8(args). */
int skinny_linear_int8_default_plan(const skinny_linear_t *args, int32_t compute_units, skinny_linear_plan_t *out);

#ifdef __cplusplus
}
#endif

#endif /* SKINNY_OPS_H */

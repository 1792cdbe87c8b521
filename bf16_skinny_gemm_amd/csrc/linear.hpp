// Device code shared by the kernels of skinny_linear_bf16 / _fp8 (include/skinny_ops.h):
// arguments, the epilogue, and the matrix instructions on bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"
#include "skinny_ops.h"

namespace skg {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct LinArgs {
    const uint8_t *x, *w[2];
    const float *xs, *ws[2];   // scales of 8-bit x and W
    const uint16_t *bias[2];   // or null
    const uint16_t *res;       // or null
    void *y;
    int64_t ldx;               // bytes
    int64_t ldr, ldy;          // elements
    int M, N, K;               // K in elements
    int kb;                    // 128-column blocks of K (block scales)
    int act, out_f32;
};

__device__ __forceinline__ float activate(float z, int act)
{
    switch (act) {  // uniform: a scalar branch
    case SKINNY_ACT_RELU:
        return z < 0.0f ? 0.0f : z;  // NaN stays
    case SKINNY_ACT_SILU:
        return z / (1.0f + __expf(-z));
    case SKINNY_ACT_GELU:
        return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case SKINNY_ACT_GELU_TANH: {
        // 0.5 (1 + tanh u) = 1 / (1 + exp(-2u)): no cancellation for negative z
        const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
        return z / (1.0f + __expf(-u2));
    }
    default:
        return z;
    }
}

// One output from its sums: z of W0 (scaled), u of W1.
template <bool GATED>
__device__ __forceinline__ float finish(const LinArgs &a, float z, float u, int m, int n)
{
    if (a.bias[0])
        z += bf16_to_f32(a.bias[0][n]);
    z = activate(z, a.act);
    if constexpr (GATED) {
        if (a.bias[1])
            u += bf16_to_f32(a.bias[1][n]);
        z *= u;
    } else {
        if (a.res)
            z += bf16_to_f32(a.res[(int64_t)m * a.ldr + n]);
    }
    return z;
}

__device__ __forceinline__ void put(const LinArgs &a, float v, int m, int n)
{
    if (a.out_f32)
        static_cast<float *>(a.y)[(int64_t)m * a.ldy + n] = v;
    else
        static_cast<uint16_t *>(a.y)[(int64_t)m * a.ldy + n] = f32_to_bf16(v);
}

// D[i][j] += sum_k A[i][k] B[j][k] for 16 x 16 outputs. A lane holds, of its row
// (lane % 16) of A and of B, the LB * 16 bytes that the same lane of the other operand
// multiplies: which columns of K those are is the caller's choice, the same for A and B.
// D of a lane: column lane % 16, rows lane / 16 * 4 + 0..3.
__device__ __forceinline__ f32x4 mfma_bf16(const u32x4 &a, const u32x4 &b, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   c, 0, 0, 0);
}

__device__ __forceinline__ f32x4 mfma_fp8(const u32x4 &a0, const u32x4 &a1, const u32x4 &b0, const u32x4 &b1,
                                          const f32x4 &c)
{
    const i32x8 a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
    const i32x8 b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
    // formats 0 = e4m3 for both; scale operands 0 select the form without scales
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Sixteen e4m3 values as bfloat16, which holds each of them (v_cvt_scalef32_pk_bf16_fp8).
__device__ __forceinline__ void widen(const u32x4 &v, u32x4 &lo, u32x4 &hi)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        lo[2 * i] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, false));
        lo[2 * i + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, true));
        hi[2 * i] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 + i], 1.0f, false));
        hi[2 * i + 1] =
            __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 + i], 1.0f, true));
    }
}

// The product of 32 bytes per lane, EXACT or with the 8-bit matrix instruction. That one
// adds its products in groups of eight, each cut off (towards zero) at 2^-13 of the
// group's largest: measured 1.7e-5 of the result's norm on normal values, a hundredth of
// a bfloat16 output's rounding but a hundred times a float32 sum's. EXACT widens both
// operands to bfloat16 and takes the bfloat16 instruction, whose products are exact and
// whose sums round in float32, at half its rate and 16 conversions per operand and lane:
// taken for float32 outputs, and where the kernel waits for memory anyway.
template <bool EXACT>
__device__ __forceinline__ f32x4 mfma_bytes(const u32x4 (&a)[2], const u32x4 (&b)[2], f32x4 c)
{
    if constexpr (!EXACT) {
        return mfma_fp8(a[0], a[1], b[0], b[1], c);
    } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            u32x4 al, ah, bl, bh;
            widen(a[q], al, ah);
            widen(b[q], bl, bh);
            c = mfma_bf16(al, bl, c);
            c = mfma_bf16(ah, bh, c);
        }
        return c;
    }
}

}  // namespace skg

namespace skg_host {

// Kernels of one element type and scale mode, by form. mode: 0 bfloat16, 1 row, 2 block.
struct SmallKernel {
    const void *fn;
    int rows;       // rows of W per block
    int unit_bytes; // bytes of a row of W that one wave takes per step
    int depth;      // steps in flight
};
SmallKernel small_kernel_bf16(int M, bool gated, int nr, bool exact);
SmallKernel small_kernel_row(int M, bool gated, int nr, bool exact);
SmallKernel small_kernel_block(int M, bool gated, int nr, bool exact);

}  // namespace skg_host

// Small device functions shared by the kernels of include/skinny_ops.h.
#pragma once

#include "kernels.hpp"

namespace skg {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// The two bfloat16 values of a packed pair.
__device__ __forceinline__ float lo_f32(unsigned p) { return __builtin_bit_cast(float, p << 16); }
__device__ __forceinline__ float hi_f32(unsigned p) { return __builtin_bit_cast(float, p & 0xFFFF0000u); }

// Two floats to packed bfloat16, nearest-even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ unsigned pack_bf16(float a, float b)
{
    const f32x2 v = {a, b};
    return __builtin_bit_cast(unsigned, __builtin_convertvector(v, bf16x2_t));
}

// Vectors in memory at any alignment: global memory takes unaligned 16-byte accesses, so
// rows of odd width or stride move in the same instructions as aligned ones.
typedef u32x4 __attribute__((aligned(1))) u32x4_any;
typedef u32x2 __attribute__((aligned(1))) u32x2_any;

}  // namespace skg

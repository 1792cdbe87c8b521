// Device code shared by the kernels of skinny_linear_bf16 / _fp8 (include/skinny_ops.h):
// arguments, the epilogue, and the matrix instructions on bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ops_device.hpp"
#include "skinny_ops.h"

namespace skg {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
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

template <int ACT>
__device__ __forceinline__ float activate_as(float z)
{
    if constexpr (ACT == SKINNY_ACT_RELU) {
        return z < 0.0f ? 0.0f : z;  // NaN stays
    } else if constexpr (ACT == SKINNY_ACT_SILU) {
        return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    } else if constexpr (ACT == SKINNY_ACT_GELU) {
        // Phi(-|z|) = Q(t) t exp(-z^2 / 2) with t = 1 / (1 + 0.4 |z| / sqrt 2): the form of
        // Abramowitz and Stegun 7.1.26 with Q fitted here to the least relative error,
        // 1.3e-7 for all z, so that small values in the negative tail are right too. With
        // the roundings, that of z^2 / 2 in the exponent above all, within (32 + 3 z^2)
        // 2^-24 of the value. A call of erff took 0.4 us more at the end of a decode-size
        // launch.
        const float x = __builtin_fabsf(z) * 0.70710678118654752f;
        const float t = __builtin_amdgcn_rcpf(1.0f + 0.4f * x);
        float q = 0.0251271538f;
        q = -0.0914369673f + t * q;
        q = 0.0845232531f + t * q;
        q = -0.00278964383f + t * q;
        q = 0.07071013f + t * q;
        q = 0.0842721611f + t * q;
        q = 0.103921227f + t * q;
        q = 0.112834804f + t * q;
        q = 0.112837933f + t * q;
        const float tail = q * t * __expf(-x * x);
        return z * (z < 0.0f ? tail : 1.0f - tail);  // z - z * tail would be NaN at infinity
    } else if constexpr (ACT == SKINNY_ACT_GELU_TANH) {
        // 0.5 (1 + tanh u) = 1 / (1 + exp(-2u)): no cancellation for negative z
        const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
        return z * __builtin_amdgcn_rcpf(1.0f + __expf(-u2));
    } else {
        return z;
    }
}

// One scalar branch for all of a lane's values.
template <int COUNT>
__device__ __forceinline__ void activate(float (&z)[COUNT], int act)
{
    auto all = [&](auto ac) {
#pragma unroll
        for (int e = 0; e < COUNT; ++e)
            z[e] = activate_as<decltype(ac)::value>(z[e]);
    };
    switch (act) {
    case SKINNY_ACT_RELU:
        return all(std::integral_constant<int, SKINNY_ACT_RELU>{});
    case SKINNY_ACT_SILU:
        return all(std::integral_constant<int, SKINNY_ACT_SILU>{});
    case SKINNY_ACT_GELU:
        return all(std::integral_constant<int, SKINNY_ACT_GELU>{});
    case SKINNY_ACT_GELU_TANH:
        return all(std::integral_constant<int, SKINNY_ACT_GELU_TANH>{});
    default:
        return;
    }
}

__device__ __forceinline__ f32x4 activate4(f32x4 v, int act)
{
    float z[4] = {v[0], v[1], v[2], v[3]};
    activate(z, act);
    return f32x4{z[0], z[1], z[2], z[3]};
}

// One output from its sums: z of W0 (scaled), u of W1.
template <bool GATED>
__device__ __forceinline__ float finish(const LinArgs &a, float z, float u, int m, int n)
{
    if (a.bias[0])
        z += bf16_to_f32(a.bias[0][n]);
    float act[1] = {z};
    activate(act, a.act);
    z = act[0];
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

__device__ __forceinline__ f32x4 widen4(u32x2 v) { return f32x4{lo_f32(v[0]), hi_f32(v[0]), lo_f32(v[1]), hi_f32(v[1])}; }

// The residual of four consecutive outputs n .. n + 3 of row m, where finish4 wants it.
__device__ __forceinline__ u32x2 residual4(const LinArgs &a, int m, int n)
{
    return a.res && n + 4 <= a.N ? *reinterpret_cast<const u32x2_any *>(a.res + (int64_t)m * a.ldr + n)
                                 : u32x2{0, 0};
}

// Four consecutive outputs n .. n + 3 of row m, of which any may lie beyond N. The sums have
// yet to be multiplied by their scales (MODE 1), xs that of the row.
template <int MODE, bool GATED>
__device__ __forceinline__ void finish4(const LinArgs &a, f32x4 z, f32x4 u, u32x2 r, float xs, int m, int n)
{
    if (n + 4 > a.N) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (n + e >= a.N)
                continue;
            float z1 = z[e], u1 = u[e];
            if constexpr (MODE == 1) {
                z1 *= xs * a.ws[0][n + e];
                if constexpr (GATED)
                    u1 *= xs * a.ws[1][n + e];
            }
            put(a, finish<GATED>(a, z1, u1, m, n + e), m, n + e);
        }
        return;
    }
    if constexpr (MODE == 1) {
        const f32x4 s0 = *reinterpret_cast<const f32x4_any *>(a.ws[0] + n);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            z[e] *= xs * s0[e];
        if constexpr (GATED) {
            const f32x4 s1 = *reinterpret_cast<const f32x4_any *>(a.ws[1] + n);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                u[e] *= xs * s1[e];
        }
    }
    if (a.bias[0])
        z += widen4(*reinterpret_cast<const u32x2_any *>(a.bias[0] + n));
    z = activate4(z, a.act);
    if constexpr (GATED) {
        if (a.bias[1])
            u += widen4(*reinterpret_cast<const u32x2_any *>(a.bias[1] + n));
        z *= u;
    } else if (a.res) {
        z += widen4(r);
    }
    const int64_t at = (int64_t)m * a.ldy + n;
    if (a.out_f32)
        *reinterpret_cast<f32x4_any *>(static_cast<float *>(a.y) + at) = z;
    else
        *reinterpret_cast<u32x2_any *>(static_cast<uint16_t *>(a.y) + at) =
            u32x2{pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3])};
}

// The columns' part of the epilogue of the outputs n .. n + 7 <= N - 1, for many rows. A
// load between a tile's stores would be waited for with all stores before it (loads and
// stores share a counter): 4096 x 4096 outputs of K = 128 took 25 us that way, 15.8 so,
// and 14.2 with stores that bypass the second-level cache, which they only pass through.
template <int MODE, bool GATED>
struct Columns8 {
    f32x4 s[1 + GATED][2];
    u32x2 b[1 + GATED][2];

    __device__ __forceinline__ void load(const LinArgs &a, int n, bool wide)
    {
#pragma unroll
        for (int q = 0; q < 1 + GATED; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (MODE == 1)
                    s[q][h] = wide ? *reinterpret_cast<const f32x4_any *>(a.ws[q] + n + 4 * h) : f32x4{0, 0, 0, 0};
                b[q][h] = wide && a.bias[q] ? *reinterpret_cast<const u32x2_any *>(a.bias[q] + n + 4 * h) : u32x2{0, 0};
            }
    }
    // the loads have arrived
    __device__ __forceinline__ void settle()
    {
#pragma unroll
        for (int q = 0; q < 1 + GATED; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (MODE == 1)
                    asm volatile("" : "+v"(s[q][h]));
                asm volatile("" : "+v"(b[q][h]));
            }
    }
    __device__ __forceinline__ void finish(const LinArgs &a, f32x4 (&z)[2], f32x4 (&u)[2], u32x4 r, int m, int n) const
    {
        float v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (MODE == 1)
                z[h] *= s[0][h];
            z[h] += widen4(b[0][h]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[h * 4 + e] = z[h][e];
        }
        activate(v, a.act);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            z[h] = f32x4{v[h * 4], v[h * 4 + 1], v[h * 4 + 2], v[h * 4 + 3]};
            if constexpr (GATED) {
                if constexpr (MODE == 1)
                    u[h] *= s[GATED][h];
                z[h] *= u[h] + widen4(b[GATED][h]);
            } else {
                z[h] += widen4(u32x2{r[2 * h], r[2 * h + 1]});
            }
        }
        const int64_t at = (int64_t)m * a.ldy + n;
        if (a.out_f32) {
            f32x4_any *y = reinterpret_cast<f32x4_any *>(static_cast<float *>(a.y) + at);
            __builtin_nontemporal_store(z[0], y);
            __builtin_nontemporal_store(z[1], y + 1);
        } else {
            const u32x4 y = {pack_bf16(z[0][0], z[0][1]), pack_bf16(z[0][2], z[0][3]), pack_bf16(z[1][0], z[1][1]),
                             pack_bf16(z[1][2], z[1][3])};
            __builtin_nontemporal_store(y, reinterpret_cast<u32x4_any *>(static_cast<uint16_t *>(a.y) + at));
        }
    }
};

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

// A kernel of linear_stream.hpp: outputs per block along N and M, stages per wave, waves,
// bytes of a stage and of LDS, matrix instructions per stage.
struct StreamKernel {
    const void *fn;
    int nb, bm, ring, waves, stage, lds, tiles;
};
constexpr int kStreamMost = 10;  // kernels of one set

// A kernel of linear_tile.hpp: outputs per block along N and M, waves, and a stage's time
// (microseconds, blocks of one compute unit one after another).
struct TileKernel {
    const void *fn;
    int nb, bm, waves;
    float stage_us;
};
constexpr int kTileMost = 4;

// The kernels that take M rows, by element type and scales; returns their number.
int stream_kernels_bf16(int M, bool gated, bool exact, StreamKernel *out);
int stream_kernels_row(int M, bool gated, bool exact, StreamKernel *out);
int stream_kernels_block(int M, bool gated, bool exact, StreamKernel *out);
int tile_kernels_bf16(bool gated, bool exact, TileKernel *out);
int tile_kernels_row(bool gated, bool exact, TileKernel *out);
int tile_kernels_block(bool gated, bool exact, TileKernel *out);

}  // namespace skg_host

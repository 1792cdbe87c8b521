// The projection kernel for few rows of x (M <= 128): W streams from HBM straight into
// the operand registers of the matrix instructions, x comes from L2.
//
// A 16 x 16 matrix instruction has 16 rows for W and 16 columns for x. With M <= 4 or
// M <= 8 most columns would be empty and a load instruction would touch 16 rows of W, 64
// bytes each. Instead the instruction is folded: its 16 rows are P rows of W times
// H = 16 / P parts of K, its 16 columns P rows of x times the same H parts,
//   A[(h, n)] = W[n][part h],  B[(h', m)] = x[m][part h'],
// so that D[(h, n)][(h', m)] with h = h' is part h of the dot product of n and m (the
// rest is not used). One load instruction then covers P rows with 1024 / P contiguous
// bytes each, and no lane loads padding. The parts are added with the partial sums of
// the block's waves, which split K between them.
#pragma once

#include "linear.hpp"

namespace skg {

// MODE: 0 bfloat16, 1 e4m3 with row scales, 2 e4m3 with block scales; EXACT: see mfma_bytes.
template <int MODE, bool EXACT, int P, int MF, int NR, bool GATED, int DEPTH>
__global__ __launch_bounds__(512) void linear_small_kernel(LinArgs a)
{
    constexpr bool FP8 = MODE != 0, BLOCK = MODE == 2;
    constexpr int H = 16 / P;
    constexpr int LB = FP8 ? 2 : 1;       // 16-byte loads per lane and operand row
    constexpr int UB = LB * 1024 / P;     // bytes of K per step
    constexpr int MATS = GATED ? 2 : 1;
    constexpr int ROWS = P * NR;
    static_assert(MF == 1 || P == 16, "more than 16 rows of x take whole instructions");
    static_assert(ROWS <= 128, "a block's rows share one row of block scales");

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int i16 = lane & 15, g = lane >> 4;
    const int rn = i16 % P, h = i16 / P;
    const int KB = FP8 ? a.K : a.K * 2;   // bytes of a row
    const int units = (KB + UB - 1) / UB;
    const int row0 = blockIdx.x * ROWS;
    int valid = a.N - row0;
    valid = valid > ROWS ? ROWS : valid;

    // W rows past N lie past the resource's end and read as zero
    __amdgpu_buffer_rsrc_t wr[MATS];
#pragma unroll
    for (int t = 0; t < MATS; ++t)
        wr[t] = make_rsrc(a.w[t] + (int64_t)row0 * KB, (unsigned)valid * (unsigned)KB);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (unsigned)(a.M - 1) * (unsigned)a.ldx + (unsigned)KB);
    const unsigned koff = (unsigned)(h * 64 * LB + g * 16);
    unsigned xoff[MF];
#pragma unroll
    for (int f = 0; f < MF; ++f) {
        const int m = f * P + rn;
        xoff[f] = m < a.M ? (unsigned)(m * (int)a.ldx) : kOutOfRange;
    }
    __amdgpu_buffer_rsrc_t xsr, wsr[MATS];
    if constexpr (BLOCK) {
        xsr = make_rsrc(a.xs, (unsigned)(a.M * a.kb) * 4u);
#pragma unroll
        for (int t = 0; t < MATS; ++t)
            wsr[t] = make_rsrc(a.ws[t] + (int64_t)(row0 / 128) * a.kb, (unsigned)a.kb * 4u);
    }

    struct Set {
        u32x4 w[DEPTH][MATS][NR][LB];
        u32x4 x[DEPTH][MF][LB];
        float xs[BLOCK ? DEPTH : 1][MF], ws[BLOCK ? DEPTH : 1][MATS];
    };
    auto load = [&](int u0, Set &s) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int u = u0 + d * waves;
#pragma unroll
            for (int q = 0; q < LB; ++q) {
                const unsigned k = (unsigned)(u * UB) + koff + q * 64;
                const bool in = k < (unsigned)KB;
#pragma unroll
                for (int t = 0; t < MATS; ++t)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        s.w[d][t][r][q] =
                            load16<true>(wr[t], in ? (unsigned)((r * P + rn) * KB) + k : kOutOfRange);
#pragma unroll
                for (int f = 0; f < MF; ++f)
                    s.x[d][f][q] = load16<false>(xr, in ? xoff[f] + k : kOutOfRange);
            }
            if constexpr (BLOCK) {
                const int b = u * H + h;
                const bool in = b < a.kb;
#pragma unroll
                for (int f = 0; f < MF; ++f) {
                    const int m = f * P + rn;
                    s.xs[d][f] = __builtin_bit_cast(
                        float, __builtin_amdgcn_raw_buffer_load_b32(
                                   xsr, (int)(in && m < a.M ? (unsigned)(m * a.kb + b) * 4u : kOutOfRange), 0, 0));
                }
#pragma unroll
                for (int t = 0; t < MATS; ++t)
                    s.ws[d][t] = __builtin_bit_cast(
                        float, __builtin_amdgcn_raw_buffer_load_b32(wsr[t], (int)(in ? (unsigned)b * 4u : kOutOfRange),
                                                                    0, 0));
            }
        }
        __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the products they overlap
    };
    f32x4 acc[MATS][NR][MF];
#pragma unroll
    for (int t = 0; t < MATS; ++t)
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int f = 0; f < MF; ++f)
                acc[t][r][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto use = [&](const Set &s) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
#pragma unroll
            for (int t = 0; t < MATS; ++t)
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int f = 0; f < MF; ++f) {
                        f32x4 &c = acc[t][r][f];
                        if constexpr (MODE == 0) {
                            c = mfma_bf16(s.w[d][t][r][0], s.x[d][f][0], c);
                        } else if constexpr (MODE == 1) {
                            c = mfma_bytes<EXACT>(s.w[d][t][r], s.x[d][f], c);
                        } else {
                            // part h of this step is one whole 128-column block
                            const f32x4 p =
                                mfma_bytes<EXACT>(s.w[d][t][r], s.x[d][f], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                            const float sc = s.xs[d][f] * s.ws[d][t];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                c[i] = __builtin_fmaf(p[i], sc, c[i]);
                        }
                    }
    };

    Set s0, s1;
    const int step = DEPTH * waves;
    int u = wave;
    load(u, s0);
    while (true) {
        const bool more = u + step < units;
        if (more)
            load(u + step, s1);
        use(s0);
        if (!more)
            break;
        u += step;
        const bool more2 = u + step < units;
        if (more2)
            load(u + step, s0);
        use(s1);
        if (!more2)
            break;
        u += step;
    }

    // Partial sums of the waves and of the parts meet in LDS, always in the same order.
    __shared__ float part[8][MATS][NR][16 * P];
#pragma unroll
    for (int f = 0; f < MF; ++f) {
        if (f)
            __syncthreads();
#pragma unroll
        for (int t = 0; t < MATS; ++t)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int dr = g * 4 + i;  // row of D: part dr / P, row dr % P of W
                    if (dr / P == h)
                        part[wave][t][r][(h * P + rn) * P + dr % P] = acc[t][r][f][i];
                }
        __syncthreads();
        for (int o = threadIdx.x; o < ROWS * P; o += blockDim.x) {
            const int nl = o % ROWS, ml = o / ROWS;
            const int r = nl / P, n = row0 + nl, m = f * P + ml;
            if (m >= a.M || n >= a.N)
                continue;
            float v[2] = {0.0f, 0.0f};
#pragma unroll
            for (int t = 0; t < MATS; ++t) {
                for (int k = 0; k < waves; ++k)
#pragma unroll
                    for (int q = 0; q < H; ++q)
                        v[t] += part[k][t][r][(q * P + ml) * P + nl % P];
                if constexpr (MODE == 1)
                    v[t] *= a.xs[m] * a.ws[t][n];
            }
            put(a, finish<GATED>(a, v[0], v[1], m, n), m, n);
        }
    }
}

}  // namespace skg

namespace skg_host {

template <int MODE, bool EXACT, int P, int MF, int NR, bool GATED, int DEPTH>
SmallKernel small_of()
{
    return SmallKernel{reinterpret_cast<const void *>(&skg::linear_small_kernel<MODE, EXACT, P, MF, NR, GATED, DEPTH>),
                       P * NR, (MODE ? 2048 : 1024) / P, DEPTH};
}

template <int MODE, bool EXACT, int NR, bool GATED>
SmallKernel small_wide(int M)
{
    if (M <= 32)
        return small_of<MODE, EXACT, 16, 2, NR, GATED, MODE ? 1 : 2>();
    return small_of<MODE, EXACT, 16, 4, NR, GATED, 1>();
}

// M <= 64. Up to 16 rows the conversions of the exact product hide behind the loads of W.
template <int MODE, int NR, bool GATED>
SmallKernel small_for(int M, bool exact)
{
    constexpr int D1 = (MODE ? 4 : 8) / (NR * (GATED ? 2 : 1));  // 8 loads of W in flight per set
    constexpr bool E = MODE != 0;
    if (M <= 4)
        return small_of<MODE, E, 4, 1, NR, GATED, D1>();
    if (M <= 8)
        return small_of<MODE, E, 8, 1, NR, GATED, D1>();
    if (M <= 16)
        return small_of<MODE, E, 16, 1, NR, GATED, D1>();
    return exact && MODE ? small_wide<MODE, E, NR, GATED>(M) : small_wide<MODE, false, NR, GATED>(M);
}

template <int MODE>
SmallKernel small_pick(int M, bool gated, int nr, bool exact)
{
    if (gated)
        return nr == 1 ? small_for<MODE, 1, true>(M, exact) : small_for<MODE, 2, true>(M, exact);
    return nr == 1 ? small_for<MODE, 1, false>(M, exact) : small_for<MODE, 2, false>(M, exact);
}

}  // namespace skg_host

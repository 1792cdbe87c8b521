// The projection kernel for up to a few hundred rows of x: W streams from HBM through LDS
// once, and K is split over the waves of a block.
//
// Every compute unit needs a part of W to stream, so the tiles of outputs are small (4 to
// 96 a side). Shared between the waves of a block along K, such a tile needs no barrier
// until its end: each wave fetches its own 128-byte parts of K (the tile's rows of W and
// x) into its own ring of stages in LDS and multiplies the whole tile, waiting for its own
// loads only, while the loads of its later stages and of the other waves are in flight.
// The loads write LDS directly, 8 rows of 128 bytes an instruction: a compute unit takes
// 64 bytes a clock that way, against 16 where an instruction loads 16 rows of 64 bytes,
// as the operand registers of the matrix instructions want them. Bound by HBM (few rows,
// medians of cold launches: 1 x 4096 x 4096 bfloat16 6.2 us, 5.5 TB/s; 1 x 12576 x 4096 e4m3
// 9.1 us, 5.6 TB/s) or by the 64 bytes a clock of W and x (many: 100 x 4096 x 8192 e4m3
// 13.5 us, 58 KB/us a compute unit over the whole launch). 8-bit integers go the same way, as
// integers: 1 x 12576 x 4096 8.2 to 10.4 us (6.2 TB/s at best), 5 x 77440 x 4096 45.9 (6.9),
// 100 x 4096 x 8192 12.0.
#pragma once

#include "lds_load.hpp"
#include "linear.hpp"

namespace skg {

// MODE: see linear.hpp; EXACT: see
// mfma_bytes. A block computes NB output features (of each
// weight, GATED) of TM * 16 rows with WAVES waves. NB = 8 fills half of an instruction's
// rows, or one half with each weight; NB = 4 (GATED) both weights' rows in one half, for
// N that fills too few compute units otherwise. A wave's part of LDS is a ring of RING stages; XR
// rows of x are loaded (8 where M <= 8, else TM * 16: what other columns of the
// instruction multiply reaches no output). NT: W is read with the non-temporal hint.
template <int MODE, bool EXACT, bool GATED, int NB, int TM, int XR, int RING, int WAVES, bool NT>
__global__ __launch_bounds__(WAVES * 64) void linear_stream_kernel(LinArgs a, int nt, int mt)
{
    constexpr bool BLOCK = MODE == kE4m3Block, HALVES = MODE == kBf16 || MODE == kInt8Row;
    constexpr int MATS = GATED ? 2 : 1;
    constexpr bool HALF = NB == 8, QUARTER = NB == 4;
    static_assert(!QUARTER || GATED, "a load takes 8 rows");
    constexpr int BN = NB * MATS, BM = TM * 16;
    constexpr int TN = (BN + 15) / 16;          // instructions along the rows of W
    constexpr int TF = HALF || QUARTER ? 1 : NB / 16;      // and along those of one weight
    constexpr int XS = (BM + 63) / 64;          // loads of x's scales, 64 each
    constexpr int SCALES = (BN + XR) * 128;     // offset of a stage's scales: of x, then of each weight
    constexpr int STAGE = SCALES + (BLOCK ? (XS + MATS) * 256 : 0);
    constexpr int LOADS = (QUARTER ? 2 : BN / 8) + XR / 8 + (BLOCK ? XS + MATS : 0);  // of one wave and stage
    constexpr int PART = WAVES * TN * TM * 1024;  // the waves' sums, after the last stage
    constexpr int SMEM = PART > WAVES * RING * STAGE ? PART : WAVES * RING * STAGE;
    static_assert(XR <= BM && 128 % NB == 0, "tile");
    __shared__ __attribute__((aligned(16))) uint8_t smem[SMEM];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;

    // Workgroups go to the 8 XCDs in turn; a run of neighbouring tiles, which share W,
    // goes to one of them.
    const int total = nt * mt;
    const int q8 = total / 8, r8 = total % 8;
    const int xcd = blockIdx.x % 8;
    const int t = xcd * q8 + (xcd < r8 ? xcd : r8) + (int)(blockIdx.x / 8);
    const int n0 = t / mt * NB, m0 = t % mt * BM;

    const int KB = MODE == kBf16 ? a.K * 2 : a.K;
    const int stages = (KB + 127) / 128;
    const int vn = a.N - n0 < NB ? a.N - n0 : NB;
    const int vm = a.M - m0 < BM ? a.M - m0 : BM;
    u32x4 wr[MATS], wsr[MATS], xsr;
#pragma unroll
    for (int q = 0; q < MATS; ++q)
        wr[q] = rsrc_words(a.w[q] + (int64_t)n0 * KB, (unsigned)vn * (unsigned)KB);
    const u32x4 xr = rsrc_words(a.x + (int64_t)m0 * a.ldx, (unsigned)(vm - 1) * (unsigned)a.ldx + (unsigned)KB);
    if constexpr (BLOCK) {
        xsr = rsrc_words(a.xs + (int64_t)m0 * a.kb, (unsigned)(vm * a.kb) * 4u);
#pragma unroll
        for (int q = 0; q < MATS; ++q)  // the tile's features lie in one block of 128
            wsr[q] = rsrc_words(a.ws[q] + (int64_t)(n0 / 128) * a.kb, (unsigned)a.kb * 4u);
    }
    const uint8_t *ring = smem + wave * RING * STAGE;
    const unsigned lds0 =
        (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)smem + wave * RING * STAGE;
    const int lrow = lane >> 3;
    // piece j of row r lies at position j ^ (r % 8) of the row's 128 bytes
    const unsigned piece = (unsigned)((lane & 7) ^ lrow) * 16u;

    auto issue = [&](int s, int slot) {
        const unsigned k = (unsigned)s * 128u + piece;
        const bool in = k < (unsigned)KB;
        const unsigned lds = lds0 + (unsigned)(slot * STAGE);
        if constexpr (QUARTER) {  // lane i writes at lds + 16 i, whichever lanes are off
            const unsigned at = in ? (unsigned)(lrow & 3) * (unsigned)KB + k : kOutOfRange;
            if (lane < 32)
                load_to_lds<NT>(wr[0], at, lds);
            else
                load_to_lds<NT>(wr[MATS - 1], at, lds);
        }
#pragma unroll
        for (int q = 0; q < MATS; ++q)
#pragma unroll
            for (int c = 0; c < NB / 8; ++c)
                load_to_lds<NT>(wr[q], in ? (unsigned)(c * 8 + lrow) * (unsigned)KB + k : kOutOfRange,
                            lds + (unsigned)(q * NB + c * 8) * 128u);
#pragma unroll
        for (int c = 0; c < XR / 8; ++c)
            load_to_lds(xr, in ? (unsigned)(c * 8 + lrow) * (unsigned)a.ldx + k : kOutOfRange,
                        lds + (unsigned)(BN + c * 8) * 128u);
        if constexpr (BLOCK) {
#pragma unroll
            for (int c = 0; c < XS; ++c) {
                const int m = c * 64 + lane;
                load4_to_lds(xsr, m < vm ? (unsigned)(m * a.kb + s) * 4u : kOutOfRange, lds + SCALES + 256u * c);
            }
#pragma unroll
            for (int q = 0; q < MATS; ++q)
                load4_to_lds(wsr[q], (unsigned)s * 4u, lds + SCALES + 256u * (XS + q));
        }
    };

    using sums = sums_t<MODE>;
    sums acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[i][j] = sums{0, 0, 0, 0};
    const int p0 = (g ^ (i16 & 7)) * 16, p1 = ((g + 4) ^ (i16 & 7)) * 16;

#pragma unroll
    for (int d = 0; d < RING; ++d)
        if (wave + d * WAVES < stages)
            issue(wave + d * WAVES, d);
    int slot = 0;
    for (int s = wave; s < stages; s += WAVES) {
        if (s + (RING - 1) * WAVES < stages)
            stage_wait<(RING - 1) * LOADS>();
        else
            stage_wait<0>();
        const uint8_t *st = ring + slot * STAGE;
        u32x4 af[TN][2], bf[TM][2];
        float sc[BLOCK ? TN : 1][BLOCK ? TM : 1];
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const int r = BN == 8 ? i16 & 7 : i * 16 + i16;
            af[i][0] = *reinterpret_cast<const u32x4 *>(st + r * 128 + p0);
            af[i][1] = *reinterpret_cast<const u32x4 *>(st + r * 128 + p1);
        }
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int r = BN + (XR == 8 ? i16 & 7 : j * 16 + i16);
            bf[j][0] = *reinterpret_cast<const u32x4 *>(st + r * 128 + p0);
            bf[j][1] = *reinterpret_cast<const u32x4 *>(st + r * 128 + p1);
        }
        if constexpr (BLOCK) {
            const float *f = reinterpret_cast<const float *>(st + SCALES);
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    sc[i][j] = f[j * 16 + i16] * f[64 * (XS + (QUARTER ? g & 1 : HALF && GATED ? g >> 1 : i / TF)) + lane];
        }
        lds_read_wait();  // the stage is in registers: its slot may be written again
        if (s + RING * WAVES < stages)
            issue(s + RING * WAVES, slot);
        slot = slot + 1 == RING ? 0 : slot + 1;
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                sums &c = acc[i][j];
                if constexpr (HALVES) {
                    c = mfma_half(af[i][0], bf[j][0], c);
                    c = mfma_half(af[i][1], bf[j][1], c);
                } else if constexpr (!BLOCK) {
                    c = mfma_bytes<EXACT>(af[i], bf[j], c);
                } else {
                    const f32x4 p = mfma_bytes<EXACT>(af[i], bf[j], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        c[e] = __builtin_fmaf(p[e], sc[i][j], c[e]);
                }
            }
    }

    // the waves' sums meet in LDS, added in the order of the waves
    __syncthreads();
    sums *part = reinterpret_cast<sums *>(smem);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            part[((wave * TN + i) * TM + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    constexpr int SLOTS = QUARTER ? 16 : HALF ? 32 : 64;  // lanes that hold outputs (of the first weight)
    for (int o = threadIdx.x; o < TF * TM * SLOTS; o += WAVES * 64) {
        const int l = o % SLOTS, j = o / SLOTS % TM, i = o / SLOTS / TM;
        const int m = m0 + j * 16 + (l & 15), n = n0 + i * 16 + (l >> 4) * 4;
        if (m >= a.M || n >= a.N)
            continue;
        const u32x2 r = residual4(a, m, n);
        sums z = sums{0, 0, 0, 0}, u = z;
#pragma unroll
        for (int k = 0; k < WAVES; ++k) {
            z += part[((k * TN + i) * TM + j) * 64 + l];
            if constexpr (GATED)
                u += HALF || QUARTER ? part[(k * TM + j) * 64 + SLOTS + l] : part[((k * TN + TF + i) * TM + j) * 64 + l];
        }
        finish4<MODE, GATED>(a, to_f32(z), to_f32(u), r, row_scaled(MODE) ? a.xs[m] : 1.0f, m, n);
    }
}

}  // namespace skg

namespace skg_host {

template <int MODE, bool EXACT, bool GATED, int NB, int TM, int XR, int RING, int WAVES, bool NT>
StreamKernel stream_of()
{
    constexpr int MATS = GATED ? 2 : 1, BN = NB * MATS, TN = (BN + 15) / 16;
    constexpr int STAGE = (BN + XR) * 128 + (MODE == skg::kE4m3Block ? ((TM + 3) / 4 + MATS) * 256 : 0);
    constexpr int RINGS = WAVES * RING * STAGE, PART = WAVES * TN * TM * 1024;
    return StreamKernel{
        reinterpret_cast<const void *>(&skg::linear_stream_kernel<MODE, EXACT, GATED, NB, TM, XR, RING, WAVES, NT>),
        NB, TM * 16, RING, WAVES, STAGE, RINGS > PART ? RINGS : PART, TN * TM};
}

// The kernels for M rows. Up to 16 rows one instruction takes all of x, W is read once
// (non-temporal), and the conversions of the exact 8-bit product hide behind its loads.
template <int MODE, bool EXACT, bool GATED>
int stream_set(int M, StreamKernel *out)
{
    constexpr bool E = MODE == skg::kE4m3Row || MODE == skg::kE4m3Block;
    int n = 0;
    if (M <= 8) {
        out[n++] = stream_of<MODE, E, GATED, 8, 1, 8, 2, 8, true>();
        out[n++] = stream_of<MODE, E, GATED, 8, 1, 8, 3, 8, true>();
        out[n++] = stream_of<MODE, E, GATED, 16, 1, 8, 2, 4, true>();
        out[n++] = stream_of<MODE, E, GATED, 16, 1, 8, 2, 8, true>();
        if constexpr (GATED)  // 8 x 1024 x 8192 bfloat16 8.4 us against 10.0 with 8 features a block
            out[n++] = stream_of<MODE, E, GATED, 4, 1, 8, 3, 8, true>();
    } else if (M <= 16) {
        out[n++] = stream_of<MODE, E, GATED, 8, 1, 16, 2, 8, true>();
        out[n++] = stream_of<MODE, E, GATED, 16, 1, 16, 2, 4, true>();
        out[n++] = stream_of<MODE, E, GATED, 16, 1, 16, 2, 8, true>();
        out[n++] = stream_of<MODE, E, GATED, 32, 1, 16, 2, 4, true>();
        if constexpr (GATED)
            out[n++] = stream_of<MODE, E, GATED, 4, 1, 16, 2, 8, true>();
    } else {
        out[n++] = stream_of<MODE, EXACT, GATED, 16, 1, 16, 1, 8, false>();
        out[n++] = stream_of<MODE, EXACT, GATED, 16, 2, 32, 2, 4, false>();
        out[n++] = stream_of<MODE, EXACT, GATED, 32, 2, 32, 1, 4, false>();
        out[n++] = stream_of<MODE, EXACT, GATED, 32, 2, 32, 2, 4, false>();
        out[n++] = stream_of<MODE, EXACT, GATED, 32, 4, 64, 1, 4, false>();
        out[n++] = stream_of<MODE, EXACT, GATED, 32, 4, 64, 1, 8, false>();
        if constexpr (!(EXACT && MODE == skg::kE4m3Block))  // where the registers hold it
            out[n++] = stream_of<MODE, EXACT, GATED, GATED ? 32 : 64, 6, 96, 1, 6, false>();
        if constexpr (!GATED) {
            out[n++] = stream_of<MODE, EXACT, GATED, 64, 3, 48, 1, 4, false>();
            out[n++] = stream_of<MODE, EXACT, GATED, 64, 4, 64, 1, 4, false>();
            out[n++] = stream_of<MODE, EXACT, GATED, 64, 4, 64, 1, 8, false>();
        }
    }
    static_assert(kStreamMost >= 10, "the largest set");
    return n;
}

template <int MODE>
int stream_pick(int M, bool gated, bool exact, StreamKernel *out)
{
    if constexpr (MODE == skg::kE4m3Row || MODE == skg::kE4m3Block)
        if (exact)
            return gated ? stream_set<MODE, true, true>(M, out) : stream_set<MODE, true, false>(M, out);
    return gated ? stream_set<MODE, false, true>(M, out) : stream_set<MODE, false, false>(M, out);
}

}  // namespace skg_host

// The projection kernel for many rows of x: blocks of BN x BM outputs, both operands
// staged through LDS.
//
// A stage is 128 bytes of K (64 bfloat16 or 128 e4m3: one block of scales) of the
// block's BN rows of W and BM rows of x. It is fetched by buffer loads that write LDS
// directly, one stage ahead of the products, into the other of two buffers; the only
// synchronisation per stage is one wait and one barrier. The loads write LDS in lane
// order, so the layout is chosen by what each lane asks for: piece j (16 bytes) of row r
// lies at position j ^ (r % 8) of the row's 128 bytes, and the 16-byte operand reads of
// eight neighbouring rows then touch every bank once.
//
// W is the A operand (rows of D) and x the B operand (columns), so a lane holds four
// consecutive output features of one row of y.
#pragma once

#include "linear.hpp"

namespace skg {

// A buffer load of 16 bytes per lane into LDS, lane i at lds + 16 i. Written as one
// instruction block because the compiler makes every later LDS read wait for all loads
// into LDS it knows of; it has no output register, and stage_wait() waits for it. M0
// holds the LDS address; nothing else in these kernels uses M0 (the compiler reserves it
// and sets it right before its own uses).
__device__ __forceinline__ void load_to_lds(const u32x4 &rsrc, unsigned offset, unsigned lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(offset), "s"(rsrc)
                 : "memory");
}

// This wave's loads into LDS have landed.
__device__ __forceinline__ void stage_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ u32x4 rsrc_words(const void *base, unsigned bytes)
{
    const unsigned long long p = (unsigned long long)base;
    u32x4 r;
    r[0] = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)p);
    r[1] = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)(p >> 32)) & 0xFFFFu;
    r[2] = (unsigned)__builtin_amdgcn_readfirstlane((int)bytes);
    r[3] = kBufferFlags;
    return r;
}

// MODE and EXACT as in linear_small.hpp. WN x WM waves, each TN x TM instructions of
// 16 x 16.
template <int MODE, bool EXACT, bool GATED, int WN, int WM, int TN, int TM>
__global__ __launch_bounds__(WN *WM * 64) void linear_tile_kernel(LinArgs a, int nt, int mt)
{
    constexpr bool FP8 = MODE != 0, BLOCK = MODE == 2;
    constexpr int WAVES = WN * WM;
    constexpr int BN = WN * TN * 16, BM = WM * TM * 16;
    constexpr int MATS = GATED ? 2 : 1;
    constexpr int NB = BN / MATS;          // output features per block
    constexpr int TF = TN / MATS;          // instructions per wave along them
    constexpr int STAGE = (BN + BM) * 128;
    constexpr int WL = NB / 8 / WAVES, XL = BM / 8 / WAVES;  // loads per wave and stage
    static_assert(TN % MATS == 0 && NB % (8 * WAVES) == 0 && BM % (8 * WAVES) == 0, "whole loads per wave");
    __shared__ uint8_t smem[2][STAGE];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int wn = wave % WN, wm = wave / WN;

    // Workgroups go to the 8 XCDs in turn. Each XCD takes a contiguous run of tiles, in
    // groups of 8 rows of tiles by column, so that its L2 serves one group's W and x.
    const int total = nt * mt;
    const int q8 = total / 8, r8 = total % 8;
    const int xcd = blockIdx.x % 8, at = blockIdx.x / 8;
    const int t = xcd * q8 + (xcd < r8 ? xcd : r8) + at;
    constexpr int GROUP = 8;
    const int per = GROUP * nt;
    const int first = t / per * GROUP;
    const int rows = mt - first < GROUP ? mt - first : GROUP;
    const int n0 = (t % per) / rows * NB, m0 = (first + (t % per) % rows) * BM;

    const int KB = FP8 ? a.K : a.K * 2;
    const int stages = (KB + 127) / 128;
    const int vn = a.N - n0 < NB ? a.N - n0 : NB;
    const int vm = a.M - m0 < BM ? a.M - m0 : BM;
    u32x4 wr[MATS];
#pragma unroll
    for (int q = 0; q < MATS; ++q)
        wr[q] = rsrc_words(a.w[q] + (int64_t)n0 * KB, (unsigned)vn * (unsigned)KB);
    const u32x4 xr = rsrc_words(a.x + (int64_t)m0 * a.ldx, (unsigned)(vm - 1) * (unsigned)a.ldx + (unsigned)KB);
    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)&smem[0][0];
    const int lrow = lane >> 3;
    const unsigned piece = (unsigned)((lane & 7) ^ lrow) * 16u;

    auto issue = [&](int s) {
        const unsigned k = (unsigned)s * 128u + piece;
        const bool in = k < (unsigned)KB;
        const unsigned lds = lds0 + (unsigned)(s & 1) * STAGE;
#pragma unroll
        for (int q = 0; q < MATS; ++q)
#pragma unroll
            for (int i = 0; i < WL; ++i) {
                const int c = wave * WL + i;  // 8 rows each
                load_to_lds(wr[q], in ? (unsigned)(c * 8 + lrow) * (unsigned)KB + k : kOutOfRange,
                            lds + (unsigned)(q * NB + c * 8) * 128u);
            }
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int c = wave * XL + i;
            load_to_lds(xr, in ? (unsigned)(c * 8 + lrow) * (unsigned)a.ldx + k : kOutOfRange,
                        lds + (unsigned)(BN + c * 8) * 128u);
        }
    };

    // scales of the block of K that stage s holds: x per row, W per 128 features
    float xsc[BLOCK ? TM : 1], wsc[BLOCK ? TN : 1];
    auto scales = [&](int s) {
        if constexpr (BLOCK) {
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int m = m0 + (wm * TM + j) * 16 + i16;
                xsc[j] = a.xs[(int64_t)(m < a.M ? m : a.M - 1) * a.kb + s];
            }
#pragma unroll
            for (int i = 0; i < TN; ++i) {
                const int n = n0 + (wn * TF + i % TF) * 16;
                wsc[i] = a.ws[i / TF][(int64_t)((n < a.N ? n : a.N - 1) / 128) * a.kb + s];
            }
        }
    };

    f32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // rows of this wave's fragments in a stage; piece p of row r is at p ^ (r % 8)
    int arow[TN], brow[TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
        arow[i] = (i / TF) * NB + (wn * TF + i % TF) * 16 + i16;
#pragma unroll
    for (int j = 0; j < TM; ++j)
        brow[j] = BN + (wm * TM + j) * 16 + i16;
    const int p0 = (g ^ (i16 & 7)) * 16, p1 = ((g + 4) ^ (i16 & 7)) * 16;

    issue(0);
    scales(0);
    for (int s = 0; s < stages; ++s) {
        stage_wait();
        __syncthreads();  // the stage is whole, and every wave has left the other buffer
        float xc[BLOCK ? TM : 1], wc[BLOCK ? TN : 1];
        if constexpr (BLOCK) {
#pragma unroll
            for (int j = 0; j < TM; ++j)
                xc[j] = xsc[j];
#pragma unroll
            for (int i = 0; i < TN; ++i)
                wc[i] = wsc[i];
        }
        if (s + 1 < stages) {
            issue(s + 1);
            scales(s + 1);
        }
        const uint8_t *st = smem[s & 1];
        if constexpr (!FP8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 af[TN], bf[TM];
#pragma unroll
                for (int i = 0; i < TN; ++i)
                    af[i] = *reinterpret_cast<const u32x4 *>(st + arow[i] * 128 + (h ? p1 : p0));
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    bf[j] = *reinterpret_cast<const u32x4 *>(st + brow[j] * 128 + (h ? p1 : p0));
#pragma unroll
                for (int i = 0; i < TN; ++i)
#pragma unroll
                    for (int j = 0; j < TM; ++j)
                        acc[i][j] = mfma_bf16(af[i], bf[j], acc[i][j]);
            }
        } else {
            u32x4 bf[TM][2];
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                bf[j][0] = *reinterpret_cast<const u32x4 *>(st + brow[j] * 128 + p0);
                bf[j][1] = *reinterpret_cast<const u32x4 *>(st + brow[j] * 128 + p1);
            }
#pragma unroll
            for (int i = 0; i < TN; ++i) {
                const u32x4 af[2] = {*reinterpret_cast<const u32x4 *>(st + arow[i] * 128 + p0),
                                     *reinterpret_cast<const u32x4 *>(st + arow[i] * 128 + p1)};
#pragma unroll
                for (int j = 0; j < TM; ++j) {
                    if constexpr (BLOCK) {
                        const f32x4 p = mfma_bytes<EXACT>(af, bf[j], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                        const float sc = xc[j] * wc[i];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[i][j][e] = __builtin_fmaf(p[e], sc, acc[i][j][e]);
                    } else {
                        acc[i][j] = mfma_bytes<EXACT>(af, bf[j], acc[i][j]);
                    }
                }
            }
        }
    }

#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int m = m0 + (wm * TM + j) * 16 + i16;
        if (m >= a.M)
            continue;
        const float xs = MODE == 1 ? a.xs[m] : 1.0f;
#pragma unroll
        for (int i = 0; i < TF; ++i) {
            const int n = n0 + (wn * TF + i) * 16 + g * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (n + e >= a.N)
                    continue;
                float z = acc[i][j][e], u = GATED ? acc[TF * (MATS - 1) + i][j][e] : 0.0f;
                if constexpr (MODE == 1) {
                    z *= xs * a.ws[0][n + e];
                    if constexpr (GATED)
                        u *= xs * a.ws[1][n + e];
                }
                put(a, finish<GATED>(a, z, u, m, n + e), m, n + e);
            }
        }
    }
}

}  // namespace skg

namespace skg_host {

struct TileKernel {
    const void *fn;
    int bn, bm, threads;  // outputs per block along N and M
};

// size 0: the smallest tile, 2: the largest
template <int MODE, bool EXACT, bool GATED>
TileKernel tile_of(int size)
{
    using namespace skg;
    constexpr int G = GATED ? 2 : 1;
    if (size == 0)
        return {reinterpret_cast<const void *>(&linear_tile_kernel<MODE, EXACT, GATED, 2, 2, 2, 2>), 64 / G, 64, 256};
    if (size == 1)
        return {reinterpret_cast<const void *>(&linear_tile_kernel<MODE, EXACT, GATED, 2, 2, 4, 4>), 128 / G, 128, 256};
    return {reinterpret_cast<const void *>(&linear_tile_kernel<MODE, EXACT, GATED, 4, 2, 4, 8>), 256 / G, 256, 512};
}

template <int MODE>
TileKernel tile_pick(bool gated, bool exact, int size)
{
    if constexpr (MODE != 0)
        if (exact) {  // rare and slower: the two smaller tiles serve it
            size = size > 1 ? 1 : size;
            return gated ? tile_of<MODE, true, true>(size) : tile_of<MODE, true, false>(size);
        }
    return gated ? tile_of<MODE, false, true>(size) : tile_of<MODE, false, false>(size);
}

TileKernel tile_kernel_bf16(bool gated, bool exact, int size);
TileKernel tile_kernel_row(bool gated, bool exact, int size);
TileKernel tile_kernel_block(bool gated, bool exact, int size);

}  // namespace skg_host

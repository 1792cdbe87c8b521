// The projection kernel for many rows of x: blocks of outputs whose W and x are staged
// through LDS and shared by the block's waves.
//
// A stage is 128 bytes of K (64 bfloat16 or 128 e4m3: one block of scales) of the block's
// rows of W and x, fetched by buffer loads that write LDS directly, in lane order, so the
// layout is chosen by what each lane asks for: piece j (16 bytes) of row r lies at position
// j ^ (r % 8) of the row's 128 bytes, and the 16-byte operand reads of eight neighbouring
// rows touch every bank once.
//
// W is the A operand (rows of D) and x the B operand (columns), so a lane holds four
// consecutive output features of one row of y. A wave multiplies TN x TM fragments; per
// stage it reads TN + TM of them from LDS, so large wave tiles keep LDS below the matrix
// pipe: 128 x 128 outputs read 32 KB a stage for 2048 clocks of products.
//
// Within a stage the wave goes along its TN fragments of W, reading the next while it
// multiplies the current one with all TM of x. Behind the last of those reads comes the
// stage's main barrier: the next stage is whole, and the buffer of this stage's W is
// free. The products that are left (one and a half rows) cover the reads of the next
// stage's x and first W fragment and the issue of later loads. A second barrier early in a
// stage, which each wave reaches when its reads of x have returned, frees the buffer of that
// stage's x. With three buffers for W
// and two for x the loads are issued two stages ahead: fetched one stage ahead, the
// largest tile's stages took 3900 clocks for 2048 clocks of products.
//
// The loop over the stages has no branch (behind one, the compiler moved the sums between
// the two register files at every step): stages past the last read zeros, since every
// load past K does, and add nothing.
//
// Bound by the matrix pipe at the clock that it leaves (1.75 GHz of 2.4 while products of
// 4096 rows run one after another): 4096^3 in bfloat16 96 to 105 us by the card (1310 to
// 1430 TF), 107 to 118 with residual, activation and cold inputs; e4m3 with row scales
// 4096 x 4096 x 8192 in 92 to 97 (2830 to 2990 TF), 101 to 108 with bias, residual and cold
// inputs. 8-bit integers are at the same rate: 4095 x 4096 x 8192 with bias and residual in
// 102 to 109, and exact. With block scales, where each product has four multiply-adds behind it and no tile is
// larger than 256 x 128, 4096^3 takes 74 to 78 against 51 to 53. For float32 outputs of
// 8-bit inputs both operands are widened at every use: 4096 x 4096 x 8192 307 to 318 with row
// scales, 339 to 353 with block scales. At the tiles of 128 x 128, by what a compute unit
// takes into LDS (32 KB a stage at some 75 KB/us).
#pragma once

#include "lds_load.hpp"
#include "linear.hpp"

namespace skg {

// MODE and EXACT as in mfma_bytes. WN x WM waves, each TN x TM fragments of 16 x 16
// (GATED: half of TN for each weight).
template <int MODE, bool EXACT, bool GATED, int WN, int WM, int TN, int TM>
__global__ __launch_bounds__(WN *WM * 64) void linear_tile_kernel(LinArgs a, int nt, int mt)
{
    constexpr bool BLOCK = MODE == kE4m3Block, HALVES = MODE == kBf16 || MODE == kInt8Row;
    constexpr bool PINNED = !BLOCK;  // products and reads of a stage stay in source order
    constexpr int WAVES = WN * WM;
    constexpr int BN = WN * TN * 16, BM = WM * TM * 16;
    constexpr int MATS = GATED ? 2 : 1;
    constexpr int NB = BN / MATS;          // output features per block
    constexpr int TF = TN / MATS;          // fragments per wave along them
    constexpr int WBUFS = 3, XBUFS = 2;
    constexpr int WBUF = BN * 128, XBUF = BM * 128;
    constexpr int WL = NB / 8 / WAVES, XL = BM / 8 / WAVES;  // loads per wave and stage
    constexpr int XS = XL + (BLOCK ? 1 + MATS : 0);          // of x and the scales
    constexpr int LOADS = MATS * WL + XS;
    // scales of a stage, per wave: one float for each of its rows of x and fragments of W
    constexpr int SBUF = BLOCK ? (1 + MATS) * 256 : 0;
    constexpr int SLOTS = TM / 2 + TM;     // products behind a stage's main barrier
    static_assert(TN >= 4 && TN % 2 == 0 && TN % MATS == 0 && TM % 2 == 0, "fragments");
    static_assert(NB % (8 * WAVES) == 0 && BM % (8 * WAVES) == 0, "whole loads per wave");
    static_assert(TM <= 4 || !BLOCK, "a wave's scales of x are one load");
    __shared__ __attribute__((aligned(16))) uint8_t smem[WBUFS * WBUF + XBUFS * XBUF + WAVES * XBUFS * SBUF];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int wn = wave % WN, wm = wave / WN;

    // Workgroups go to the 8 XCDs in turn. Each XCD takes a contiguous run of tiles, in
    // groups of 4 or 8 rows of tiles by column, so that its L2 serves one group's W and x.
    const int total = nt * mt;
    const int q8 = total / 8, r8 = total % 8;
    const int xcd = blockIdx.x % 8, at = blockIdx.x / 8;
    const int t = xcd * q8 + (xcd < r8 ? xcd : r8) + at;
    constexpr int GROUP = BN * BM >= 65536 ? 4 : 8;  // 4096^3 took 121 us against 128 with 8
    const int per = GROUP * nt;
    const int first = t / per * GROUP;
    const int rows = mt - first < GROUP ? mt - first : GROUP;
    const int n0 = (t % per) / rows * NB, m0 = (first + (t % per) % rows) * BM;

    const int KB = MODE == kBf16 ? a.K * 2 : a.K;
    const int stages = (KB + 127) / 128;
    const int vn = a.N - n0 < NB ? a.N - n0 : NB;
    const int vm = a.M - m0 < BM ? a.M - m0 : BM;
    u32x4 wr[MATS];
#pragma unroll
    for (int q = 0; q < MATS; ++q)
        wr[q] = rsrc_words(a.w[q] + (int64_t)n0 * KB, (unsigned)vn * (unsigned)KB);
    const u32x4 xr = rsrc_words(a.x + (int64_t)m0 * a.ldx, (unsigned)(vm - 1) * (unsigned)a.ldx + (unsigned)KB);
    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)smem;
    const int lrow = lane >> 3;
    const unsigned piece = (unsigned)((lane & 7) ^ lrow) * 16u;

    const int sbase = WBUFS * WBUF + XBUFS * XBUF + wave * XBUFS * SBUF;  // this wave's scales
    u32x4 xsr, wsr[MATS];
    if constexpr (BLOCK) {
        xsr = rsrc_words(a.xs + (int64_t)m0 * a.kb, (unsigned)(vm * a.kb) * 4u);
#pragma unroll
        for (int q = 0; q < MATS; ++q)
            wsr[q] = rsrc_words(a.ws[q] + (int64_t)(n0 / 128) * a.kb,
                                (unsigned)((n0 % 128 + vn + 127) / 128 * a.kb) * 4u);
    }
    // load l of this wave's share of stage s of W, into the buffer at `buf`, and of x
    auto issue_w = [&](int s, unsigned buf, auto lc) {
        constexpr int l = decltype(lc)::value, q = l / WL, i = l % WL;
        const unsigned k = (unsigned)s * 128u + piece;
        const int c = wave * WL + i;  // 8 rows each
        load_to_lds(wr[q], k < (unsigned)KB ? (unsigned)(c * 8 + lrow) * (unsigned)KB + k : kOutOfRange,
                    lds0 + buf + (unsigned)(q * NB + c * 8) * 128u);
    };
    auto issue_x = [&](int s, int par, auto lc) {
        constexpr int l = decltype(lc)::value;
        if constexpr (l < XL) {
            const unsigned k = (unsigned)s * 128u + piece;
            const int c = wave * XL + l;
            load_to_lds(xr, k < (unsigned)KB ? (unsigned)(c * 8 + lrow) * (unsigned)a.ldx + k : kOutOfRange,
                        lds0 + WBUFS * WBUF + (unsigned)(par * XBUF + c * 8 * 128));
        } else if constexpr (l == XL) {
            const int m = wm * TM * 16 + lane;
            load4_to_lds(xsr, lane < TM * 16 && m < vm && s < a.kb ? (unsigned)(m * a.kb + s) * 4u : kOutOfRange,
                         lds0 + (unsigned)(sbase + par * SBUF));
        } else {
            constexpr int q = l - XL - 1;
            const int n = n0 % 128 + (wn * TF + lane) * 16;  // lane: a fragment of W
            load4_to_lds(wsr[q],
                         lane < TF && n - n0 % 128 < vn && s < a.kb ? (unsigned)(n / 128 * a.kb + s) * 4u : kOutOfRange,
                         lds0 + (unsigned)(sbase + par * SBUF + 256 * (1 + q)));
        }
    };

    // scales of the block of K that a stage holds, by the parity of the stage
    float xsc[2][BLOCK ? TM : 1], wsc[2][BLOCK ? TN : 1];
    auto read_scales = [&](auto pc) {
        constexpr int p = decltype(pc)::value;
        if constexpr (BLOCK) {
            const float *f = reinterpret_cast<const float *>(smem + sbase + p * SBUF);
#pragma unroll
            for (int j = 0; j < TM; ++j)
                xsc[p][j] = f[j * 16 + i16];
#pragma unroll
            for (int i = 0; i < TN; ++i)
                wsc[p][i] = f[64 * (1 + i / TF) + i % TF];
        }
    };

    using sums = sums_t<MODE>;
    sums acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[i][j] = sums{0, 0, 0, 0};

    // this lane's pieces of a fragment's row; piece p of row r is at p ^ (r % 8)
    const int p0 = (g ^ (i16 & 7)) * 16, p1 = ((g + 4) ^ (i16 & 7)) * 16;
    const int abase = wn * TF * 16 + i16, bbase = wm * TM * 16 + i16;
    u32x4 af[2][2], bf[2][TM][2];
    auto read_a = [&](const uint8_t *st, int i, u32x4 (&f)[2]) {
        const uint8_t *r = st + (abase + (i / TF) * NB + i % TF * 16) * 128;
        f[0] = *reinterpret_cast<const u32x4 *>(r + p0);
        f[1] = *reinterpret_cast<const u32x4 *>(r + p1);
    };
    auto read_b = [&](const uint8_t *st, int j, u32x4 (&f)[2]) {
        const uint8_t *r = st + (bbase + j * 16) * 128;
        f[0] = *reinterpret_cast<const u32x4 *>(r + p0);
        f[1] = *reinterpret_cast<const u32x4 *>(r + p1);
    };

    // wcur, wnext: the buffers of W of stages s and s + 1; that of s + 3 is wcur again
    auto stage = [&](int s, unsigned wcur, unsigned wnext, auto pc) {
        constexpr int P = decltype(pc)::value;
        const uint8_t *st = smem + wcur, *xn = smem + WBUFS * WBUF + (P ^ 1) * XBUF;
        static_for<0, TN>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            if constexpr (i + 1 < TN)
                read_a(st, i + 1, af[(i + 1) & 1]);
            // the two products of a sum stay TM apart: back to back, the second would wait
            if constexpr (HALVES)
                static_for<0, TM>([&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    acc[i][j] = mfma_half(af[i & 1][0], bf[P][j][0], acc[i][j]);
                });
            static_for<0, TM>([&](auto jc) {
                constexpr int j = decltype(jc)::value;
                sums &c = acc[i][j];
                if constexpr (HALVES) {
                    c = mfma_half(af[i & 1][1], bf[P][j][1], c);
                } else if constexpr (!BLOCK) {
                    c = mfma_bytes<EXACT>(af[i & 1], bf[P][j], c);
                } else {
                    const f32x4 p = mfma_bytes<EXACT>(af[i & 1], bf[P][j], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                    const float sc = xsc[P][j] * wsc[P][i];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        c[e] = __builtin_fmaf(p[e], sc, c[e]);
                }
                if constexpr (i == 0 && j == TM - 1) {
                    // This wave's reads of the stage's x and scales have returned; behind the
                    // barrier every wave's have, and their buffers are free. The wait stands
                    // here because the compiler may move the products, which would ask for
                    // it, behind the barrier. Where the order is pinned the two youngest
                    // reads are fragment 1 of W, which stay under way: waiting for them too
                    // takes up to 3% of a launch (e4m3 1500 x 2380 x 2048 12.0 -> 12.3 us).
                    lds_read_wait<PINNED && !EXACT ? 2 : 0>();
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                }
                if constexpr (i == 1)
                    static_for<j * XS / TM, (j + 1) * XS / TM>([&](auto l) { issue_x(s + 2, P, l); });
                if constexpr (i == TN - 2 && j == TM / 2 - 1) {
                    // This wave has read the stage's W, and its loads of the next stage are
                    // done: behind them are those of W and x two stages ahead.
                    lds_read_wait();
                    stage_wait<LOADS>();
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                }
                if constexpr ((i == TN - 2 && j >= TM / 2) || i == TN - 1) {
                    constexpr int q = i == TN - 1 ? TM / 2 + j : j - TM / 2;
                    if constexpr (q < TM)
                        read_b(xn, q, bf[P ^ 1][q]);
                    if constexpr (q == TM) {
                        read_a(smem + wnext, 0, af[0]);
                        read_scales(std::integral_constant<int, P ^ 1>{});
                    }
                    static_for<q * (MATS * WL) / SLOTS, (q + 1) * (MATS * WL) / SLOTS>(
                        [&](auto l) { issue_w(s + 3, wcur, l); });
                }
                if constexpr (PINNED)
                    __builtin_amdgcn_sched_barrier(0);
            });
        });
    };

    // loads in the order in which the stages wait for them
    auto all_w = [&](int s) {
        static_for<0, MATS * WL>([&](auto l) { issue_w(s, (unsigned)(s * WBUF), l); });
    };
    auto all_x = [&](int s) { static_for<0, XS>([&](auto l) { issue_x(s, s, l); }); };
    all_w(0);
    all_x(0);
    all_w(1);
    all_x(1);
    all_w(2);
    stage_wait<LOADS + MATS * WL>();
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TM; ++j)
        read_b(smem + WBUFS * WBUF, j, bf[0][j]);
    read_a(smem, 0, af[0]);
    read_scales(std::integral_constant<int, 0>{});
    unsigned w0 = 0, w1 = WBUF, w2 = 2 * WBUF;
    for (int s = 0; s < stages; s += 2) {
        stage(s, w0, w1, std::integral_constant<int, 0>{});
        stage(s + 1, w1, w2, std::integral_constant<int, 1>{});
        const unsigned w = w0;
        w0 = w2;
        w2 = w1;
        w1 = w;
    }

    // The sums go through LDS, so that a wave stores whole rows of the tile: straight from
    // the registers a store instruction covers 32 bytes of each of 16 rows. Outside its
    // stages the tile of 256 x 256 spends 12 us of 4096^3 this way, 30 without. Piece p (4
    // outputs) of row r lies at position p ^ (r % 16), so neither side meets on a bank.
    constexpr int SMEM = WBUFS * WBUF + XBUFS * XBUF + WAVES * XBUFS * SBUF;
    constexpr int PASSES = BN * BM * 4 > SMEM ? 2 : 1;
    constexpr int JP = TM / PASSES, RP = WM * JP * 16;  // fragments per wave, rows per pass
    constexpr int PL = NB / 8;                          // lanes per row, 8 outputs each
    constexpr int RI = 64 / PL, ITERS = RP / (RI * WAVES);
    static_assert(PL <= 64 && RP % (RI * WAVES) == 0 && ITERS % 2 == 0, "rows per wave");
    const int pl = lane % PL, sub = lane / PL, n = n0 + pl * 8;
    const bool wide = n + 8 <= a.N;
    Columns8<MODE, GATED> cols;
    cols.load(a, n, wide);
    // row k of this lane in pass q; its residuals are loaded before the first store, too
    auto row_of = [&](int k) { return (k * WAVES + wave) * RI + sub; };
    auto m_of = [&](int q, int row) { return m0 + (row / (JP * 16) * TM + q * JP) * 16 + row % (JP * 16); };
    u32x4 res[GATED ? 1 : PASSES * ITERS];
    if constexpr (!GATED)
        if (a.res) {
#pragma unroll
            for (int k = 0; k < PASSES * ITERS; ++k) {
                const int m = m_of(k / ITERS, row_of(k % ITERS));
                res[k] = m < a.M && wide ? *reinterpret_cast<const u32x4_any *>(a.res + (int64_t)m * a.ldr + n)
                                         : u32x4{0, 0, 0, 0};
            }
        }
    float xsv[MODE == kInt8Row ? TM : 1];  // integer sums are multiplied when they become floats
    if constexpr (row_scaled(MODE)) {
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int m = m0 + (wm * TM + j) * 16 + i16;
            const float xs = m < a.M ? a.xs[m] : 0.0f;
            if constexpr (MODE == kInt8Row) {
                xsv[j] = xs;
            } else {
#pragma unroll
                for (int i = 0; i < TN; ++i)
                    acc[i][j] *= xs;
            }
        }
    }
    cols.settle();
    stage_wait();  // the loads past the last stage have written their zeros
    static_for<0, PASSES>([&](auto qc) {
        constexpr int q = decltype(qc)::value;
        __syncthreads();
        static_for<0, JP>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            const int row = (wm * JP + j) * 16 + i16;
            static_for<0, TN>([&](auto ic) {
                constexpr int i = decltype(ic)::value;
                const int p = ((i / TF) * NB + (wn * TF + i % TF) * 16) / 4 + g;
                *reinterpret_cast<f32x4 *>(smem + row * (BN * 4) + (p ^ i16) * 16) =
                    MODE == kInt8Row ? to_f32(acc[i][q * JP + j]) * xsv[MODE == kInt8Row ? q * JP + j : 0]
                                     : to_f32(acc[i][q * JP + j]);
            });
        });
        __syncthreads();
        auto sums_of = [&](int row, f32x4 (&z)[2], f32x4 (&u)[2]) {
            const uint8_t *at_row = smem + row * (BN * 4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                z[h] = *reinterpret_cast<const f32x4 *>(at_row + ((pl * 2 + h) ^ (row & 15)) * 16);
                u[h] = GATED ? *reinterpret_cast<const f32x4 *>(at_row + ((NB / 4 + pl * 2 + h) ^ (row & 15)) * 16) : z[h];
            }
        };
        if (GATED || !a.res) {
#pragma unroll 2
            for (int k = 0; k < ITERS; ++k) {
                const int row = row_of(k), m = m_of(q, row);
                f32x4 z[2], u[2];
                sums_of(row, z, u);
                if (m < a.M && wide)
                    cols.finish(a, z, u, u32x4{0, 0, 0, 0}, m, n);
            }
        } else if constexpr (!GATED) {
            if constexpr (q == 0)
#pragma unroll
                for (int k = 0; k < PASSES * ITERS; ++k)
                    asm volatile("" : "+v"(res[k]));
#pragma unroll
            for (int k = 0; k < ITERS; ++k) {
                const int row = row_of(k), m = m_of(q, row);
                f32x4 z[2], u[2];
                sums_of(row, z, u);
                if (m < a.M && wide)
                    cols.finish(a, z, u, res[q * ITERS + k], m, n);
            }
        }
        if (vn % 8)  // the columns behind the last eight
#pragma unroll 1
            for (int o = threadIdx.x; o < RP * 8; o += WAVES * 64) {
                const int row = o / 8, m = m_of(q, row), c = (vn & ~7) + o % 8;
                const float *at = reinterpret_cast<const float *>(smem + row * (BN * 4) + c % 4 * 4);
                if (c < vn && m < a.M) {
                    float z = at[(c / 4 ^ (row & 15)) * 4], u = at[((NB * GATED + c) / 4 ^ (row & 15)) * 4];
                    if constexpr (row_scaled(MODE)) {
                        z *= a.ws[0][n0 + c];
                        u *= a.ws[GATED][n0 + c];
                    }
                    put(a, finish<GATED>(a, z, u, m, n0 + c), m, n0 + c);
                }
            }
    });
}

}  // namespace skg

namespace skg_host {

template <int MODE, bool EXACT, bool GATED, int WN, int WM, int TN, int TM>
TileKernel tile_of(float stage_us)
{
    return TileKernel{reinterpret_cast<const void *>(&skg::linear_tile_kernel<MODE, EXACT, GATED, WN, WM, TN, TM>),
                      WN * TN * 16 / (GATED ? 2 : 1), WM * TM * 16, WN * WM, stage_us};
}

// The stage times were fitted beside the other constants of the choice of kernel: full
// chip, a compute unit's blocks one after another (two of 128 x 128 run beside each
// other). The tile of 128 x 128 has 4 waves for bfloat16 (fewer operand reads from LDS; 8
// waves fitted the same time) and 8 for 8-bit products (more of them to cover a wait where a
// compute unit has one block: 0.42 us a stage against 0.63 with row scales, 0.65 against 0.76
// with block scales).
template <int MODE, bool EXACT, bool GATED>
int tile_set(TileKernel *out)
{
    int n = 0;
    if constexpr (EXACT) {  // for float32 outputs only: one tile serves them
        out[n++] = tile_of<MODE, EXACT, GATED, 2, 2, 4, 4>(1.2f);
    } else if constexpr (MODE == skg::kE4m3Block) {
        out[n++] = tile_of<MODE, EXACT, GATED, 2, 2, 4, 2>(0.47f);
        out[n++] = tile_of<MODE, EXACT, GATED, 2, 4, 4, 2>(0.65f);
        out[n++] = tile_of<MODE, EXACT, GATED, 4, 2, 4, 4>(0.87f);
    } else if constexpr (skg::row_scaled(MODE)) {
        out[n++] = tile_of<MODE, EXACT, GATED, 2, 2, 4, 2>(0.4f);
        out[n++] = tile_of<MODE, EXACT, GATED, 2, 4, 4, 2>(0.42f);
        out[n++] = tile_of<MODE, EXACT, GATED, 4, 2, 4, 4>(0.72f);
        out[n++] = tile_of<MODE, EXACT, GATED, 2, 4, 8, 4>(1.3f);
    } else {
        out[n++] = tile_of<MODE, EXACT, GATED, 2, 2, 4, 2>(0.36f);
        out[n++] = tile_of<MODE, EXACT, GATED, 2, 2, 4, 4>(0.5f);
        out[n++] = tile_of<MODE, EXACT, GATED, 4, 2, 4, 4>(0.89f);
        out[n++] = tile_of<MODE, EXACT, GATED, 2, 4, 8, 4>(1.44f);
    }
    static_assert(kTileMost >= 4, "the largest set");
    return n;
}

template <int MODE>
int tile_pick(bool gated, bool exact, TileKernel *out)
{
    if constexpr (MODE == skg::kE4m3Row || MODE == skg::kE4m3Block)
        if (exact)
            return gated ? tile_set<MODE, true, true>(out) : tile_set<MODE, true, false>(out);
    return gated ? tile_set<MODE, false, true>(out) : tile_set<MODE, false, false>(out);
}

}  // namespace skg_host

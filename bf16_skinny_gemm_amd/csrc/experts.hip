// The experts of a mixture-of-experts layer for a few tokens (include/skinny_moe.h): two
// kernels, h = act(x Wg^T) * (x Wu^T) for every pair (token, expert), and the weighted sum
// of h Wd^T over each token's experts.
//
// Few tokens name many experts, so the weights of the experts that are named, read from HBM
// once, are all that costs: 3 I H values each. The pairs are sorted by expert; a tile is up
// to BM pairs of one expert, whose rows of x (or h) one pass over the expert's weight
// multiplies. Both kernels stream weights as linear_stream.hpp does: each wave has its own
// ring of stages of 128 bytes of K in LDS, filled by loads that write LDS, and waits for its
// own loads only.
//
//  - up: one block per tile and NB features of both weights. K = H is split over its
//    waves, whose sums meet in LDS at the end.
//  - down: one block per NB outputs of all tokens. Each wave takes a run of the stages of
//    all tiles, one after the other, so its loads go on from one expert to the next; behind
//    a tile it adds its sums, times the token's weight, to its own outputs [tokens][NB] in
//    LDS. The waves' outputs are added in the order of the waves: no atomics, the same bits
//    every time.
//
// 8-bit weights are widened to bfloat16 (exactly) and multiplied by x as it is, so that only
// h and y are rounded: at 16 rows a tile, the matrix instructions cost nothing.
#include "ops_host.hpp"

#include <cmath>
#include <cstdint>

#include "lds_load.hpp"
#include "linear.hpp"
#include "validate_moe.hpp"

namespace skg {

// The weights' types.
enum { kWBf16 = SKINNY_WEIGHTS_BF16, kWRow = SKINNY_WEIGHTS_E4M3_ROW, kWBlock = SKINNY_WEIGHTS_E4M3_BLOCK,
       kWInt8 = SKINNY_WEIGHTS_INT8_ROW };
constexpr bool scaled_rows(int type) { return type == kWRow || type == kWInt8; }

struct ExpertArgs {
    const uint16_t *x;
    const int *ids;
    const float *weights;
    const uint8_t *w[2], *wd;   // gate and up, down
    const float *s[2], *sd;     // their scales
    const uint16_t *res;        // or null
    uint16_t *y, *h;
    unsigned *plan;             // [0] tiles; from [4]: expert | pairs << 10 | first pair << 16 of each
    u32x4 *entries;             // for each pair, by expert: token, its weight
    int64_t ldx, ldr, ldy;      // elements
    int64_t up_bytes, down_bytes;  // from one expert's weight to the next
    int64_t up_scales, down_scales;
    int M, E, k, H, I;
    int act;
};

constexpr int kMostPairs = skg_host::kExpertsRows * skg_host::kMaxExpertsK;  // 4096: 12 bits and one
constexpr int kMostTiles = skg_host::kMaxExperts + kMostPairs / 8;
static_assert(skg_host::kMaxExperts <= 1 << 10 && kMostPairs <= 1 << 15, "a tile is one word");

// Sixteen 8-bit integers as bfloat16.
__device__ __forceinline__ void widen_int8(const u32x4 &v, u32x4 &lo, u32x4 &hi)
{
    auto two = [](unsigned w, int at) {
        const float a = (float)(int8_t)(w >> at), b = (float)(int8_t)(w >> (at + 8));
        // both are bfloat16 values: their upper halves
        return __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, b), __builtin_bit_cast(unsigned, a), 0x07060302u);
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        lo[2 * i] = two(v[i], 0);
        lo[2 * i + 1] = two(v[i], 16);
        hi[2 * i] = two(v[2 + i], 0);
        hi[2 * i + 1] = two(v[2 + i], 16);
    }
}

template <int TYPE>
__device__ __forceinline__ void widen_weight(const u32x4 &v, u32x4 &lo, u32x4 &hi)
{
    if constexpr (TYPE == kWInt8)
        widen_int8(v, lo, hi);
    else
        widen(v, lo, hi);
}

// x (or h) of a stage lies in PLANES planes of [rows][128 bytes], a column of weights beside
// the same column of x: the 16 bytes of an 8-bit weight beside two pieces of 16 bytes.
template <int TYPE>
constexpr int planes() { return TYPE == kWBf16 ? 1 : 2; }

// One fragment of weights (the lane's pieces g and g + 4 of its row), widened.
template <int TYPE>
struct Fragment {
    u32x4 v[2 * planes<TYPE>()];

    __device__ __forceinline__ void read(const uint8_t *row, int g, int swizzle)
    {
        const u32x4 a = *reinterpret_cast<const u32x4 *>(row + (g ^ swizzle) * 16);
        const u32x4 b = *reinterpret_cast<const u32x4 *>(row + ((g + 4) ^ swizzle) * 16);
        if constexpr (TYPE == kWBf16) {
            v[0] = a;
            v[1] = b;
        } else {
            widen_weight<TYPE>(a, v[0], v[1]);
            widen_weight<TYPE>(b, v[2], v[3]);
        }
    }
};

// The lane's pieces of x that meet Fragment::v; `plane` bytes from one plane to the next.
template <int TYPE>
__device__ __forceinline__ void read_x(const uint8_t *row, int g, int swizzle, int plane, u32x4 (&v)[2 * planes<TYPE>()])
{
    if constexpr (TYPE == kWBf16) {
        v[0] = *reinterpret_cast<const u32x4 *>(row + (g ^ swizzle) * 16);
        v[1] = *reinterpret_cast<const u32x4 *>(row + ((g + 4) ^ swizzle) * 16);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] = *reinterpret_cast<const u32x4 *>(row + (q / 2) * plane + ((2 * g + q % 2) ^ swizzle) * 16);
    }
}

// ---- the pairs by expert -----------------------------------------------------------

struct Tile {
    int expert, first, pairs;  // expert < 0: there is no such tile
};

// Pairs of up to one wave: every wave sorts them in its lanes. Returns tile t; *pair: in lane
// r the r-th pair of the tile.
template <int BM>
__device__ __forceinline__ Tile find_tile_wave(const ExpertArgs &a, int P, int t, int *pair)
{
    const int lane = threadIdx.x & 63;
    int id = lane < P ? a.ids[lane] : -1;
    id = (unsigned)id < (unsigned)a.E ? id : 0x7FFFFFFF;
    int rank = 0, less = 0;
    for (int q = 0; q < P; ++q) {
        const int o = __builtin_amdgcn_readlane(id, q);
        rank += o == id && q < lane;
        less += o < id;
    }
    const int pos = lane < P ? less + rank : lane;  // where the pair goes
    const int sid = __builtin_amdgcn_ds_permute(pos * 4, id);
    const int srank = __builtin_amdgcn_ds_permute(pos * 4, rank);
    const int spair = __builtin_amdgcn_ds_permute(pos * 4, lane);
    const unsigned long long firsts = __ballot(lane < P && sid != 0x7FFFFFFF && srank % BM == 0);
    const int before = __builtin_amdgcn_mbcnt_hi((unsigned)(firsts >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)firsts, 0));
    const unsigned long long at = __ballot((firsts >> lane & 1) && before == t);
    if (!at)
        return Tile{-1, 0, 0};
    const int first = __builtin_ctzll(at);
    const int expert = __builtin_amdgcn_readlane(sid, first);
    const int pairs = __popcll(__ballot(sid == expert && lane >= first && lane < first + BM));
    *pair = __builtin_amdgcn_ds_bpermute((first + lane) * 4, spair);
    return Tile{expert, first, pairs};
}

// More pairs: counted by expert in LDS by the whole block.
struct Counts {
    int pairs[skg_host::kMaxExperts];   // of each expert; then, of the plan, its first pair
    uint16_t ids[kMostPairs];           // of each pair; 0xFFFF: none
    int found[4];
    uint16_t list[64];                  // pairs of the tile
};

// Ends behind a barrier.
template <int THREADS>
__device__ __forceinline__ void count_pairs(const ExpertArgs &a, int P, Counts &c)
{
    for (int e = threadIdx.x; e < a.E; e += THREADS)
        c.pairs[e] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < P; p += THREADS) {
        const int id = a.ids[p];
        const bool in = (unsigned)id < (unsigned)a.E;
        c.ids[p] = in ? (uint16_t)id : (uint16_t)0xFFFF;
        if (in)
            atomicAdd(&c.pairs[id], 1);  // integers: the order changes nothing
    }
    __syncthreads();
}

// Inclusive sums over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(v, d, 64);
        v += lane >= d ? o : 0;
    }
    return v;
}

// The first wave: this lane's experts [lo, hi), and the pairs and tiles before them.
template <int BM>
__device__ __forceinline__ void before_lane(const ExpertArgs &a, const Counts &c, int &lo, int &hi, int &pairs, int &tiles)
{
    const int lane = threadIdx.x & 63, per = (a.E + 63) / 64;
    lo = lane * per < a.E ? lane * per : a.E;
    hi = lo + per < a.E ? lo + per : a.E;
    int np = 0, nt = 0;
    for (int e = lo; e < hi; ++e) {
        np += c.pairs[e];
        nt += (c.pairs[e] + BM - 1) / BM;
    }
    pairs = wave_scan(np) - np;
    tiles = wave_scan(nt) - nt;
}

// Tile t of the block's counted pairs, its pairs in c.list.
template <int BM>
__device__ __forceinline__ Tile find_tile_block(const ExpertArgs &a, int P, int t, Counts &c)
{
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        if (lane == 0)
            c.found[0] = -1;
        int lo, hi, pairs, tiles;
        before_lane<BM>(a, c, lo, hi, pairs, tiles);
        for (int e = lo; e < hi; ++e) {
            const int n = c.pairs[e], nt = (n + BM - 1) / BM;
            if (t >= tiles && t < tiles + nt) {
                const int r = (t - tiles) * BM;
                c.found[0] = e;
                c.found[1] = pairs + r;
                c.found[2] = n - r < BM ? n - r : BM;
                c.found[3] = r;
            }
            pairs += n;
            tiles += nt;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
        const int e = c.found[0], r0 = c.found[3], n = c.found[2];
        if (e >= 0)
            for (int p0 = 0, seen = 0; p0 < P && seen < r0 + n; p0 += 64) {
                const bool mine = p0 + lane < P && c.ids[p0 + lane] == e;
                const unsigned long long b = __ballot(mine);
                const int r = seen + __builtin_amdgcn_mbcnt_hi((unsigned)(b >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)b, 0)) - r0;
                if (mine && r >= 0 && r < n)
                    c.list[r] = (uint16_t)(p0 + lane);
                seen += __popcll(b);
            }
    }
    __syncthreads();
    return Tile{__builtin_amdgcn_readfirstlane(c.found[0]), __builtin_amdgcn_readfirstlane(c.found[1]),
                __builtin_amdgcn_readfirstlane(c.found[2])};
}

// The tiles and the sorted pairs for the second kernel, written by one block of the first.
template <int BM, int THREADS>
__device__ __forceinline__ void write_plan(const ExpertArgs &a, int P, Counts &c)
{
    if (threadIdx.x < 64) {
        int lo, hi, pairs, tiles;
        before_lane<BM>(a, c, lo, hi, pairs, tiles);
        for (int e = lo; e < hi; ++e) {
            const int n = c.pairs[e];
            for (int r = 0; r < n; r += BM)
                a.plan[4 + tiles++] = (unsigned)e | (unsigned)(n - r < BM ? n - r : BM) << 10 | (unsigned)(pairs + r) << 16;
            c.pairs[e] = pairs;
            pairs += n;
        }
        if (threadIdx.x == 63)
            a.plan[0] = (unsigned)tiles;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += THREADS) {
        int at = c.pairs[e];
        for (int p = 0; p < P; ++p)
            if (c.ids[p] == e)
                a.entries[at++] = u32x4{(unsigned)(p / a.k), __builtin_bit_cast(unsigned, a.weights[p]), 0, 0};
    }
}

// ---- up ------------------------------------------------------------------------------

// blockIdx.x == 0 writes the plan; the others take a tile each (blockIdx.x - 1) / nt and NB
// features. WAVE: the pairs fit one wave.
template <int TYPE, int NB, int BM, int RING, int WAVES, bool WAVE>
__global__ __launch_bounds__(WAVES * 64) void experts_up_kernel(ExpertArgs a, int nt)
{
    constexpr bool BLOCK = TYPE == kWBlock;
    constexpr int PLANES = planes<TYPE>();
    constexpr bool HALF = NB == 8;
    constexpr int BN = 2 * NB, TN = BN / 16, TM = (BM + 15) / 16;
    constexpr int TF = HALF ? 1 : NB / 16;
    constexpr int XAT = BN * 128, XPLANE = BM * 128, SAT = XAT + PLANES * XPLANE;
    constexpr int STAGE = SAT + (BLOCK ? 512 : 0);
    constexpr int LOADS = BN / 8 + PLANES * BM / 8 + (BLOCK ? 2 : 0);
    constexpr int PART = WAVES * TN * TM * 1024, RINGS = WAVES * RING * STAGE;
    constexpr int PLAN = (int)sizeof(Counts);
    constexpr int SMEM = RINGS > PART ? (RINGS > PLAN ? RINGS : PLAN) : (PART > PLAN ? PART : PLAN);
    static_assert(BM % 8 == 0 && BM <= 64 && 128 % NB == 0 && (RING - 1) * LOADS < 64, "tile");
    __shared__ __attribute__((aligned(16))) uint8_t smem[SMEM];
    Counts &counts = *reinterpret_cast<Counts *>(smem);

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int P = a.M * a.k;
    if (blockIdx.x == 0) {
        count_pairs<WAVES * 64>(a, P, counts);
        write_plan<BM, WAVES * 64>(a, P, counts);
        return;
    }
    const int t = (int)(blockIdx.x - 1) / nt, n0 = (int)(blockIdx.x - 1) % nt * NB;
    Tile tile;
    int pair = 0;
    if constexpr (WAVE) {
        tile = find_tile_wave<BM>(a, P, t, &pair);
    } else {
        count_pairs<WAVES * 64>(a, P, counts);
        tile = find_tile_block<BM>(a, P, t, counts);
        pair = counts.list[lane];
        __syncthreads();  // the ring is written over the counts
    }
    if (tile.expert < 0)
        return;

    const int KB = TYPE == kWBf16 ? a.H * 2 : a.H;
    const int stages = (KB + 127) / 128;
    const int vn = a.I - n0 < NB ? a.I - n0 : NB;
    const int hb = (a.H + 127) / 128;
    u32x4 wr[2], wsr[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        wr[q] = rsrc_words(a.w[q] + tile.expert * a.up_bytes + (int64_t)n0 * KB, (unsigned)vn * (unsigned)KB);
        if constexpr (BLOCK)
            wsr[q] = rsrc_words(a.s[q] + tile.expert * a.up_scales + (int64_t)(n0 / 128) * hb, (unsigned)hb * 4u);
    }
    const unsigned ldx = (unsigned)a.ldx * 2u, XB = (unsigned)a.H * 2u;
    const u32x4 xr = rsrc_words(a.x, (unsigned)(a.M - 1) * ldx + XB);
    const uint8_t *ring = smem + wave * RING * STAGE;
    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)smem + wave * RING * STAGE;
    const int lrow = lane >> 3;
    const unsigned piece = (unsigned)((lane & 7) ^ lrow) * 16u;
    // the rows of x that this lane loads pieces of
    unsigned xat[BM / 8];
#pragma unroll
    for (int c = 0; c < BM / 8; ++c) {
        const int r = c * 8 + lrow, p = __builtin_amdgcn_ds_bpermute(r * 4, pair);
        xat[c] = r < tile.pairs ? (unsigned)(p / a.k) * ldx : kOutOfRange;
    }

    auto issue = [&](int s, int slot) {
        const unsigned k = (unsigned)s * 128u + piece;
        const unsigned lds = lds0 + (unsigned)(slot * STAGE);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int c = 0; c < NB / 8; ++c)
                load_to_lds<true>(wr[q], k < (unsigned)KB ? (unsigned)(c * 8 + lrow) * (unsigned)KB + k : kOutOfRange,
                                  lds + (unsigned)(q * NB + c * 8) * 128u);
#pragma unroll
        for (int h = 0; h < PLANES; ++h) {
            const unsigned b = (unsigned)(s * PLANES + h) * 128u + piece;
#pragma unroll
            for (int c = 0; c < BM / 8; ++c)
                load_to_lds(xr, b < XB && xat[c] != kOutOfRange ? xat[c] + b : kOutOfRange,
                            lds + XAT + (unsigned)(h * XPLANE + c * 1024));
        }
        if constexpr (BLOCK) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                load4_to_lds(wsr[q], (unsigned)s * 4u, lds + SAT + 256u * q);
        }
    };

    f32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
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
        Fragment<TYPE> af[TN];
        u32x4 bf[TM][2 * PLANES];
        float sc[TN];
#pragma unroll
        for (int i = 0; i < TN; ++i)
            af[i].read(st + (i * 16 + i16) * 128, g, i16 & 7);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int r = BM == 8 ? i16 & 7 : j * 16 + i16;
            read_x<TYPE>(st + XAT + r * 128, g, r & 7, XPLANE, bf[j]);
        }
        if constexpr (BLOCK) {
            const float *f = reinterpret_cast<const float *>(st + SAT);
#pragma unroll
            for (int i = 0; i < TN; ++i)
                sc[i] = f[64 * (HALF ? g >> 1 : i / TF) + lane];
        }
        lds_read_wait();  // the stage is in registers: its slot may be written again
        if (s + RING * WAVES < stages)
            issue(s + RING * WAVES, slot);
        slot = slot + 1 == RING ? 0 : slot + 1;
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                f32x4 p = BLOCK ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][j];
#pragma unroll
                for (int q = 0; q < 2 * PLANES; ++q)
                    p = mfma_bf16(af[i].v[q], bf[j][q], p);
                if constexpr (BLOCK) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][j][e] = __builtin_fmaf(p[e], sc[i], acc[i][j][e]);
                } else {
                    acc[i][j] = p;
                }
            }
    }

    // the waves' sums meet in LDS, added in the order of the waves
    __syncthreads();
    f32x4 *part = reinterpret_cast<f32x4 *>(smem);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            part[((wave * TN + i) * TM + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    constexpr int SLOTS = HALF ? 32 : 64;  // lanes that hold outputs of the gate
    for (int o = threadIdx.x; o < TF * TM * SLOTS; o += WAVES * 64) {
        const int l = o % SLOTS, j = o / SLOTS % TM, i = o / SLOTS / TM;
        const int r = j * 16 + (l & 15), n = n0 + i * 16 + (l >> 4) * 4;
        if (r >= tile.pairs || n >= a.I)
            continue;
        f32x4 z = f32x4{0.0f, 0.0f, 0.0f, 0.0f}, u = z;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            z += part[((w * TN + i) * TM + j) * 64 + l];
            u += HALF ? part[(w * TM + j) * 64 + SLOTS + l] : part[((w * TN + TF + i) * TM + j) * 64 + l];
        }
        // I is a multiple of 8: all four are there
        if constexpr (scaled_rows(TYPE)) {
            z *= *reinterpret_cast<const f32x4_any *>(a.s[0] + tile.expert * a.up_scales + n);
            u *= *reinterpret_cast<const f32x4_any *>(a.s[1] + tile.expert * a.up_scales + n);
        }
        z = activate4(z, a.act) * u;
        *reinterpret_cast<u32x2 *>(a.h + (int64_t)(tile.first + r) * a.I + n) = u32x2{pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3])};
    }
}

// ---- down ----------------------------------------------------------------------------

// MC: tokens that the block has room for.
template <int TYPE, int NB, int BM, int RING, int WAVES, int MC>
__global__ __launch_bounds__(WAVES * 64) void experts_down_kernel(ExpertArgs a, int most_tiles)
{
    constexpr bool BLOCK = TYPE == kWBlock;
    constexpr int PLANES = planes<TYPE>();
    constexpr int TM = (BM + 15) / 16;
    constexpr int XAT = NB * 128, XPLANE = BM * 128, EAT = XAT + PLANES * XPLANE;
    constexpr int STAGE = EAT + 1024 + (TYPE == kWBf16 ? 0 : 256);  // a load of entries takes 64 places
    constexpr int LOADS = NB / 8 + PLANES * BM / 8 + 1 + (TYPE == kWBf16 ? 0 : 1);
    constexpr int OUTS = MC * NB;  // floats of a wave
    static_assert((NB == 8 || NB == 16) && BM % 8 == 0 && BM <= 32 && (RING - 1) * LOADS < 64, "tile");
    __shared__ __attribute__((aligned(16))) uint8_t smem[WAVES * RING * STAGE];
    __shared__ __attribute__((aligned(16))) float outs[WAVES * OUTS];
    __shared__ unsigned tiles[kMostTiles];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * NB;
    for (int i = threadIdx.x; i < most_tiles; i += WAVES * 64)
        tiles[i] = a.plan[4 + i];
    const int nt = __builtin_amdgcn_readfirstlane((int)a.plan[0]);
    float *out = outs + wave * OUTS;
    for (int i = lane; i < a.M * NB / 4; i += 64)
        reinterpret_cast<f32x4 *>(out)[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    __syncthreads();

    const int KB = TYPE == kWBf16 ? a.I * 2 : a.I;
    const unsigned XB = (unsigned)a.I * 2u;
    const int stages = (KB + 127) / 128, ib = (a.I + 127) / 128;
    const int vn = a.H - n0 < NB ? a.H - n0 : NB;
    const int total = nt * stages;
    const int from = (int)((int64_t)total * wave / WAVES), to = (int)((int64_t)total * (wave + 1) / WAVES);
    const uint8_t *ring = smem + wave * RING * STAGE;
    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)smem + wave * RING * STAGE;
    const int lrow = lane >> 3;
    const unsigned piece = (unsigned)((lane & 7) ^ lrow) * 16u;

    // the tile and stage that are loaded next
    int it = from < to ? from / stages : 0, is = from < to ? from % stages : 0;
    u32x4 wr, hr, er, sr;
    auto enter = [&](int t) {
        const unsigned v = __builtin_amdgcn_readfirstlane((int)tiles[t]);
        const int e = (int)(v & 1023u), pairs = (int)(v >> 10 & 63u), first = (int)(v >> 16);
        wr = rsrc_words(a.wd + e * a.down_bytes + (int64_t)n0 * KB, (unsigned)vn * (unsigned)KB);
        hr = rsrc_words(a.h + (int64_t)first * a.I, (unsigned)pairs * XB);
        er = rsrc_words(a.entries + first, (unsigned)pairs * 16u);
        if constexpr (BLOCK)
            sr = rsrc_words(a.sd + e * a.down_scales + (int64_t)(n0 / 128) * ib, (unsigned)ib * 4u);
        else if constexpr (scaled_rows(TYPE))
            sr = rsrc_words(a.sd + e * a.down_scales + n0, (unsigned)vn * 4u);
    };
    auto issue = [&](int slot) {
        const unsigned k = (unsigned)is * 128u + piece;
        const unsigned lds = lds0 + (unsigned)(slot * STAGE);
#pragma unroll
        for (int c = 0; c < NB / 8; ++c)
            load_to_lds<true>(wr, k < (unsigned)KB ? (unsigned)(c * 8 + lrow) * (unsigned)KB + k : kOutOfRange,
                              lds + (unsigned)c * 1024u);
#pragma unroll
        for (int h = 0; h < PLANES; ++h) {
            const unsigned b = (unsigned)(is * PLANES + h) * 128u + piece;
#pragma unroll
            for (int c = 0; c < BM / 8; ++c)  // rows beyond the tile's lie beyond the resource
                load_to_lds(hr, b < XB ? (unsigned)(c * 8 + lrow) * XB + b : kOutOfRange,
                            lds + XAT + (unsigned)(h * XPLANE + c * 1024));
        }
        load_to_lds(er, (unsigned)lane * 16u, lds + EAT);
        if constexpr (BLOCK)
            load4_to_lds(sr, (unsigned)is * 4u, lds + EAT + 1024u);
        else if constexpr (scaled_rows(TYPE))
            load4_to_lds(sr, lane < NB ? (unsigned)lane * 4u : kOutOfRange, lds + EAT + 1024u);
        if (++is == stages) {
            is = 0;
            if (++it < nt)
                enter(it);
        }
    };

    f32x4 acc[TM];
    auto clear = [&] {
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    clear();
    int ct = it, cs = is;  // the tile and stage that are multiplied next
    if (from < to) {
        enter(it);
#pragma unroll
        for (int d = 0; d < RING; ++d)
            if (from + d < to)
                issue(d);
    }
    int slot = 0;
    for (int s = from; s < to; ++s) {
        if (s + RING <= to)
            stage_wait<(RING - 1) * LOADS>();
        else
            stage_wait<0>();
        const uint8_t *st = ring + slot * STAGE;
        Fragment<TYPE> af;
        u32x4 bf[TM][2 * PLANES], entry[TM];
        float sc = 1.0f;
        f32x4 rows = {1.0f, 1.0f, 1.0f, 1.0f};
        const bool last = ++cs == stages || s + 1 == to;
        af.read(st + (NB == 8 ? i16 & 7 : i16) * 128, g, i16 & 7);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int r = BM == 8 ? i16 & 7 : j * 16 + i16;
            read_x<TYPE>(st + XAT + r * 128, g, r & 7, XPLANE, bf[j]);
            entry[j] = *reinterpret_cast<const u32x4 *>(st + EAT + r * 16);
        }
        if constexpr (BLOCK)
            sc = *reinterpret_cast<const float *>(st + EAT + 1024 + lane * 4);
        else if constexpr (scaled_rows(TYPE))
            rows = *reinterpret_cast<const f32x4 *>(st + EAT + 1024 + (g * 4 % NB) * 4);
        lds_read_wait();  // the stage is in registers: its slot may be written again
        if (s + RING < to)
            issue(slot);
        slot = slot + 1 == RING ? 0 : slot + 1;
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            f32x4 p = BLOCK ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[j];
#pragma unroll
            for (int q = 0; q < 2 * PLANES; ++q)
                p = mfma_bf16(af.v[q], bf[j][q], p);
            if constexpr (BLOCK) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[j][e] = __builtin_fmaf(p[e], sc, acc[j][e]);
            } else {
                acc[j] = p;
            }
        }
        if (last) {
            const int pairs = (int)(__builtin_amdgcn_readfirstlane((int)tiles[ct]) >> 10 & 63);
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int c = j * 16 + i16;
                const bool live = c < pairs && (NB == 16 || g < 2);
                const int token = (int)entry[j][0];
                const unsigned weight = entry[j][1];  // a bit_cast of the element itself takes the first one
                f32x4 v = acc[j] * __builtin_bit_cast(float, weight);
                if constexpr (scaled_rows(TYPE))
                    v *= rows;
                f32x4 *at = reinterpret_cast<f32x4 *>(out + token * NB + g * 4);
                // the pairs of an expert are in the order of their tokens: one that names it
                // twice has two pairs side by side, which must not add at the same time
                const int beside = __shfl_up(token, 1, 16);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                if (!__ballot(live && i16 > 0 && token == beside)) {
                    if (live)
                        *at += v;
                } else {
                    for (int i = 0; i < 16; ++i) {
                        if (live && i16 == i)
                            *at += v;
                        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    }
                }
            }
            clear();
        }
        if (cs == stages) {
            cs = 0;
            ++ct;
        }
    }

    __syncthreads();
    for (int o = threadIdx.x; o < a.M * NB / 4; o += WAVES * 64) {
        const int m = o / (NB / 4), n = n0 + o % (NB / 4) * 4;
        if (n >= a.H)
            continue;
        u32x2 r = {0, 0};  // H is a multiple of 8: all four are there
        if (a.res)
            r = *reinterpret_cast<const u32x2_any *>(a.res + m * a.ldr + n);
        f32x4 z = widen4(r);
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            v += *reinterpret_cast<const f32x4 *>(outs + w * OUTS + o * 4);
        if (a.res)
            v += z;
        *reinterpret_cast<u32x2_any *>(a.y + m * a.ldy + n) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
}

// ---- any alignment, stride and size ---------------------------------------------------

// Value i of a weight.
template <int TYPE>
__device__ __forceinline__ float weight_at(const uint8_t *w, int64_t i)
{
    if constexpr (TYPE == kWBf16)
        return bf16_to_f32(reinterpret_cast<const uint16_t *>(w)[i]);
    else if constexpr (TYPE == kWInt8)
        return (float)reinterpret_cast<const int8_t *>(w)[i];
    else
        return __builtin_amdgcn_cvt_f32_fp8((int)w[i], 0);
}

__device__ __forceinline__ float any_sum(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        v += __shfl_xor(v, d, 64);
    return v;
}

// One wave per pair and feature: h of pair p is row p.
template <int TYPE>
__global__ __launch_bounds__(256) void experts_up_any_kernel(ExpertArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t all = (int64_t)a.M * a.k * a.I, step = (int64_t)gridDim.x * 4;
    const int hb = (a.H + 127) / 128;
    for (int64_t o = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); o < all; o += step) {
        const int p = (int)(o / a.I), n = (int)(o % a.I), e = a.ids[p];
        if ((unsigned)e >= (unsigned)a.E)
            continue;
        const uint16_t *x = a.x + (int64_t)(p / a.k) * a.ldx;
        float v[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint8_t *w = a.w[q] + e * a.up_bytes;
            const float *s = TYPE == kWBf16 ? nullptr : a.s[q] + e * a.up_scales;
            float sum = 0.0f;
            for (int i = lane; i < a.H; i += 64) {
                const float t = bf16_to_f32(x[i]) * weight_at<TYPE>(w, (int64_t)n * a.H + i);
                if constexpr (TYPE == kWBlock)
                    sum = __builtin_fmaf(t, s[(int64_t)(n >> 7) * hb + (i >> 7)], sum);
                else
                    sum += t;
                if (i > 0x7FFFFFFF - 64)
                    break;
            }
            sum = any_sum(sum);
            v[q] = scaled_rows(TYPE) ? sum * s[n] : sum;
        }
        float z[1] = {v[0]};
        activate(z, a.act);
        if (lane == 0)
            a.h[o] = f32_to_bf16(z[0] * v[1]);
    }
}

// One wave per token and output.
template <int TYPE>
__global__ __launch_bounds__(256) void experts_down_any_kernel(ExpertArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t all = (int64_t)a.M * a.H, step = (int64_t)gridDim.x * 4;
    const int ib = (a.I + 127) / 128;
    for (int64_t o = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); o < all; o += step) {
        const int m = (int)(o / a.H), n = (int)(o % a.H);
        float y = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int p = m * a.k + j, e = a.ids[p];
            if ((unsigned)e >= (unsigned)a.E)
                continue;
            const uint8_t *w = a.wd + e * a.down_bytes;
            const float *s = TYPE == kWBf16 ? nullptr : a.sd + e * a.down_scales;
            float sum = 0.0f;
            for (int i = lane; i < a.I; i += 64) {
                const float t = bf16_to_f32(a.h[(int64_t)p * a.I + i]) * weight_at<TYPE>(w, (int64_t)n * a.I + i);
                if constexpr (TYPE == kWBlock)
                    sum = __builtin_fmaf(t, s[(int64_t)(n >> 7) * ib + (i >> 7)], sum);
                else
                    sum += t;
                if (i > 0x7FFFFFFF - 64)
                    break;
            }
            sum = any_sum(sum);
            y = __builtin_fmaf(scaled_rows(TYPE) ? sum * s[n] : sum, a.weights[p], y);
        }
        if (lane == 0) {
            if (a.res)
                y += bf16_to_f32(a.res[m * a.ldr + n]);
            a.y[m * a.ldy + n] = f32_to_bf16(y);
        }
    }
}

}  // namespace skg

namespace skg_host {
namespace {

// A launch holds fewer than 2^32 threads; blocks here have at most 512.
constexpr int64_t kMaxBlocks = 1 << 22;

// One tile height with its kernels: the first, for pairs of one wave or more, and the second,
// for up to 16, 64 or 128 tokens.
struct ExpertsKernels {
    const void *up[2], *down[3];
    int up_features, down_features, up_waves, down_waves[3], rows;
};

template <int TYPE, int BM>
const ExpertsKernels &kernels_of()
{
    using namespace skg;
    constexpr bool BYTES = TYPE != kWBf16;
    constexpr int RU = BM == 32 && BYTES ? 1 : 2, R8 = BM == 8 ? 3 : 2, R4 = BM == 32 && BYTES ? 2 : 3;
    static const ExpertsKernels k = {{(const void *)&experts_up_kernel<TYPE, 8, BM, RU, 8, false>,
                                      (const void *)&experts_up_kernel<TYPE, 8, BM, RU, 8, true>},
                                     {(const void *)&experts_down_kernel<TYPE, 16, BM, BM == 32 ? 1 : R8, 8, 16>,
                                      (const void *)&experts_down_kernel<TYPE, 16, BM, R4, 4, 64>,
                                      (const void *)&experts_down_kernel<TYPE, 16, BM, R4, 4, 128>},
                                     8, 16, 8, {8, 4, 4}, BM};
    return k;
}

template <int TYPE>
const ExpertsKernels &kernels_for(int rows)
{
    return rows <= 8 ? kernels_of<TYPE, 8>() : rows <= 16 ? kernels_of<TYPE, 16>() : kernels_of<TYPE, 32>();
}

template <int TYPE>
int run_type(const skg::ExpertArgs &a, bool vector, hipStream_t stream)
{
    using namespace skg;
    ExpertArgs args = a;
    const int P = a.M * a.k;
    // pairs of an expert that has any, were the pairs spread evenly
    const double some = a.E * (1.0 - std::pow(1.0 - 1.0 / a.E, P)), even = P / some;
    const ExpertsKernels &k = kernels_for<TYPE>(even <= 4.0 ? 8 : even <= 10.0 ? 16 : 32);
    int most = a.E + P / k.rows;  // tiles, at most
    most = P < most ? P : most;
    int nt = (a.I + k.up_features - 1) / k.up_features;
    if (!vector || (int64_t)most * nt > kMaxBlocks) {
        void *p[] = {&args};
        const int64_t up = ((int64_t)a.M * a.k * a.I + 3) / 4, down = ((int64_t)a.M * a.H + 3) / 4;
        const int st = ops_launch((const void *)&experts_up_any_kernel<TYPE>, dim3((unsigned)(up < (1 << 20) ? up : 1 << 20)),
                                  256, p, stream);
        return st != SKINNY_OK ? st
                               : ops_launch((const void *)&experts_down_any_kernel<TYPE>,
                                            dim3((unsigned)(down < (1 << 20) ? down : 1 << 20)), 256, p, stream);
    }
    void *up[] = {&args, &nt};
    const int st = ops_launch(k.up[P <= 64], dim3((unsigned)(1 + most * nt)), k.up_waves * 64, up, stream);
    if (st != SKINNY_OK)
        return st;
    const int room = a.M <= 16 ? 0 : a.M <= 64 ? 1 : 2;
    void *down[] = {&args, &most};
    return ops_launch(k.down[room], dim3((unsigned)((a.H + k.down_features - 1) / k.down_features)), k.down_waves[room] * 64,
                      down, stream);
}

}  // namespace
}  // namespace skg_host

extern "C" {

size_t skinny_experts_workspace_bytes(int32_t M, int32_t k, int32_t E, int32_t I)
{
    using namespace skg_host;
    return experts_sizes_ok(M, k, E, I) && M > 0 ? (size_t)experts_space(M, k, E, I).bytes : 0;
}

int skinny_experts(const skinny_experts_t *e, hipStream_t stream)
{
    using namespace skg_host;
    int st = validate_experts(e);
    if (st != SKINNY_OK || e->M == 0)
        return st;
    int cus = 0;
    st = ops_device(&cus);
    if (st != SKINNY_OK)
        return st;
    const int size = e->type == SKINNY_WEIGHTS_BF16 ? 2 : 1;
    const ExpertsSpace space = experts_space(e->M, e->k, e->E, e->I);
    uint8_t *ws = static_cast<uint8_t *>(e->workspace);
    skg::ExpertArgs a{};
    a.w[0] = static_cast<const uint8_t *>(e->w_gate);
    a.w[1] = static_cast<const uint8_t *>(e->w_up);
    a.wd = static_cast<const uint8_t *>(e->w_down);
    a.s[0] = e->gate_scale;
    a.s[1] = e->up_scale;
    a.sd = e->down_scale;
    a.plan = reinterpret_cast<unsigned *>(ws);
    a.entries = reinterpret_cast<skg::u32x4 *>(ws + space.entries);
    a.h = reinterpret_cast<uint16_t *>(ws + space.h);
    a.ldx = e->ldx;
    a.ldr = e->ldr;
    a.ldy = e->ldy;
    a.up_bytes = e->up_stride * size;
    a.down_bytes = e->down_stride * size;
    a.up_scales = e->up_scale_stride;
    a.down_scales = e->down_scale_stride;
    a.E = e->E;
    a.k = e->k;
    a.H = e->H;
    a.I = e->I;
    a.act = e->act;
    const bool vector = experts_vector_ok(*e);
    for (int64_t m = 0; m < e->M; m += kExpertsRows) {
        a.M = (int)(e->M - m < kExpertsRows ? e->M - m : kExpertsRows);
        a.x = static_cast<const uint16_t *>(e->x) + m * e->ldx;
        a.ids = e->ids + m * e->k;
        a.weights = e->weights + m * e->k;
        a.res = e->residual ? static_cast<const uint16_t *>(e->residual) + m * e->ldr : nullptr;
        a.y = static_cast<uint16_t *>(e->y) + m * e->ldy;
        switch (e->type) {
        case SKINNY_WEIGHTS_BF16:
            st = run_type<skg::kWBf16>(a, vector, stream);
            break;
        case SKINNY_WEIGHTS_E4M3_ROW:
            st = run_type<skg::kWRow>(a, vector, stream);
            break;
        case SKINNY_WEIGHTS_E4M3_BLOCK:
            st = run_type<skg::kWBlock>(a, vector, stream);
            break;
        default:
            st = run_type<skg::kWInt8>(a, vector, stream);
            break;
        }
        if (st != SKINNY_OK)
            return st;
    }
    return SKINNY_OK;
}

}  // extern "C"

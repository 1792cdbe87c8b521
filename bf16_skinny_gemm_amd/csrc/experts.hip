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
//  - up: 8 features of both weights for one tile at a time; every block takes an equal run of
//    them.
//  - down: 16 outputs of all tokens at a time, for each of them the stages of all tiles; every
//    block takes an equal run of all that. Of its part of 16 outputs, each wave takes a run of
//    stages, so its loads go on from one expert to the next; behind a tile it adds its sums,
//    times the token's weight, to its own outputs [tokens][16] in LDS. The waves' outputs
//    are added in the order of the waves, and where several blocks share 16 outputs, their
//    parts in the order of the blocks by the one that ends last: the same bits every time.
//
// 8-bit weights are widened to bfloat16 (exactly) and multiplied by x as it is, so that only
// h and y are rounded.
//
// What it measured, cold weights, both kernels by the trace (least of 36): one token, 8 experts of
// 4096 x 1024 in bfloat16 22.9 + 13.1 us (5.6 TB/s); 5 tokens, 8 of 288 experts of that size
// with block scales 52.4 + 27.8 (5.9); 61 tokens, 6 of 64 of 2048 x 1408 in int8 61.6 + 44.5
// (5.2); 37 tokens, 2 of 16 of 4096 x 1536 in bfloat16 61.2 + 38.3 (6.0). Reads alone reach 6.8 TB/s
// on this card: HBM bounds the first kernel and the second one in bfloat16. With 8-bit weights
// and 16 rows the second one has 4.1 TB/s: a block takes in twice as many bytes of h as of the weights, in a
// ring of two stages, and its reads of h meet in the banks of LDS (0.33 of the active cycles,
// 0.25 to 0.37 in all kernels of 8-bit weights, 0.02 at most in those of bfloat16).
// Three tokens, 4 of 64 of 2048 x 768 with row scales take 12.4 + 10.4 (2.3 TB/s): an empty
// launch of the first kernel, with its plan, is 2.2 to 4 us and of the second 4, and each wave
// has 9 stages, fewer than two rings. Equal runs cost the largest calls of few tokens 3% against
// blocks that the hardware hands out, and gain all others up to half.
#include "ops_host.hpp"

#include <cstdint>

#include "experts_plan.hpp"
#include "lds_load.hpp"
#include "linear.hpp"

namespace skg {

// The weights' types.
enum { kWBf16 = SKINNY_WEIGHTS_BF16, kWRow = SKINNY_WEIGHTS_E4M3_ROW, kWBlock = SKINNY_WEIGHTS_E4M3_BLOCK,
       kWInt8 = SKINNY_WEIGHTS_INT8_ROW };
constexpr bool scaled_rows(int type) { return type == kWRow || type == kWInt8; }

// Division of x < 2^31 by a number that the host knows: (x + high word of mul x) >> shift, with
// mul = floor(2^32 (2^shift - d) / d) + 1 and 2^shift the least power >= d (Granlund and
// Montgomery). Six divisions at run time took 1.4 us of a launch.
struct Divisor {
    unsigned mul, shift;

    __device__ __forceinline__ int of(int x) const { return (int)((__umulhi(mul, (unsigned)x) + (unsigned)x) >> shift); }
};

struct ExpertArgs {
    const uint16_t *x;
    const int *ids;
    const float *weights;
    const uint8_t *w[2], *wd;   // gate and up, down
    const float *s[2], *sd;     // their scales
    const uint16_t *res;        // or null
    uint16_t *y, *h;
    unsigned *plan;             // [0] tiles, [1..3] the second kernel's Runs; from [4], of each tile:
                                // expert | pairs << 10 | first pair << 16
    u32x4 *entries;             // for each pair, by expert: token, its weight
    u32x4 *begins;              // of the second kernel's blocks: set of outputs, stage, stages in all
    unsigned *arrived;          // see there
    float *parts;
    int64_t ldx, ldr, ldy;      // elements
    int64_t up_bytes, down_bytes;  // from one expert's weight to the next
    int64_t up_scales, down_scales;
    int M, E, k, H, I;
    int act;
    Divisor by_k, by_grid, by_features, by_up, by_down;  // k, blocks, I / 8, the stages of H and of I
};

using skg_host::kMostPairs, skg_host::kMostTiles, skg_host::split_h, skg_host::h_rows;
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

template <int TYPE>
constexpr int planes() { return skg_host::planes_of(TYPE); }

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

// Rows of x (or h) in LDS: planes of [BM][128 bytes], whose 16-byte pieces are placed by the
// row (with 4 rows a plane also by its parity), as the load instructions of 8 such rows do it.
template <int BM>
__device__ __forceinline__ int x_swizzle(int row, int plane) { return BM == 4 ? (row & 3) | (plane & 1) << 2 : row & 7; }

// The lane's pieces of x that meet Fragment::v, of row `row` of the planes at `at`, the first
// of which has the number `plane`.
template <int TYPE, int BM>
__device__ __forceinline__ void read_x(const uint8_t *at, int row, int plane, int g, u32x4 (&v)[2 * planes<TYPE>()])
{
#pragma unroll
    for (int q = 0; q < 2 * planes<TYPE>(); ++q) {
        const int h = TYPE == kWBf16 ? 0 : q / 2, piece = TYPE == kWBf16 ? g + 4 * q : 2 * g + q % 2;
        v[q] = *reinterpret_cast<const u32x4 *>(at + (h * BM + row) * 128 + (piece ^ x_swizzle<BM>(row, plane + h)) * 16);
    }
}

// ---- the pairs by expert -----------------------------------------------------------

// The plan of a pass in LDS, made by every block for itself: the tiles (expert | pairs << 10 |
// first pair << 16) and each sorted pair's token.
template <bool WAVE>
struct Plan {
    unsigned tiles[WAVE ? skg_host::kWavePairs : kMostTiles];
    uint8_t tokens[WAVE ? skg_host::kWavePairs : kMostPairs];
    int count;
};
static_assert(sizeof(Plan<true>) == skg_host::plan_bytes(true) && sizeof(Plan<false>) == skg_host::plan_bytes(false), "in LDS");

// What making it takes beside: which tokens name an expert, and where its pairs start.
struct Scratch {
    unsigned named[skg_host::kMaxExperts][skg_host::kExpertsRows / 32];
    int first[skg_host::kMaxExperts], tile[skg_host::kMaxExperts];
    uint16_t ids[kMostPairs];  // 0xFFFF: none
    int twice;                 // some token names an expert twice
};

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

__device__ __forceinline__ void put_entry(const ExpertArgs &a, int at, int p)
{
    a.entries[at] = u32x4{(unsigned)a.by_k.of(p), __builtin_bit_cast(unsigned, a.weights[p]), 0, 0};
}

// Up to 64 pairs: the first wave sorts them in its lanes, by expert and then by pair.
template <int BM>
__device__ __forceinline__ void plan_wave(const ExpertArgs &a, int P, Plan<true> &plan)
{
    if (threadIdx.x >= 64)
        return;
    const int lane = threadIdx.x;
    const int named = lane < P ? a.ids[lane] : -1;
    const bool in = (unsigned)named < (unsigned)a.E;
    const int id = in ? named : 0x7FFFFFFF;
    int rank = 0, less = 0, pairs = 0;
    for (int q = 0; q < P; ++q) {
        const int o = __builtin_amdgcn_readlane(id, q);
        rank += o == id && q < lane;
        pairs += o == id;
        less += o < id;
    }
    const int pos = less + rank;
    const bool first = in && rank % BM == 0;
    // the tiles before this one: the first pairs of tiles at smaller places
    int before = 0;
    for (int q = 0; q < P; ++q) {
        const int o = __builtin_amdgcn_readlane(first ? pos : 0x7FFFFFFF, q);
        before += o < pos;
    }
    if (in) {
        plan.tokens[pos] = (uint8_t)a.by_k.of(lane);
        if (blockIdx.x == 0)
            put_entry(a, pos, lane);
    }
    if (first)
        plan.tiles[before] = (unsigned)id | (unsigned)(pairs - rank < BM ? pairs - rank : BM) << 10 | (unsigned)pos << 16;
    const int count = __popcll(__ballot(first));
    if (lane == 0)
        plan.count = count;
}

// More: a bit for each token in a mask of each expert, so that a pair's place is the number of
// bits before its own. Only where a token names an expert twice are pairs counted one by one.
template <int BM, int THREADS>
__device__ __forceinline__ void plan_block(const ExpertArgs &a, int P, Plan<false> &plan, Scratch &s)
{
    const int t = threadIdx.x;
    constexpr int WORDS = skg_host::kExpertsRows / 32;
    for (int i = t; i < a.E * WORDS; i += THREADS)
        s.named[0][i] = 0;
    if (t == 0)
        s.twice = 0;
    __syncthreads();
    for (int p = t; p < P; p += THREADS) {
        const int id = a.ids[p], m = a.by_k.of(p);
        const bool in = (unsigned)id < (unsigned)a.E;
        s.ids[p] = in ? (uint16_t)id : (uint16_t)0xFFFF;
        if (in && (atomicOr(&s.named[id][m / 32], 1u << (m % 32)) >> (m % 32) & 1))
            s.twice = 1;
    }
    __syncthreads();
    const bool twice = s.twice != 0;
    auto pairs_of = [&](int e) {
        int n = 0;
        if (!twice) {
#pragma unroll
            for (int w = 0; w < WORDS; ++w)
                n += __popc(s.named[e][w]);
        } else {
            for (int p = 0; p < P; ++p)
                n += s.ids[p] == e;
        }
        return n;
    };
    for (int e = t; e < a.E; e += THREADS)
        s.first[e] = pairs_of(e);
    __syncthreads();
    if (t < 64) {
        const int per = (a.E + 63) / 64, lo = t * per < a.E ? t * per : a.E, hi = lo + per < a.E ? lo + per : a.E;
        int np = 0, nt = 0;
        for (int e = lo; e < hi; ++e) {
            np += s.first[e];
            nt += (s.first[e] + BM - 1) / BM;
        }
        int pairs = wave_scan(np) - np, tiles = wave_scan(nt) - nt;
        if (t == 63)
            plan.count = tiles + nt;
        for (int e = lo; e < hi; ++e) {
            const int n = s.first[e];
            s.first[e] = pairs;
            s.tile[e] = tiles;
            pairs += n;
            tiles += (n + BM - 1) / BM;
        }
    }
    __syncthreads();
    for (int e = t; e < a.E; e += THREADS) {
        const int n = pairs_of(e), first = s.first[e], tile = s.tile[e];
        for (int r = 0; r < n; r += BM)
            plan.tiles[tile + r / BM] = (unsigned)e | (unsigned)(n - r < BM ? n - r : BM) << 10 | (unsigned)(first + r) << 16;
    }
    for (int p = t; p < P; p += THREADS) {
        const int e = s.ids[p], m = a.by_k.of(p);
        if (e == 0xFFFF)
            continue;
        int at = s.first[e];
        if (!twice) {
            for (int w = 0; w < m / 32; ++w)
                at += __popc(s.named[e][w]);
            at += __popc(s.named[e][m / 32] & ((1u << (m % 32)) - 1));
        } else {
            for (int q = 0; q < p; ++q)
                at += s.ids[q] == e;
        }
        plan.tokens[at] = (uint8_t)m;
        if (blockIdx.x == 0)
            put_entry(a, at, p);
    }
}

// ---- runs ------------------------------------------------------------------------------

// A line of things in `runs` runs of sizes that differ by one at most: the first `more` runs have
// per + 1 things.
struct Runs {
    unsigned runs, per, more;

    __device__ __forceinline__ unsigned start(unsigned r) const { return r * per + (r < more ? r : more); }
    __device__ __forceinline__ unsigned of(unsigned at) const
    {
        const unsigned head = more * (per + 1);
        return at < head ? at / (per + 1) : more + (at - head) / per;
    }
};

// `all` things in at most `most` = gridDim.x runs, none of them empty.
__device__ __forceinline__ Runs runs_of(unsigned all, unsigned most, const Divisor &by_most)
{
    if (all <= most)
        return Runs{all, 1, 0};
    const unsigned per = (unsigned)by_most.of((int)all);
    return Runs{most, per, all - per * most};
}

// What the second kernel's blocks take: nj sets of 16 outputs with T stages each, in one line.
// Up to kWhole stages are worth less than what blocks that share a set pay for it: then the
// runs are of whole sets.
constexpr int kWhole = 64;
constexpr int per_stage(int type) { return type == kWBf16 ? 64 : 128; }

template <int TYPE, int THREADS>
__device__ __forceinline__ void write_runs(const ExpertArgs &a, int tiles)
{
    const int nj = (a.H + 15) / 16, T = tiles * ((a.I + per_stage(TYPE) - 1) / per_stage(TYPE));
    if (T == 0)
        return;
    const int unit = T <= kWhole ? T : 1;
    const unsigned all = (unsigned)(nj * (T / unit)), runs = all < skg_host::kDownBlocks ? all : skg_host::kDownBlocks;
    const Runs share{runs, all / runs, all % runs};
    if (threadIdx.x == 0) {
        a.plan[1] = share.runs;
        a.plan[2] = share.per;
        a.plan[3] = share.more;
    }
    for (unsigned b = threadIdx.x; b < runs; b += THREADS) {
        const unsigned w0 = share.start(b) * unit, w1 = share.start(b + 1) * unit;
        a.begins[b] = u32x4{w0 / T, w0 % T, w1 - w0, 0};
    }
}

// ---- up ------------------------------------------------------------------------------

// A unit is 8 features of both weights (16 rows of an instruction: gate, then up) for one
// tile. Each block takes a run of units, tile by tile, and each of its waves an equal run of
// their stages, its loads going on from one unit to the next; only a unit that lies in several
// waves' runs waits for the tile's end, where its parts are added in the order of the waves.
// The instruction's halves meet by an exchange of lanes, so a unit needs no barrier.
// RESIDENT: the tile's rows of x stay in LDS (XROOM bytes of it), which leaves the ring to the
// weights: what a unit streams is bound by the bytes in flight. Otherwise a stage holds its
// part of them too.
// WAVE: the pairs fit one wave.
template <int TYPE, int BM, int RING, int WAVES, bool WAVE, bool RESIDENT, int XROOM>
__global__ __launch_bounds__(WAVES * 64) void experts_up_kernel(ExpertArgs a)
{
    constexpr bool BLOCK = TYPE == kWBlock;
    constexpr int PLANES = planes<TYPE>();
    constexpr int TM = (BM + 15) / 16, XR = (BM + 7) / 8;
    constexpr int XAT = 16 * 128, XPLANE = BM * 128, SAT = XAT + (RESIDENT ? 0 : PLANES * XPLANE);
    constexpr int STAGE = skg_host::up_stage(TYPE, BM, RESIDENT);
    constexpr int LOADS = 2 + (RESIDENT ? 0 : PLANES * BM / 8) + (TYPE == kWBf16 ? 0 : 2);
    constexpr int RINGS = WAVES * RING * STAGE, ROOM = RINGS + (RESIDENT ? XROOM : 0);
    constexpr int SMEM = !WAVE && (int)sizeof(Scratch) > ROOM ? (int)sizeof(Scratch) : ROOM;
    static_assert((BM == 4 || BM % 8 == 0) && BM <= 32 && RING * LOADS < 64 && RING * STAGE >= TM * 1024, "tile");
    static_assert(RESIDENT || BM >= 8, "a stage's load of x takes 8 rows");
    __shared__ __attribute__((aligned(16))) uint8_t smem[SMEM];
    __shared__ Plan<WAVE> plan;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int P = a.M * a.k;
    if constexpr (WAVE)
        plan_wave<BM>(a, P, plan);
    else
        plan_block<BM, WAVES * 64>(a, P, plan, *reinterpret_cast<Scratch *>(smem));
    __syncthreads();
    const int tiles = __builtin_amdgcn_readfirstlane(plan.count);
    if (blockIdx.x == 0) {  // for the second kernel
        for (int i = threadIdx.x; i < skg_host::kDownBlocks; i += WAVES * 64)
            a.arrived[i] = 0;
        for (int i = threadIdx.x; i < tiles; i += WAVES * 64)
            a.plan[4 + i] = plan.tiles[i];
        if (threadIdx.x == 0)
            a.plan[0] = (unsigned)tiles;
        write_runs<TYPE, WAVES * 64>(a, tiles);
    }

    const int KB = TYPE == kWBf16 ? a.H * 2 : a.H;
    const int stages = (KB + 127) / 128;
    const int nf = (a.I + 7) / 8, hb = (a.H + 127) / 128;
    const Runs share = runs_of((unsigned)(tiles * nf), gridDim.x, a.by_grid);
    if (blockIdx.x >= share.runs)
        return;
    const int u0 = (int)share.start(blockIdx.x), u1 = (int)share.start(blockIdx.x + 1);
    const unsigned ldx = (unsigned)a.ldx * 2u, XB = (unsigned)a.H * 2u;
    const u32x4 xr = rsrc_words(a.x, (unsigned)(a.M - 1) * ldx + XB);
    uint8_t *ring = smem + wave * RING * STAGE;
    const unsigned smem0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)smem;
    const unsigned lds0 = smem0 + wave * RING * STAGE;
    const int lrow = lane >> 3;
    const unsigned piece = (unsigned)((lane & 7) ^ lrow) * 16u;

    for (int u = u0; u < u1;) {
        const int t = a.by_features.of(u), f0 = u - t * nf;
        const int nu = u1 - u < nf - f0 ? u1 - u : nf - f0;  // units of this tile
        u += nu;
        const unsigned word = __builtin_amdgcn_readfirstlane((int)plan.tiles[t]);
        const int e = (int)(word & 1023u), pairs = (int)(word >> 10 & 63u), first = (int)(word >> 16);
        const unsigned total = (unsigned)(nu * stages);
        auto start = [&](int w) { return (int)(total / WAVES * w + total % WAVES * w / WAVES); };
        const int from = start(wave), to = start(wave + 1), n = to - from;  // stages of this wave

        // the rows of x that this lane loads pieces of
        unsigned xat[XR];
#pragma unroll
        for (int c = 0; c < XR; ++c) {
            const int r = BM == 4 ? lrow & 3 : c * 8 + lrow;
            xat[c] = r < pairs ? (unsigned)plan.tokens[first + r] * ldx : kOutOfRange;
        }
        if constexpr (RESIDENT) {
            constexpr int EACH = BM == 4 ? 2 : 1;  // planes of a load
            const int all = stages * PLANES;  // with zeros behind x's end, where the weights have them too
            for (int p = wave * EACH; p < all; p += WAVES * EACH) {
                const unsigned b = (unsigned)(p + (BM == 4 ? lrow >> 2 : 0)) * 128u + piece;
#pragma unroll
                for (int c = 0; c < XR; ++c)
                    load_to_lds(xr, b < XB && xat[c] != kOutOfRange ? xat[c] + b : kOutOfRange,
                                smem0 + RINGS + (unsigned)(p * XPLANE + c * 1024));
            }
        }

        const int skipped = a.by_up.of(from);  // units before the run
        int iu = f0 + skipped, is = from - skipped * stages;  // what is loaded next
        u32x4 wr[2], sr[2];
        auto enter_unit = [&] {
            const int n0 = iu * 8, vn = a.I - n0 < 8 ? a.I - n0 : 8;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                wr[q] = rsrc_words(a.w[q] + e * a.up_bytes + (int64_t)n0 * KB, (unsigned)vn * (unsigned)KB);
                if constexpr (BLOCK)
                    sr[q] = rsrc_words(a.s[q] + e * a.up_scales + (int64_t)(n0 / 128) * hb, (unsigned)hb * 4u);
                else if constexpr (scaled_rows(TYPE))
                    sr[q] = rsrc_words(a.s[q] + e * a.up_scales + n0, (unsigned)vn * 4u);
            }
        };
        auto issue = [&](int slot) {
            const unsigned k = (unsigned)is * 128u + piece;
            const unsigned lds = lds0 + (unsigned)(slot * STAGE);
            const unsigned at = k < (unsigned)KB ? (unsigned)lrow * (unsigned)KB + k : kOutOfRange;
            load_to_lds<true>(wr[0], at, lds);
            load_to_lds<true>(wr[1], at, lds + 1024u);
            if constexpr (!RESIDENT) {
#pragma unroll
                for (int h = 0; h < PLANES; ++h) {
                    const unsigned b = (unsigned)(is * PLANES + h) * 128u + piece;
#pragma unroll
                    for (int c = 0; c < XR; ++c)
                        load_to_lds(xr, b < XB && xat[c] != kOutOfRange ? xat[c] + b : kOutOfRange,
                                    lds + XAT + (unsigned)(h * XPLANE + c * 1024));
                }
            }
            if constexpr (TYPE != kWBf16) {  // 8 floats of each weight: its features' scales, or the block's
                const unsigned f = BLOCK ? (unsigned)is * 4u : (unsigned)(lane & 7) * 4u;
                if (lane < 8) {  // lane i writes at lds + 4 i, the others nothing
                    load4_to_lds(sr[0], f, lds + SAT);
                    load4_to_lds(sr[1], f, lds + SAT + 32u);
                }
            }
            if (++is == stages) {
                is = 0;
                if (++iu < f0 + nu)
                    enter_unit();
            }
        };

        f32x4 acc[TM], head[TM], scale = {1.0f, 1.0f, 1.0f, 1.0f};  // head: see below
        auto clear = [&] {
#pragma unroll
            for (int j = 0; j < TM; ++j)
                acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        };
        clear();
#pragma unroll
        for (int j = 0; j < TM; ++j)
            head[j] = acc[j];
        // h of a whole unit: lanes 0..31 hold the gate's sums, 32..63 the up projection's
        auto finish = [&](int unit) {
            const int f = unit * 8 + (g & 1) * 4;
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                f32x4 z = acc[j], o;
                if constexpr (scaled_rows(TYPE))
                    z *= scale;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    o[q] = __shfl_xor(z[q], 32, 64);
                const int r = j * 16 + i16;
                if (lane < 32 && r < pairs && f < a.I) {  // I is a multiple of 8: all four are there
                    z = activate4(z, a.act) * o;
                    const u32x2 hi = {pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3])};
                    uint16_t *at = a.h + (int64_t)(first + r) * a.I * (split_h(BM) ? 2 : 1) + f;
                    *reinterpret_cast<u32x2 *>(at) = hi;
                    if constexpr (split_h(BM)) {
                        z -= widen4(hi);
                        *reinterpret_cast<u32x2 *>(at + a.I) = u32x2{pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3])};
                    }
                }
            }
        };

        // the unit and stage that are multiplied next, and whether its sums began in this wave
        int cu = iu, cs = is;
        bool whole = cs == 0;
        if (n > 0) {
            enter_unit();
#pragma unroll
            for (int d = 0; d < RING; ++d)
                if (d < n)
                    issue(d);
        }
        if constexpr (RESIDENT) {  // x has landed, here and in the other waves
            if (n >= RING)
                stage_wait<RING * LOADS>();
            else
                stage_wait<0>();
            __syncthreads();
        }
        int slot = 0;
        for (int s = 0; s < n; ++s) {
            if (s + RING <= n)
                stage_wait<(RING - 1) * LOADS>();
            else
                stage_wait<0>();
            const uint8_t *st = ring + slot * STAGE;
            Fragment<TYPE> af;
            u32x4 bf[TM][2 * PLANES];
            float sc = 1.0f;
            af.read(st + i16 * 128, g, i16 & 7);
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int r = BM <= 8 ? i16 % BM : j * 16 + i16;
                if constexpr (RESIDENT)
                    read_x<TYPE, BM>(smem + RINGS + cs * PLANES * XPLANE, r, cs * PLANES, g, bf[j]);
                else
                    read_x<TYPE, BM>(st + XAT, r, 0, g, bf[j]);
            }
            if constexpr (BLOCK)
                sc = *reinterpret_cast<const float *>(st + SAT + (g >> 1) * 32);
            else if constexpr (scaled_rows(TYPE))
                scale = *reinterpret_cast<const f32x4 *>(st + SAT + g * 16);
            lds_read_wait();  // the stage is in registers: its slot may be written again
            if (s + RING < n)
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
                    for (int q = 0; q < 4; ++q)
                        acc[j][q] = __builtin_fmaf(p[q], sc, acc[j][q]);
                } else {
                    acc[j] = p;
                }
            }
            if (++cs == stages) {
                cs = 0;
                if (whole) {
                    finish(cu);
                } else {  // the end of a unit that an earlier wave began: its ring is still
                          // being written, so the sums wait in registers
#pragma unroll
                    for (int j = 0; j < TM; ++j)
                        head[j] = acc[j];
                }
                whole = true;
                clear();
                ++cu;
            }
        }

        // Units in several runs: a wave whose run began inside one leaves that part of its
        // sums, and the wave that began it adds them up.
        const bool inside = skipped * stages != from;  // the run began inside a unit
        const bool through = inside && !whole;   // and did not reach its end
        if (inside)
#pragma unroll
            for (int j = 0; j < TM; ++j)
                *reinterpret_cast<f32x4 *>(ring + (j * 64 + lane) * 16) = through ? acc[j] : head[j];
        __syncthreads();
        if (n > 0 && whole && cs != 0) {
            const int unit_end = to - cs + stages;
            for (int w = wave + 1; w < WAVES; ++w) {
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    acc[j] += *reinterpret_cast<const f32x4 *>(smem + w * RING * STAGE + (j * 64 + lane) * 16);
                if (start(w + 1) >= unit_end)
                    break;
            }
            finish(cu);
        }
        if (u < u1)
            __syncthreads();  // the next tile is written over x and the parts
    }
}

// ---- down ----------------------------------------------------------------------------

// s_waitcnt operand: vmcnt 0, the other counters left at their largest.
constexpr int kWaitStores = 0x0F70;

// MC: tokens that the block has room for.
template <int TYPE, int BM, int RING, int WAVES, int MC>
__global__ __launch_bounds__(WAVES * 64) void experts_down_kernel(ExpertArgs a, int most_tiles)
{
    constexpr bool BLOCK = TYPE == kWBlock;
    constexpr int PLANES = planes<TYPE>();
    constexpr int TM = (BM + 15) / 16;
    constexpr bool SPLIT = split_h(BM);
    constexpr int HR = h_rows(BM);  // rows of h in LDS: split, those of the first values, then the others
    constexpr int XAT = 2048, XPLANE = HR * 128, EAT = XAT + PLANES * XPLANE, SAT = EAT + BM * 16;
    constexpr int STAGE = skg_host::down_stage(TYPE, BM);
    constexpr int HLOADS = PLANES * HR / 8;  // 8 rows each
    constexpr int LOADS = 2 + HLOADS + 1 + (TYPE == kWBf16 ? 0 : 1);
    constexpr int OUTS = MC * 16;  // floats of a wave
    static_assert((BM == 4 || BM % 8 == 0) && BM <= 32 && (RING - 1) * LOADS < 64, "tile");
    __shared__ __attribute__((aligned(16))) uint8_t smem[WAVES * RING * STAGE];
    __shared__ __attribute__((aligned(16))) float outs[WAVES * OUTS];
    __shared__ unsigned tiles[kMostTiles];
    __shared__ unsigned earlier;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    // one round trip for the plan: scalar loads would come behind the tiles'
    int zero = 0;
    asm volatile("" : "+v"(zero));
    const u32x4 head = *reinterpret_cast<const u32x4 *>(a.plan + zero), run = a.begins[(int)blockIdx.x + zero];
    for (int i = threadIdx.x; i < most_tiles; i += WAVES * 64)
        tiles[i] = a.plan[4 + i];
    const int nt = __builtin_amdgcn_readfirstlane((int)head[0]);
    const Runs share{(unsigned)__builtin_amdgcn_readfirstlane((int)head[1]), (unsigned)__builtin_amdgcn_readfirstlane((int)head[2]),
                     (unsigned)__builtin_amdgcn_readfirstlane((int)head[3])};
    float *out = outs + wave * OUTS;

    const int KB = TYPE == kWBf16 ? a.I * 2 : a.I;
    const unsigned XB = (unsigned)a.I * 2u;
    const int stages = (KB + 127) / 128, ib = (a.I + 127) / 128;
    const uint8_t *ring = smem + wave * RING * STAGE;
    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)smem + wave * RING * STAGE;
    const int lrow = lane >> 3;
    const unsigned piece = (unsigned)((lane & 7) ^ lrow) * 16u;

    // four outputs of a token, from their sum
    auto store = [&](int o, int n0, f32x4 v) {
        const int m = o / 4, n = n0 + o % 4 * 4;
        if (n >= a.H)
            return;  // H is a multiple of 8: all four are there or none
        if (a.res)
            v += widen4(*reinterpret_cast<const u32x2_any *>(a.res + m * a.ldr + n));
        *reinterpret_cast<u32x2_any *>(a.y + m * a.ldy + n) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    };

    const int nj = (a.H + 15) / 16, T = nt * stages;
    if (T == 0) {  // no pair names an expert
        for (int j = blockIdx.x; j < nj; j += gridDim.x)
            for (int o = threadIdx.x; o < a.M * 4; o += WAVES * 64)
                store(o, j * 16, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
        return;
    }
    if (blockIdx.x >= share.runs)
        return;
    int j = __builtin_amdgcn_readfirstlane((int)run[0]), begin = __builtin_amdgcn_readfirstlane((int)run[1]);
    int left = __builtin_amdgcn_readfirstlane((int)run[2]);
    for (; left > 0; ++j, begin = 0) {
        const int len = left < T - begin ? left : T - begin;
        left -= len;
        const int n0 = j * 16, vn = a.H - n0 < 16 ? a.H - n0 : 16;
        const int from = begin + len / WAVES * wave + len % WAVES * wave / WAVES;
        const int to = begin + len / WAVES * (wave + 1) + len % WAVES * (wave + 1) / WAVES;
        __syncthreads();  // tiles are there; the outputs before have been read
        for (int i = lane; i < a.M * 4; i += 64)
            reinterpret_cast<f32x4 *>(out)[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        int it = a.by_down.of(from), is = from - it * stages;  // the tile and stage that are loaded next
        u32x4 wr, hr, er, sr;
        auto enter = [&] {
            const unsigned v = __builtin_amdgcn_readfirstlane((int)tiles[it]);
            const int e = (int)(v & 1023u), pairs = (int)(v >> 10 & 63u), first = (int)(v >> 16);
            wr = rsrc_words(a.wd + e * a.down_bytes + (int64_t)n0 * KB, (unsigned)vn * (unsigned)KB);
            hr = rsrc_words(a.h + (int64_t)first * a.I * (SPLIT ? 2 : 1), (unsigned)pairs * XB * (SPLIT ? 2 : 1));
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
            for (int c = 0; c < 2; ++c)
                load_to_lds<true>(wr, k < (unsigned)KB ? (unsigned)(c * 8 + lrow) * (unsigned)KB + k : kOutOfRange,
                                  lds + (unsigned)c * 1024u);
            // rows beyond the tile's lie beyond the resource
#pragma unroll
            for (int h = 0; h < PLANES; ++h) {
                const unsigned b = (unsigned)(is * PLANES + h) * 128u + piece;
#pragma unroll
                for (int c = 0; c < HR / 8; ++c) {
                    const int r = c * 8 + lrow;  // of LDS
                    const unsigned row = SPLIT ? (unsigned)(r % BM * 2 + r / BM) : (unsigned)r;
                    load_to_lds(hr, b < XB ? row * XB + b : kOutOfRange, lds + XAT + (unsigned)(h * XPLANE + c * 1024));
                }
            }
            if (lane < BM)  // lane i writes at lds + 16 i (4 i), the others nothing
                load_to_lds(er, (unsigned)lane * 16u, lds + EAT);
            if constexpr (TYPE != kWBf16)
                if (lane < 16)
                    load4_to_lds(sr, BLOCK ? (unsigned)is * 4u : (unsigned)lane * 4u, lds + SAT);
            if (++is == stages) {
                is = 0;
                if (++it < nt)
                    enter();
            }
        };

        f32x4 acc[TM];
        auto clear = [&] {
#pragma unroll
            for (int i = 0; i < TM; ++i)
                acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        };
        clear();
        int ct = it, cs = is;  // the tile and stage that are multiplied next
        if (from < to) {
            enter();
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
            af.read(st + i16 * 128, g, i16 & 7);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int r = SPLIT ? i16 % BM : i * 16 + i16;
                read_x<TYPE, HR>(st + XAT, SPLIT ? r + i16 / 8 * BM : r, 0, g, bf[i]);
                entry[i] = *reinterpret_cast<const u32x4 *>(st + EAT + r * 16);
            }
            if constexpr (BLOCK)
                sc = *reinterpret_cast<const float *>(st + SAT);
            else if constexpr (scaled_rows(TYPE))
                rows = *reinterpret_cast<const f32x4 *>(st + SAT + g * 16);
            lds_read_wait();  // the stage is in registers: its slot may be written again
            if (s + RING < to)
                issue(slot);
            slot = slot + 1 == RING ? 0 : slot + 1;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                f32x4 p = BLOCK ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[i];
#pragma unroll
                for (int q = 0; q < 2 * PLANES; ++q)
                    p = mfma_bf16(af.v[q], bf[i][q], p);
                if constexpr (BLOCK) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][e] = __builtin_fmaf(p[e], sc, acc[i][e]);
                } else {
                    acc[i] = p;
                }
            }
            if (last) {
                const int pairs = (int)(__builtin_amdgcn_readfirstlane((int)tiles[ct]) >> 10 & 63);
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    if constexpr (SPLIT)  // both parts of h, in the columns up to 7
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // where the first part's sum is infinite or NaN, it is all: what the second
                            // one has of an infinite weight or h is NaN, or has another sign
                            const float rest = __shfl_xor(acc[i][e], 8, 64);
                            acc[i][e] += __builtin_fabsf(acc[i][e]) < __builtin_inff() ? rest : 0.0f;
                        }
                    const bool live = i * 16 + i16 < pairs;
                    const int token = (int)entry[i][0];
                    const unsigned weight = entry[i][1];  // a bit_cast of the element itself takes the first one
                    f32x4 v = acc[i] * __builtin_bit_cast(float, weight);
                    if constexpr (scaled_rows(TYPE))
                        v *= rows;
                    f32x4 *at = reinterpret_cast<f32x4 *>(out + token * 16 + g * 4);
                    // the pairs of an expert are in the order of their tokens: one that names it
                    // twice has two pairs side by side, which must not add at the same time
                    const int beside = __shfl_up(token, 1, 16);
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    if (!__ballot(live && i16 > 0 && token == beside)) {
                        if (live)
                            *at += v;
                    } else {
                        for (int c = 0; c < 16; ++c) {
                            if (live && i16 == c)
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
        auto sum = [&](int o) {
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < WAVES; ++k)
                v += *reinterpret_cast<const f32x4 *>(outs + k * OUTS + o * 4);
            return v;
        };
        if (len == T) {
            for (int o = threadIdx.x; o < a.M * 4; o += WAVES * 64)
                store(o, n0, sum(o));
        } else {
            // A block shares its first and its last 16 outputs at most. The parts go past the
            // caches of the XCDs (agent scope), a block counts itself behind its stores, and the
            // one that finds all others counted adds the parts up.
            auto part = [&](int b) { return a.parts + (2 * b + ((int)a.begins[b][0] != j)) * (a.M * 16); };
            float *mine = part(blockIdx.x);
            for (int o = threadIdx.x; o < a.M * 4; o += WAVES * 64) {
                const f32x4 v = sum(o);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    __hip_atomic_store(mine + o * 4 + e, v[e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
            __builtin_amdgcn_s_waitcnt(kWaitStores);
            __syncthreads();
            // the blocks with the first and the last stage of these outputs
            const int b0 = (int)share.of(j * T), b1 = (int)share.of(j * T + T - 1);
            if (threadIdx.x == 0)
                earlier = __hip_atomic_fetch_add(a.arrived + b0, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            if (earlier == (unsigned)(b1 - b0))
                for (int o = threadIdx.x; o < a.M * 4; o += WAVES * 64) {
                    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
                    for (int b = b0; b <= b1; ++b) {
                        const float *p = part(b) + o * 4;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] += __hip_atomic_load(p + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    }
                    store(o, n0, v);
                }
        }
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

// One wave per pair and feature: h of pair p is row p, in float32.
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
            reinterpret_cast<float *>(a.h)[o] = z[0] * v[1];
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
                const float t = reinterpret_cast<const float *>(a.h)[(int64_t)p * a.I + i] * weight_at<TYPE>(w, (int64_t)n * a.I + i);
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

template <int TYPE, int BM, bool WAVE, int RING>
const void *up_resident_fn()
{
    constexpr UpPlan U = up_resident(TYPE, BM, WAVE, RING);
    return (const void *)&skg::experts_up_kernel<TYPE, BM, U.ring, U.waves, WAVE, true, U.room>;
}

// The first kernel of a plan that up_plan() made for tiles of BM rows.
template <int TYPE, int BM, bool WAVE>
const void *up_fn(const UpPlan &u)
{
    if constexpr (resident_offered(TYPE, BM, WAVE))
        if (u.room)
            return u.ring == kResidentRings[0]   ? up_resident_fn<TYPE, BM, WAVE, kResidentRings[0]>()
                   : u.ring == kResidentRings[1] ? up_resident_fn<TYPE, BM, WAVE, kResidentRings[1]>()
                                                 : up_resident_fn<TYPE, BM, WAVE, kResidentRings[2]>();
    constexpr UpPlan U = up_streamed(TYPE, BM, WAVE);
    return (const void *)&skg::experts_up_kernel<TYPE, U.rows, U.ring, U.waves, WAVE, false, 0>;
}

template <int TYPE, int BM, int TOKENS>
const void *down_fn_of()
{
    constexpr DownPlan D = down_of(TYPE, BM, TOKENS);
    return (const void *)&skg::experts_down_kernel<TYPE, BM, D.ring, D.waves, TOKENS>;
}

template <int TYPE, int BM>
const void *down_fn(const DownPlan &d)
{
    // tiles of 32 rows are for more than 16 tokens
    return d.tokens == 16   ? down_fn_of<TYPE, BM == 32 ? 16 : BM, 16>()
           : d.tokens == 64 ? down_fn_of<TYPE, BM, 64>()
                            : down_fn_of<TYPE, BM, 128>();
}

skg::Divisor divisor(unsigned d)
{
    unsigned shift = 0;
    while ((UINT64_C(1) << shift) < d)
        ++shift;
    return skg::Divisor{(unsigned)((((UINT64_C(1) << shift) - d) << 32) / d + 1), shift};
}

// The element-wise kernels.
template <int TYPE>
int run_any(skg::ExpertArgs &a, hipStream_t stream)
{
    void *args[] = {&a};
    const int64_t up = ((int64_t)a.M * a.k * a.I + 3) / 4, down = ((int64_t)a.M * a.H + 3) / 4, most = 1 << 20;
    const int st = ops_launch((const void *)&skg::experts_up_any_kernel<TYPE>, dim3((unsigned)(up < most ? up : most)), 256,
                              args, stream);
    return st != SKINNY_OK ? st
                           : ops_launch((const void *)&skg::experts_down_any_kernel<TYPE>,
                                        dim3((unsigned)(down < most ? down : most)), 256, args, stream);
}

// Both kernels with tiles of BM rows.
template <int TYPE, int BM>
int run_rows(skg::ExpertArgs &a, int cus, hipStream_t stream)
{
    const int P = a.M * a.k;
    const bool wave = P <= kWavePairs;
    const UpPlan up = up_plan(TYPE, BM, wave, a.H);
    int most = a.E + P / up.rows;  // tiles, at most
    most = P < most ? P : most;
    // the kernels count units and stages in 32 bits
    const int64_t features = ((int64_t)a.I + 7) / 8, sets = ((int64_t)a.H + 15) / 16, per = skg::per_stage(TYPE);
    const int64_t up_stages = (a.H + per - 1) / per, down_stages = (a.I + per - 1) / per;
    if (most * features > INT32_MAX || features * up_stages > INT32_MAX || most * down_stages * sets > INT32_MAX)
        return run_any<TYPE>(a, stream);
    a.by_grid = divisor((unsigned)cus);
    a.by_features = divisor((unsigned)features);
    a.by_up = divisor((unsigned)up_stages);
    a.by_down = divisor((unsigned)down_stages);
    void *args[] = {&a, &most};
    const int st = ops_launch(wave ? up_fn<TYPE, BM, true>(up) : up_fn<TYPE, BM, false>(up), dim3((unsigned)cus), up.waves * 64,
                              args, stream);
    if (st != SKINNY_OK)
        return st;
    const DownPlan down = down_of(TYPE, up.rows, tokens_room(a.M));
    return ops_launch(up.rows == BM ? down_fn<TYPE, BM>(down) : down_fn<TYPE, 8>(down), dim3((unsigned)kDownBlocks),
                      down.waves * 64, args, stream);
}

template <int TYPE>
int run_type(const skg::ExpertArgs &a, bool vector, int cus, hipStream_t stream)
{
    skg::ExpertArgs args = a;
    if (!vector)
        return run_any<TYPE>(args, stream);
    const int rows = tile_rows(TYPE, a.M, a.E, a.k, a.H);
    return rows == 4    ? run_rows<TYPE, 4>(args, cus, stream)
           : rows == 8  ? run_rows<TYPE, 8>(args, cus, stream)
           : rows == 16 ? run_rows<TYPE, 16>(args, cus, stream)
                        : run_rows<TYPE, 32>(args, cus, stream);
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
    a.begins = reinterpret_cast<skg::u32x4 *>(ws + space.begins);
    a.arrived = reinterpret_cast<unsigned *>(ws + space.arrived);
    a.parts = reinterpret_cast<float *>(ws + space.parts);
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
    a.by_k = divisor((unsigned)e->k);
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
            st = run_type<skg::kWBf16>(a, vector, cus, stream);
            break;
        case SKINNY_WEIGHTS_E4M3_ROW:
            st = run_type<skg::kWRow>(a, vector, cus, stream);
            break;
        case SKINNY_WEIGHTS_E4M3_BLOCK:
            st = run_type<skg::kWBlock>(a, vector, cus, stream);
            break;
        default:
            st = run_type<skg::kWInt8>(a, vector, cus, stream);
            break;
        }
        if (st != SKINNY_OK)
            return st;
    }
    return SKINNY_OK;
}

}  // extern "C"

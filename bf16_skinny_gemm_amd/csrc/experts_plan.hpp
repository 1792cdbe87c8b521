// Which kernels a call of skinny_experts takes (include/skinny_moe.h), and the sizes in LDS that
// decide it: plain C++ with no HIP code, so that a test on the CPU asks exactly these.
#pragma once

#include <cmath>
#include <cstdint>

#include "validate_moe.hpp"

namespace skg_host {

constexpr int kMostPairs = kExpertsRows * kMaxExpertsK;  // 4096: 12 bits and one
constexpr int kMostTiles = kMaxExperts + kMostPairs / 4;

// x (or h) of a stage lies in this many planes of [rows][128 bytes], a column of weights beside
// the same column of x: the 16 bytes of an 8-bit weight beside two pieces of 16 bytes.
constexpr int planes_of(int type) { return type == SKINNY_WEIGHTS_BF16 ? 1 : 2; }

// Tiles of up to 8 rows leave half of the instruction's 16 columns free. There h is held as two
// bfloat16 values, the rounded one and what it leaves, in the columns 0..7 and 8..15: 16 bits of
// it for no product more, where one rounding of it would be as large an error as that of y. It
// costs nothing with 4 rows, and 6 us of 96 with 8 (37 tokens, 16 experts of 4096 x 1536,
// bfloat16), where a compute unit takes in as much of h as of the weights. Tiles of more rows
// hold h in one bfloat16 value, as a projection of its own would store it, and their outputs are
// off by 0.0024 of the result's norm where 0.0017 is y's own rounding: a choice for the speed of
// batches. Two values there double the second kernel's products and its intake of h; both
// kernels, in microseconds, with one and with two: 61 tokens, 6 of 64 of 2048 x 1408, int8 113 and
// 134, bfloat16 183 and 206; 100 tokens, 8 of 64 of 4096 x 1024, int8 226 and 266; 128 tokens, 12 of
// 64 of that size, int8 300 and 423, bfloat16 409 and 492.
constexpr bool split_h(int rows) { return rows <= 8; }
constexpr int h_rows(int rows) { return split_h(rows) ? 2 * rows : rows; }

// Bytes of a stage: weights, x or h, and what belongs to them.
constexpr int up_stage(int type, int rows, bool resident)
{
    return 2048 + (resident ? 0 : planes_of(type) * rows * 128) + (type == SKINNY_WEIGHTS_BF16 ? 0 : 64);
}
constexpr int down_stage(int type, int rows)
{
    return 2048 + planes_of(type) * h_rows(rows) * 128 + rows * 16 + (type == SKINNY_WEIGHTS_BF16 ? 0 : 64);
}

constexpr int kLds = 163840;

// Of the plan of a pass, for pairs of one wave (up to 64) or more: a word for each tile, a byte
// for each pair, and the number of tiles.
constexpr int kWavePairs = 64;
constexpr int plan_bytes(bool wave) { return wave ? 5 * kWavePairs + 4 : 4 * kMostTiles + kMostPairs + 4; }

// As many stages as fit, 6 at most.
constexpr int ring_of(int bytes, int waves, int stage) { return bytes / (waves * stage) < 6 ? bytes / (waves * stage) : 6; }

// A first kernel: its tiles' rows, waves, stages of a wave, and the bytes of a tile's x in LDS (0:
// x is streamed with the weights).
struct UpPlan {
    int rows, waves, ring, room;
};

constexpr UpPlan up_resident(int type, int rows, bool wave, int ring)
{
    return UpPlan{rows, 8, ring, (kLds - plan_bytes(wave) - 64 - ring * 8 * up_stage(type, rows, true)) / 1024 * 1024};
}

constexpr UpPlan up_streamed(int type, int rows, bool wave)
{
    const int b = rows == 4 ? 8 : rows, waves = rows == 32 && type != SKINNY_WEIGHTS_BF16 ? 4 : 8;
    return UpPlan{b, waves, ring_of(kLds - plan_bytes(wave) - 64, waves, up_stage(type, b, false)), 0};
}

constexpr int kResidentRings[] = {6, 4, 3};

// 8-bit weights, 32 rows and 64 pairs: x is wide
constexpr bool resident_offered(int type, int rows, bool wave) { return rows < 32 || type == SKINNY_WEIGHTS_BF16 || !wave; }

// The first kernel for tiles of so many rows and H inputs.
inline UpPlan up_plan(int type, int rows, bool wave, int64_t H)
{
    if (resident_offered(type, rows, wave))
        for (int ring : kResidentRings) {
            const UpPlan u = up_resident(type, rows, wave, ring);
            if ((2 * H + 255) / 256 * 256 * rows <= u.room)
                return u;
        }
    return up_streamed(type, rows, wave);
}

// A second kernel, and the tokens that it has room for.
struct DownPlan {
    int rows, waves, ring, tokens;
};

constexpr DownPlan down_of(int type, int rows, int tokens)
{
    const int waves = tokens == 128 || (rows == 32 && type != SKINNY_WEIGHTS_BF16) ? 4 : 8;
    return DownPlan{rows, waves, ring_of(kLds - 4 * kMostTiles - 16 - waves * tokens * 64, waves, down_stage(type, rows)), tokens};
}

// That behind a first kernel of so many rows; tiles of 32 are for more than 16 tokens.
constexpr int tokens_room(int M) { return M <= 16 ? 16 : M <= 64 ? 64 : 128; }

// Rows of a tile, for a pass of M tokens. The ids are on the device, so those that name no expert
// count as pairs here.
inline int tile_rows(int type, int M, int E, int k, int H)
{
    const int P = M * k;
    // pairs of an expert that has any, were the pairs spread evenly
    const double some = E * (1.0 - std::pow(1.0 - 1.0 / E, P)), even = P / some;
    // A tile's rows of x (or h) cost LDS and loads whether there are pairs for them or not, and an
    // expert with more pairs than rows is read again, from the caches at best. With narrow x,
    // 16 rows of it stay in LDS. Both kernels, in microseconds, with 8 and with 16 rows:
    // 61 tokens, 64 experts of 2048 x 1408, int8 (5.7 pairs each) 129 and 107; 32 tokens, 64 of
    // 4096 x 1024, e4m3 (2.4) 116 and 124, with 4 rows 121, and (4.1) 147 and 150, with 4 rows 185.
    // With 16 and with 32: 100 tokens, 64 of 4096 x 1024,
    // int8 (12.5) 221 and 267; 128 tokens, 8 of 4096 x 1536, int8 (32) 96 and 79, 8 of
    // 2048 x 1024 (64) 59 and 62; 128 tokens, 64 of 4096 x 1024, bfloat16 (20) 539 and 365.
    const bool bytes = type != SKINNY_WEIGHTS_BF16, narrow = H <= 2560;
    const double eight = narrow ? 4.5 : 7.0, sixteen = bytes ? (narrow ? 64.0 : 20.0) : narrow ? 14.0 : 11.0;
    return even <= 2.0 ? 4 : even <= eight ? 8 : even <= sixteen || M <= 16 ? 16 : 32;
}

}  // namespace skg_host

// Host-side argument checks of include/skinny_moe.h: plain C++ with no HIP code, like
// validate_ops.hpp, so that a sanitizer build on the CPU runs exactly these.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "skinny_moe.h"
#include "validate_ops.hpp"

namespace skg_host {

constexpr int32_t kMaxExperts = 1024, kMaxRouteK = 64, kMaxRouteGroups = 64, kMaxExpertsK = 32;

// Contiguous: one row.
inline Block flat(const void *p, uint64_t bytes) { return Block{p, p ? 1u : 0u, bytes, bytes}; }

// The extent of a block of any length is representable.
inline bool reaches(const Block &b)
{
    if (!b.p || !b.rows || !b.width)
        return true;
    if (b.rows == 1)
        return b.width <= kMaxExtent && reinterpret_cast<uintptr_t>(b.p) <= UINTPTR_MAX - b.width;
    return block_ok(b);
}

inline int validate_route(const skinny_route_t *a)
{
    if (!a || a->M < 0 || a->E < 1 || a->E > kMaxExperts || a->k < 1 || a->k > kMaxRouteK)
        return SKINNY_ERR_INVALID_ARG;
    if (a->groups < 1 || a->groups > kMaxRouteGroups || a->E % a->groups || a->kept < 1 || a->kept > a->groups ||
        a->k > a->kept * (a->E / a->groups))
        return SKINNY_ERR_INVALID_ARG;
    if (a->score < SKINNY_SCORE_SOFTMAX || a->score > SKINNY_SCORE_SIGMOID || a->renormalize < 0 || a->renormalize > 1 ||
        !std::isfinite(a->scale))
        return SKINNY_ERR_INVALID_ARG;
    if (a->M == 0)
        return SKINNY_OK;
    if (!a->logits || !a->ids || !a->weights || !ld_ok(a->ldl, a->E))
        return SKINNY_ERR_INVALID_ARG;
    if (!aligned(a->logits, 4) || !aligned(a->bias, 4) || !aligned(a->ids, 4) || !aligned(a->weights, 4))
        return SKINNY_ERR_INVALID_ARG;
    const uint64_t M = (uint64_t)a->M, E = (uint64_t)a->E, out = 4 * M * (uint64_t)a->k;
    const Block l{a->logits, M, 4 * E, 4 * (uint64_t)a->ldl}, b = flat(a->bias, 4 * E), i = flat(a->ids, out),
                w = flat(a->weights, out);
    for (const Block *p : {&l, &b, &i, &w})
        if (!reaches(*p))
            return SKINNY_ERR_INVALID_ARG;
    if (!disjoint(i, l) || !disjoint(i, b) || !disjoint(i, w) || !disjoint(w, l) || !disjoint(w, b))
        return SKINNY_ERR_INVALID_ARG;
    return SKINNY_OK;
}

// Rows of one pair of launches: the pairs of that many rows are sorted at once.
constexpr int32_t kExpertsRows = 128;

// Blocks of the second kernel.
constexpr int32_t kDownBlocks = 256;

// The workspace: the order of the pairs (16 bytes for the number of tiles and the second kernel's
// runs, 4 for each tile, 16 for each pair), h in up to 4 bytes a value, and for each of the second
// kernel's blocks 16 bytes, a counter and two sets of 16 outputs of every row.
struct ExpertsSpace {
    uint64_t entries, h, begins, arrived, parts, bytes;  // offsets, and all of it
};

inline ExpertsSpace experts_space(int32_t M, int32_t k, int32_t E, int32_t I)
{
    const uint64_t rows = (uint64_t)(M < kExpertsRows ? M : kExpertsRows), pairs = rows * (uint64_t)k;
    // every expert may have a tile that is not full
    const uint64_t most = pairs < (uint64_t)E + pairs / 4 ? pairs : (uint64_t)E + pairs / 4;
    ExpertsSpace s{};
    s.entries = 16 + (4 * most + 15) / 16 * 16;
    s.h = s.entries + 16 * pairs;
    s.begins = s.h + (4 * pairs * (uint64_t)I + 15) / 16 * 16;
    s.arrived = s.begins + 16 * (uint64_t)kDownBlocks;
    s.parts = s.arrived + 4 * (uint64_t)kDownBlocks;
    s.bytes = s.parts + 2 * (uint64_t)kDownBlocks * rows * 64;
    return s;
}

inline bool experts_sizes_ok(int32_t M, int32_t k, int32_t E, int32_t I)
{
    return M >= 0 && k >= 1 && k <= kMaxExpertsK && E >= 1 && E <= kMaxExperts && I >= 1;
}

inline int validate_experts(const skinny_experts_t *a)
{
    if (!a || !experts_sizes_ok(a->M, a->k, a->E, a->I) || a->H < 1)
        return SKINNY_ERR_INVALID_ARG;
    if (a->act < SKINNY_ACT_NONE || a->act > SKINNY_ACT_SILU || a->type < SKINNY_WEIGHTS_BF16 ||
        a->type > SKINNY_WEIGHTS_INT8_ROW)
        return SKINNY_ERR_INVALID_ARG;
    const bool bytes = a->type != SKINNY_WEIGHTS_BF16, blocks = a->type == SKINNY_WEIGHTS_E4M3_BLOCK;
    if (!bytes && (a->gate_scale || a->up_scale || a->down_scale))
        return SKINNY_ERR_INVALID_ARG;
    if (a->M == 0)
        return SKINNY_OK;
    if (!a->x || !a->ids || !a->weights || !a->w_gate || !a->w_up || !a->w_down || !a->y || !a->workspace)
        return SKINNY_ERR_INVALID_ARG;
    if (bytes && (!a->gate_scale || !a->up_scale || !a->down_scale))
        return SKINNY_ERR_INVALID_ARG;
    const uint64_t M = (uint64_t)a->M, E = (uint64_t)a->E, k = (uint64_t)a->k, H = (uint64_t)a->H, I = (uint64_t)a->I;
    const uint64_t e = bytes ? 1 : 2, hb = (H + 127) / 128, ib = (I + 127) / 128;
    const uint64_t one = H * I, up_scales = blocks ? ib * hb : I, down_scales = blocks ? ib * hb : H;
    if (!ld_ok(a->ldx, a->H) || !ld_ok(a->ldy, a->H) || (a->residual && !ld_ok(a->ldr, a->H)))
        return SKINNY_ERR_INVALID_ARG;
    auto stride_ok = [](int64_t s, uint64_t least) { return s >= 0 && (uint64_t)s >= least && (uint64_t)s <= kMaxStride / 4; };
    if (!stride_ok(a->up_stride, one) || !stride_ok(a->down_stride, one) ||
        (bytes && (!stride_ok(a->up_scale_stride, up_scales) || !stride_ok(a->down_scale_stride, down_scales))))
        return SKINNY_ERR_INVALID_ARG;
    if (!aligned(a->x, 2) || !aligned(a->y, 2) || !aligned(a->residual, 2) || !aligned(a->ids, 4) || !aligned(a->weights, 4) ||
        !aligned(a->w_gate, e) || !aligned(a->w_up, e) || !aligned(a->w_down, e) || !aligned(a->gate_scale, 4) ||
        !aligned(a->up_scale, 4) || !aligned(a->down_scale, 4) || !aligned(a->workspace, 16))
        return SKINNY_ERR_INVALID_ARG;
    const uint64_t need = experts_space(a->M, a->k, a->E, a->I).bytes;
    if (a->workspace_bytes < need)
        return SKINNY_ERR_INVALID_ARG;
    const Block y{a->y, M, 2 * H, 2 * (uint64_t)a->ldy}, ws = flat(a->workspace, need);
    const Block res{a->residual, a->residual ? M : 0, 2 * H, a->residual ? 2 * (uint64_t)a->ldr : 0};
    const Block in[] = {{a->x, M, 2 * H, 2 * (uint64_t)a->ldx},
                        flat(a->ids, 4 * M * k),
                        flat(a->weights, 4 * M * k),
                        {a->w_gate, E, e * one, e * (uint64_t)a->up_stride},
                        {a->w_up, E, e * one, e * (uint64_t)a->up_stride},
                        {a->w_down, E, e * one, e * (uint64_t)a->down_stride},
                        {a->gate_scale, a->gate_scale ? E : 0, 4 * up_scales, 4 * (uint64_t)a->up_scale_stride},
                        {a->up_scale, a->up_scale ? E : 0, 4 * up_scales, 4 * (uint64_t)a->up_scale_stride},
                        {a->down_scale, a->down_scale ? E : 0, 4 * down_scales, 4 * (uint64_t)a->down_scale_stride}};
    if (!reaches(y) || !reaches(res) || !reaches(ws) || !disjoint(y, ws) || !disjoint(ws, res))
        return SKINNY_ERR_INVALID_ARG;
    for (const Block &b : in)
        if (!reaches(b) || !disjoint(y, b) || !disjoint(ws, b))
            return SKINNY_ERR_INVALID_ARG;
    if (!(disjoint(y, res) || same_rows(y, res)))
        return SKINNY_ERR_INVALID_ARG;
    return SKINNY_OK;
}

// x, the weights and h can be read in 16-byte pieces, and the 32-bit byte offsets of the
// kernels' buffer resources reach: 128 rows of x, 32 of h (16 where it has two parts), 16 of a
// weight.
inline bool experts_vector_ok(const skinny_experts_t &a)
{
    const int64_t piece = a.type == SKINNY_WEIGHTS_BF16 ? 8 : 16;
    return a.H % piece == 0 && a.I % piece == 0 && a.up_stride % piece == 0 && a.down_stride % piece == 0 && a.ldx % 8 == 0 &&
           aligned(a.x, 16) && aligned(a.w_gate, 16) && aligned(a.w_up, 16) && aligned(a.w_down, 16) &&
           a.ldx <= (INT64_C(1) << 22) && a.H <= (1 << 22) && a.I <= (1 << 22);
}

}  // namespace skg_host

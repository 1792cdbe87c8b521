// Host-side argument checks of include/skinny_ops.h: plain C++ with no HIP code, like
// validate.hpp, so that a sanitizer build on the CPU runs exactly these.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "skinny_ops.h"
#include "validate.hpp"

namespace skg_host {

// A row-strided block of memory: `rows` rows of `width` bytes, `stride` bytes apart.
struct Block {
    const void *p;
    uint64_t rows, width, stride;
};

// Largest row stride, in bytes, and largest extent of one matrix: far beyond any
// device's memory, and small enough that the arithmetic below cannot wrap.
constexpr uint64_t kMaxStride = 1ull << 40;
constexpr uint64_t kMaxExtent = 1ull << 46;

inline uint64_t extent(const Block &b)
{
    return b.rows && b.width ? (b.rows - 1) * b.stride + b.width : 0;
}

// The extent of the block is representable and does not wrap the address space.
inline bool block_ok(const Block &b)
{
    if (!b.rows || !b.width)
        return true;
    if (b.stride > kMaxStride || b.width > kMaxStride)
        return false;
    if (b.rows > 1 && b.stride > kMaxExtent / (b.rows - 1))
        return false;
    const uint64_t e = extent(b);
    return e <= kMaxExtent && reinterpret_cast<uintptr_t>(b.p) <= UINTPTR_MAX - e;
}

// No byte in common: the extents do not meet, or (equal strides) the rows of one
// fall in the gaps of the other.
inline bool disjoint(const Block &a, const Block &b)
{
    if (!a.p || !b.p)
        return true;
    const uint64_t ea = extent(a), eb = extent(b);
    if (!ea || !eb || !overlaps(a.p, ea, b.p, eb))
        return true;
    if (a.stride != b.stride || a.rows < 2 || b.rows < 2)
        return false;
    const uint64_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const uint64_t s = a.stride;
    // where b's rows start within a's stride period
    const uint64_t r = pb >= pa ? (pb - pa) % s : (s - (pa - pb) % s) % s;
    return r >= a.width && r + b.width <= s;
}

// The same rows: an output written over an input element by element.
inline bool same_rows(const Block &a, const Block &b)
{
    return a.p == b.p && a.width == b.width && (a.stride == b.stride || a.rows < 2);
}

inline bool ld_ok(int64_t ld, int64_t width) { return ld >= width && (uint64_t)ld <= kMaxStride / 4; }

inline int validate_norm(const skinny_norm_t *a, bool fp8)
{
    if (!a || a->M < 0 || a->D < 0)
        return SKINNY_ERR_INVALID_ARG;
    if (!(a->eps >= 0.0f) || std::isinf(a->eps) || (a->residual != nullptr) != (a->residual_out != nullptr))
        return SKINNY_ERR_INVALID_ARG;
    if (fp8 ? (a->group != 0 && a->group != 128) : a->group != 0)
        return SKINNY_ERR_INVALID_ARG;
    if (a->M == 0 || a->D == 0)
        return SKINNY_OK;
    const bool res = a->residual != nullptr;
    if (!a->x || !a->weight || !a->y || (fp8 && !a->scale))
        return SKINNY_ERR_INVALID_ARG;
    if (!ld_ok(a->ldx, a->D) || !ld_ok(a->ldy, a->D) || (res && (!ld_ok(a->ldr, a->D) || !ld_ok(a->ldro, a->D))))
        return SKINNY_ERR_INVALID_ARG;
    if (!aligned(a->x, 2) || !aligned(a->weight, 2) || (!fp8 && !aligned(a->y, 2)) || !aligned(a->residual, 2) ||
        !aligned(a->residual_out, 2) || (fp8 && !aligned(a->scale, 4)))
        return SKINNY_ERR_INVALID_ARG;
    const uint64_t M = (uint64_t)a->M, D = (uint64_t)a->D, ye = fp8 ? 1 : 2;
    const uint64_t groups = a->group ? (D + a->group - 1) / a->group : 1;
    const Block x{a->x, M, 2 * D, 2 * (uint64_t)a->ldx};
    const Block r{a->residual, res ? M : 0, 2 * D, res ? 2 * (uint64_t)a->ldr : 0};
    const Block ro{a->residual_out, res ? M : 0, 2 * D, res ? 2 * (uint64_t)a->ldro : 0};
    const Block w{a->weight, 1, 2 * D, 2 * D};
    const Block y{a->y, M, ye * D, ye * (uint64_t)a->ldy};
    const Block s{fp8 ? a->scale : nullptr, fp8 ? M : 0, 4 * groups, 4 * groups};
    for (const Block *b : {&x, &r, &ro, &w, &y, &s})
        if (!block_ok(*b))
            return SKINNY_ERR_INVALID_ARG;
    const bool y_is_x = !fp8 && same_rows(y, x);
    if (!(disjoint(y, x) || y_is_x) || !disjoint(y, r) || !disjoint(y, ro) || !disjoint(y, w) || !disjoint(y, s))
        return SKINNY_ERR_INVALID_ARG;
    if (!(disjoint(ro, x) || same_rows(ro, x)) || !(disjoint(ro, r) || same_rows(ro, r)) || !disjoint(ro, w) ||
        !disjoint(ro, s))
        return SKINNY_ERR_INVALID_ARG;
    // an output over one input must not meet the other input in other places
    if (!disjoint(s, x) || !disjoint(s, r) || !disjoint(s, w))
        return SKINNY_ERR_INVALID_ARG;
    return SKINNY_OK;
}

inline int validate_linear(const skinny_linear_t *a, bool fp8)
{
    if (!a || a->M < 0 || a->N < 0 || a->K < 0)
        return SKINNY_ERR_INVALID_ARG;
    if (a->act < SKINNY_ACT_NONE || a->act > SKINNY_ACT_SILU || a->out_f32 < 0 || a->out_f32 > 1)
        return SKINNY_ERR_INVALID_ARG;
    if (fp8 ? (a->scales != SKINNY_SCALES_ROW && a->scales != SKINNY_SCALES_BLOCK) : a->scales != 0)
        return SKINNY_ERR_INVALID_ARG;
    const bool gated = a->W1 != nullptr;
    if (gated ? a->residual != nullptr : a->bias1 != nullptr)
        return SKINNY_ERR_INVALID_ARG;
    if (a->M == 0 || a->N == 0)
        return SKINNY_OK;
    if (!a->y || (a->K > 0 && (!a->x || !a->W0)))
        return SKINNY_ERR_INVALID_ARG;
    if (fp8 && a->K > 0 && (!a->x_scale || !a->w0_scale || (gated && !a->w1_scale)))
        return SKINNY_ERR_INVALID_ARG;
    if (!ld_ok(a->ldx, a->K) || !ld_ok(a->ldy, a->N) || (a->residual && !ld_ok(a->ldr, a->N)))
        return SKINNY_ERR_INVALID_ARG;
    const uintptr_t ea = fp8 ? 1 : 2;
    if (!aligned(a->x, ea) || !aligned(a->W0, ea) || !aligned(a->W1, ea) || !aligned(a->bias0, 2) ||
        !aligned(a->bias1, 2) || !aligned(a->residual, 2) || !aligned(a->y, a->out_f32 ? 4 : 2))
        return SKINNY_ERR_INVALID_ARG;
    if (fp8 && (!aligned(a->x_scale, 4) || !aligned(a->w0_scale, 4) || !aligned(a->w1_scale, 4)))
        return SKINNY_ERR_INVALID_ARG;
    const uint64_t M = (uint64_t)a->M, N = (uint64_t)a->N, K = (uint64_t)a->K, e = fp8 ? 1 : 2;
    const uint64_t ye = a->out_f32 ? 4 : 2, kb = (K + 127) / 128, nb = (N + 127) / 128;
    const bool blocks = a->scales == SKINNY_SCALES_BLOCK;
    const uint64_t xs = fp8 ? 4 * M * (blocks ? kb : 1) : 0, ws = fp8 ? 4 * (blocks ? nb * kb : N) : 0;
    const Block y{a->y, M, ye * N, ye * (uint64_t)a->ldy};
    const Block res{a->residual, a->residual ? M : 0, 2 * N, a->residual ? 2 * (uint64_t)a->ldr : 0};
    const Block in[] = {{a->x, M, e * K, e * (uint64_t)a->ldx},
                        {a->W0, 1, e * N * K, e * N * K},
                        {a->W1, 1, e * N * K, e * N * K},
                        {a->x_scale, 1, xs, xs},
                        {a->w0_scale, 1, ws, ws},
                        {a->w1_scale, 1, ws, ws},
                        {a->bias0, 1, 2 * N, 2 * N},
                        {a->bias1, 1, 2 * N, 2 * N}};
    if (!block_ok(y) || !block_ok(res))
        return SKINNY_ERR_INVALID_ARG;
    for (const Block &b : in) {
        if (!b.p)
            continue;
        if (b.rows == 1 ? (b.width > kMaxExtent || reinterpret_cast<uintptr_t>(b.p) > UINTPTR_MAX - b.width)
                        : !block_ok(b))
            return SKINNY_ERR_INVALID_ARG;
        if (!disjoint(y, b))
            return SKINNY_ERR_INVALID_ARG;
    }
    if (!(disjoint(y, res) || (!a->out_f32 && same_rows(y, res))))
        return SKINNY_ERR_INVALID_ARG;
    return SKINNY_OK;
}

// Products of K 8-bit integers, each at most 2^14 in magnitude, must add up within 32 bits.
constexpr int32_t kMaxInt8Depth = 131071;

inline int validate_linear_int8(const skinny_linear_t *a)
{
    if (!a || a->scales != SKINNY_SCALES_ROW || a->K > kMaxInt8Depth)
        return SKINNY_ERR_INVALID_ARG;
    return validate_linear(a, true);
}

inline int validate_norm_int8(const skinny_norm_t *a)
{
    if (!a || a->group != 0)
        return SKINNY_ERR_INVALID_ARG;
    return validate_norm(a, true);
}

// skinny_quantize_int8: a norm's call without weight, residual and eps.
inline int validate_quantize(const skinny_norm_t *a)
{
    if (!a || a->weight || a->residual || a->residual_out || a->eps != 0.0f)
        return SKINNY_ERR_INVALID_ARG;
    skinny_norm_t with = *a;
    with.weight = a->x;  // its extent is a part of x's
    return validate_norm_int8(&with);
}

// Rows of x and W can be read in 16-byte pieces, and the 32-bit byte offsets of the
// kernels' buffer resources reach: 256 rows of x or W from a tile's first.
inline bool linear_vector_ok(const skinny_linear_t &a, bool fp8)
{
    const int64_t e = fp8 ? 1 : 2, piece = 16 / e;
    return a.K > 0 && a.K % piece == 0 && a.ldx % piece == 0 && aligned(a.x, 16) && aligned(a.W0, 16) &&
           aligned(a.W1, 16) && a.ldx <= (INT64_C(1) << 22) && a.K <= (1 << 22);
}

}  // namespace skg_host

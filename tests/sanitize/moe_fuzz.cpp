// The argument checks of include/skinny_moe.h and of the 8-bit integer entry points of
// include/skinny_ops.h (csrc/validate_moe.hpp, validate_ops.hpp) under the address and
// undefined-behaviour sanitizers: random and extreme arguments, and for every accepted call
// with small sizes the bytes it would write, checked one by one against the others'.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>

#include "../../bf16_skinny_gemm_amd/csrc/validate_moe.hpp"

namespace {

std::mt19937_64 rng(54321);

template <typename T>
T *ptr(uint64_t p)
{
    return reinterpret_cast<T *>(static_cast<uintptr_t>(p));
}

void add(std::set<uint64_t> &s, const void *p, int64_t rows, int64_t width, int64_t stride)
{
    if (!p)
        return;
    const uint64_t b = reinterpret_cast<uintptr_t>(p);
    for (int64_t r = 0; r < rows; ++r)
        for (int64_t i = 0; i < width; ++i)
            s.insert(b + (uint64_t)(r * stride + i));
}

bool within(const std::set<uint64_t> &a, uint64_t from, uint64_t bytes)
{
    const auto it = a.lower_bound(from);
    return it != a.end() && *it < from + bytes;
}

bool meet(const std::set<uint64_t> &a, const std::set<uint64_t> &b)
{
    for (uint64_t v : a)
        if (b.count(v))
            return true;
    return false;
}

int fail(const char *what, long i)
{
    std::printf("FAILED: %s at %ld\n", what, i);
    return 1;
}

}  // namespace

int main()
{
    using namespace skg_host;
    const int64_t wide[] = {0, 1, -1, 7, 8, 128, 1 << 20, 0x7FFFFFFF, INT64_MIN, INT64_MAX, INT64_C(1) << 38, INT64_C(1) << 40,
                            INT64_C(1) << 62};
    const int32_t sizes[] = {0, 1, -1, 5, 32, 64, 128, 1024, 1 << 22, 0x7FFFFFFF, INT32_MIN};
    const int64_t places[] = {0, 2, 16, 4096, 0x10000, INT64_MAX, -1, -2, -16, INT64_C(1) << 45};
    auto e64 = [&] { return wide[rng() % (sizeof(wide) / sizeof(wide[0]))]; };
    auto e32 = [&] { return sizes[rng() % (sizeof(sizes) / sizeof(sizes[0]))]; };
    auto ep = [&] { return (uint64_t)places[rng() % (sizeof(places) / sizeof(places[0]))]; };
    long accepted = 0;
    // extreme values: nothing may overflow, whatever the answer
    for (long i = 0; i < 400000; ++i) {
        skinny_route_t r{};
        r.logits = ptr<float>(ep()), r.bias = ptr<float>(ep()), r.ids = ptr<int32_t>(ep()), r.weights = ptr<float>(ep());
        r.ldl = e64(), r.M = e32(), r.E = e32(), r.k = e32(), r.score = (int)(rng() % 3), r.groups = e32(), r.kept = e32();
        r.renormalize = (int)(rng() & 1), r.scale = 1.0f;
        if (rng() & 1)
            r.groups = r.kept = 1;
        accepted += validate_route(&r) == SKINNY_OK;
        skinny_experts_t a{};
        a.x = ptr<void>(ep()), a.ids = ptr<int32_t>(ep()), a.weights = ptr<float>(ep()), a.w_gate = ptr<void>(ep());
        a.w_up = ptr<void>(ep()), a.w_down = ptr<void>(ep()), a.gate_scale = ptr<float>(ep()), a.up_scale = ptr<float>(ep());
        a.down_scale = ptr<float>(ep()), a.residual = ptr<void>(ep()), a.y = ptr<void>(ep()), a.workspace = ptr<void>(ep());
        a.workspace_bytes = (size_t)e64(), a.ldx = e64(), a.ldr = e64(), a.ldy = e64(), a.up_stride = e64();
        a.down_stride = e64(), a.up_scale_stride = e64(), a.down_scale_stride = e64();
        a.M = e32(), a.E = e32(), a.k = e32(), a.H = e32(), a.I = e32(), a.act = (int)(rng() % 6), a.type = (int)(rng() % 5);
        if (a.type == 0)
            a.gate_scale = a.up_scale = a.down_scale = nullptr;
        if (validate_experts(&a) == SKINNY_OK) {
            ++accepted;
            (void)experts_vector_ok(a);
        }
        skinny_linear_t l{};
        l.x = ptr<void>(ep()), l.W0 = ptr<void>(ep()), l.x_scale = ptr<float>(ep()), l.w0_scale = ptr<float>(ep());
        l.y = ptr<void>(ep()), l.ldx = e64(), l.ldy = e64(), l.M = e32(), l.N = e32(), l.K = e32(), l.scales = (int)(rng() % 3);
        accepted += validate_linear_int8(&l) == SKINNY_OK;
        skinny_norm_t n{};
        n.x = ptr<void>(ep()), n.weight = ptr<void>(rng() & 1 ? ep() : 0), n.y = ptr<void>(ep()), n.scale = ptr<float>(ep());
        n.ldx = e64(), n.ldy = e64(), n.M = e32(), n.D = e32();
        accepted += validate_norm_int8(&n) == SKINNY_OK;
        accepted += validate_quantize(&n) == SKINNY_OK;
    }
    // small calls in a crowded memory: what is accepted writes over no other operand
    long checked = 0;
    for (long i = 0; i < 200000; ++i) {
        auto at = [&] { return 4096 + rng() % 400 * 4; };
        skinny_route_t r{};
        r.M = 1 + (int)(rng() % 3), r.E = 1 + (int)(rng() % 9), r.k = 1 + (int)(rng() % r.E), r.ldl = r.E + (int)(rng() % 5);
        r.logits = ptr<float>(at()), r.ids = ptr<int32_t>(at()), r.weights = ptr<float>(at());
        r.bias = rng() & 1 ? ptr<float>(at()) : nullptr;
        r.groups = r.kept = 1, r.scale = 1.0f;
        if (validate_route(&r) != SKINNY_OK)
            continue;
        ++checked;
        std::set<uint64_t> in, ids, w;
        add(in, r.logits, r.M, 4 * r.E, 4 * r.ldl);
        add(in, r.bias, 1, 4 * r.E, 0);
        add(ids, r.ids, 1, 4 * r.M * r.k, 0);
        add(w, r.weights, 1, 4 * r.M * r.k, 0);
        if (meet(ids, in) || meet(w, in) || meet(ids, w))
            return fail("a router that overwrites an operand", i);
    }
    for (long i = 0; i < 100000; ++i) {
        // the workspace, the largest by far, lies before, behind or among the others
        auto at = [&] { return (1 << 20) + rng() % 1500 * 4; };
        skinny_experts_t a{};
        a.M = 1 + (int)(rng() % 3), a.E = 1 + (int)(rng() % 3), a.k = 1 + (int)(rng() % 2), a.H = 1 + (int)(rng() % 6);
        a.I = 1 + (int)(rng() % 6), a.type = (int)(rng() % 4);
        const bool bytes = a.type != 0;
        const int e = bytes ? 1 : 2, us = a.type == 2 ? 1 : a.I, ds = a.type == 2 ? 1 : a.H;
        a.x = ptr<void>(at()), a.ids = ptr<int32_t>(at()), a.weights = ptr<float>(at()), a.w_gate = ptr<void>(at());
        a.w_up = ptr<void>(at()), a.w_down = ptr<void>(at()), a.y = ptr<void>(at());
        if (rng() & 1) {
            a.residual = rng() & 1 ? a.y : ptr<void>(at());
            a.ldr = a.H + (int)(rng() % 3);
        }
        a.ldx = a.H + (int)(rng() % 4), a.ldy = rng() & 1 && a.residual ? a.ldr : a.H + (int)(rng() % 4);
        a.up_stride = a.H * a.I + (int)(rng() % 4), a.down_stride = a.H * a.I + (int)(rng() % 4);
        if (bytes) {
            a.gate_scale = ptr<float>(at()), a.up_scale = ptr<float>(at()), a.down_scale = ptr<float>(at());
            a.up_scale_stride = us + (int)(rng() % 3), a.down_scale_stride = ds + (int)(rng() % 3);
        }
        a.workspace_bytes = skg_host::experts_space(a.M, a.k, a.E, a.I).bytes;
        const uint64_t to = at() & ~15ull;
        a.workspace = ptr<void>(rng() & 1 ? to : (to - a.workspace_bytes) & ~15ull);
        if (validate_experts(&a) != SKINNY_OK)
            continue;
        ++checked;
        std::set<uint64_t> y, in, res;
        const uint64_t ws = reinterpret_cast<uintptr_t>(a.workspace), bytes_of = a.workspace_bytes;
        add(y, a.y, a.M, 2 * a.H, 2 * a.ldy);
        add(in, a.x, a.M, 2 * a.H, 2 * a.ldx);
        add(in, a.ids, 1, 4 * a.M * a.k, 0);
        add(in, a.weights, 1, 4 * a.M * a.k, 0);
        add(in, a.w_gate, a.E, e * a.H * a.I, e * a.up_stride);
        add(in, a.w_up, a.E, e * a.H * a.I, e * a.up_stride);
        add(in, a.w_down, a.E, e * a.H * a.I, e * a.down_stride);
        if (bytes) {
            add(in, a.gate_scale, a.E, 4 * us, 4 * a.up_scale_stride);
            add(in, a.up_scale, a.E, 4 * us, 4 * a.up_scale_stride);
            add(in, a.down_scale, a.E, 4 * ds, 4 * a.down_scale_stride);
        }
        add(res, a.residual, a.M, 2 * a.H, 2 * a.ldr);
        const bool same = a.residual == a.y && (a.ldr == a.ldy || a.M == 1);
        if (meet(y, in) || within(y, ws, bytes_of) || within(in, ws, bytes_of) || within(res, ws, bytes_of) || (meet(y, res) && !same))
            return fail("experts that overwrite an operand", i);
    }
    std::printf("moe validation: ok (%ld extreme calls accepted, %ld small ones checked)\n", accepted, checked);
    return checked > 1000 ? 0 : fail("too few accepted calls", checked);
}

// The argument checks of include/skinny_ops.h (csrc/validate_ops.hpp) under the address
// and undefined-behaviour sanitizers: random and extreme arguments, and for every
// accepted call with small sizes the bytes it would write, checked one by one against the
// bytes it may read and the other bytes it would write.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>

#include "../../bf16_skinny_gemm_amd/csrc/validate_ops.hpp"

namespace {

std::mt19937_64 rng(12345);

int64_t pick(std::initializer_list<int64_t> v)
{
    return *(v.begin() + rng() % v.size());
}

template <typename T>
T *ptr(uint64_t p)
{
    return reinterpret_cast<T *>(static_cast<uintptr_t>(p));
}

void add(std::set<uint64_t> &s, const void *p, int64_t rows, int64_t width, int64_t stride)
{
    const uint64_t b = reinterpret_cast<uintptr_t>(p);
    for (int64_t r = 0; r < rows; ++r)
        for (int64_t i = 0; i < width; ++i)
            s.insert(b + (uint64_t)(r * stride + i));
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
    const int64_t extremes[] = {0, 1, -1, 7, 8, 128, 1 << 20, 0x7FFFFFFF, INT64_MIN, INT64_MAX, INT64_C(1) << 38,
                                INT64_C(1) << 40, INT64_C(1) << 62};
    const int32_t sizes[] = {0, 1, -1, 5, 128, 1 << 22, 0x7FFFFFFF, INT32_MIN};
    auto e64 = [&] { return extremes[rng() % (sizeof(extremes) / sizeof(extremes[0]))]; };
    auto e32 = [&] { return sizes[rng() % (sizeof(sizes) / sizeof(sizes[0]))]; };
    auto ep = [&] { return pick({0, 2, 16, 4096, 0x10000, INT64_MAX, -1, -2, -16}); };
    long accepted = 0;
    // extreme values: nothing may overflow, whatever the answer
    for (long i = 0; i < 400000; ++i) {
        skinny_norm_t n{};
        n.x = ptr<void>(ep()), n.residual = ptr<void>(ep()), n.weight = ptr<void>(ep());
        n.residual_out = ptr<void>(ep()), n.y = ptr<void>(ep()), n.scale = ptr<float>(ep());
        n.ldx = e64(), n.ldr = e64(), n.ldro = e64(), n.ldy = e64();
        n.M = e32(), n.D = e32(), n.group = (int32_t)pick({0, 128, 1}), n.eps = 1e-6f;
        accepted += skg_host::validate_norm(&n, i & 1) == SKINNY_OK;
        skinny_linear_t a{};
        a.x = ptr<void>(ep()), a.W0 = ptr<void>(ep()), a.W1 = ptr<void>(ep());
        a.x_scale = ptr<float>(ep()), a.w0_scale = ptr<float>(ep()), a.w1_scale = ptr<float>(ep());
        a.bias0 = ptr<void>(ep()), a.bias1 = ptr<void>(ep()), a.residual = ptr<void>(ep()), a.y = ptr<void>(ep());
        a.ldx = e64(), a.ldr = e64(), a.ldy = e64();
        a.M = e32(), a.N = e32(), a.K = e32(), a.act = (int32_t)pick({0, 4, 5, -1}), a.out_f32 = (int32_t)pick({0, 1});
        a.scales = (int32_t)pick({0, 1, 2});
        const bool ok = skg_host::validate_linear(&a, i & 1) == SKINNY_OK;
        accepted += ok;
        if (ok)
            (void)skg_host::linear_vector_ok(a, i & 1);
    }
    // small calls in a crowded memory: what is accepted writes over no other operand
    long checked = 0;
    for (long i = 0; i < 200000; ++i) {
        const bool fp8 = rng() & 1;
        const uint64_t base = 4096;
        auto at = [&] { return base + rng() % 400 * 2; };
        skinny_norm_t n{};
        n.M = 1 + (int)(rng() % 3), n.D = 1 + (int)(rng() % 20);
        const bool res = rng() & 1;
        n.x = ptr<void>(at()), n.weight = ptr<void>(at()), n.y = ptr<void>(rng() % 4 ? at() : (uint64_t)n.x);
        n.ldx = n.D + (int)(rng() % 30), n.ldy = rng() % 2 ? n.ldx : n.D + (int)(rng() % 30);
        n.scale = fp8 ? ptr<float>(at() & ~3ull) : nullptr;
        n.group = fp8 && (rng() & 1) ? 128 : 0;
        if (res) {
            n.residual = ptr<void>(at()), n.ldr = rng() % 2 ? n.ldx : n.D + (int)(rng() % 30);
            n.residual_out = ptr<void>(rng() % 3 == 0 ? (uint64_t)n.residual : rng() % 3 == 0 ? (uint64_t)n.x : at());
            n.ldro = rng() % 2 ? n.ldr : n.ldx;
            if (n.ldro < n.D)
                n.ldro = n.D;
        }
        if (skg_host::validate_norm(&n, fp8) != SKINNY_OK)
            continue;
        ++checked;
        const int ye = fp8 ? 1 : 2;
        std::set<uint64_t> x, r, w, y, ro, s;
        add(x, n.x, n.M, 2 * n.D, 2 * n.ldx);
        add(w, n.weight, 1, 2 * n.D, 0);
        add(y, n.y, n.M, ye * n.D, ye * n.ldy);
        if (res) {
            add(r, n.residual, n.M, 2 * n.D, 2 * n.ldr);
            add(ro, n.residual_out, n.M, 2 * n.D, 2 * n.ldro);
        }
        if (fp8)
            add(s, n.scale, n.M, 4 * (n.group ? (n.D + 127) / 128 : 1), 4 * (n.group ? (n.D + 127) / 128 : 1));
        const bool y_x = !fp8 && n.y == n.x && (n.ldy == n.ldx || n.M == 1);
        const bool ro_x = n.residual_out == n.x && (n.ldro == n.ldx || n.M == 1);
        const bool ro_r = n.residual_out == n.residual && (n.ldro == n.ldr || n.M == 1);
        if ((meet(y, x) && !y_x) || meet(y, r) || meet(y, w) || meet(y, ro) || meet(y, s) || meet(s, x) || meet(s, r) ||
            meet(s, w) || meet(s, ro) || meet(ro, w) || (meet(ro, x) && !ro_x) || (meet(ro, r) && !ro_r))
            return fail("a norm that overwrites an operand", i);
    }
    for (long i = 0; i < 100000; ++i) {
        const bool fp8 = rng() & 1;
        auto at = [&] { return 4096 + rng() % 600 * 4; };
        skinny_linear_t a{};
        a.M = 1 + (int)(rng() % 3), a.N = 1 + (int)(rng() % 9), a.K = 1 + (int)(rng() % 9);
        const bool gated = rng() % 3 == 0;
        a.x = ptr<void>(at()), a.W0 = ptr<void>(at()), a.W1 = gated ? ptr<void>(at()) : nullptr;
        a.ldx = a.K + (int)(rng() % 9), a.ldy = a.N + (int)(rng() % 9);
        a.out_f32 = rng() & 1;
        a.y = ptr<void>(at());
        if (!gated && (rng() & 1)) {
            a.residual = rng() & 1 ? a.y : ptr<void>(at());
            a.ldr = rng() & 1 ? a.ldy : a.N + (int)(rng() % 9);
        }
        a.bias0 = rng() & 1 ? ptr<void>(at()) : nullptr;
        if (fp8) {
            a.scales = 1 + (int)(rng() & 1);
            a.x_scale = ptr<float>(at()), a.w0_scale = ptr<float>(at());
            a.w1_scale = gated ? ptr<float>(at()) : nullptr;
        }
        if (skg_host::validate_linear(&a, fp8) != SKINNY_OK)
            continue;
        ++checked;
        const int e = fp8 ? 1 : 2, ye = a.out_f32 ? 4 : 2;
        std::set<uint64_t> y, in, r;
        add(y, a.y, a.M, ye * a.N, ye * a.ldy);
        add(in, a.x, a.M, e * a.K, e * a.ldx);
        add(in, a.W0, 1, e * a.N * a.K, 0);
        if (gated)
            add(in, a.W1, 1, e * a.N * a.K, 0);
        if (a.bias0)
            add(in, a.bias0, 1, 2 * a.N, 0);
        if (fp8) {
            add(in, a.x_scale, 1, 4 * a.M, 0);
            add(in, a.w0_scale, 1, 4 * (a.scales == 1 ? a.N : 1), 0);
            if (gated)
                add(in, a.w1_scale, 1, 4 * (a.scales == 1 ? a.N : 1), 0);
        }
        if (a.residual)
            add(r, a.residual, a.M, 2 * a.N, 2 * a.ldr);
        const bool same = a.residual == a.y && !a.out_f32 && (a.ldr == a.ldy || a.M == 1);
        if (meet(y, in) || (meet(y, r) && !same))
            return fail("a projection that overwrites an operand", i);
    }
    std::printf("ops validation: ok (%ld extreme calls accepted, %ld small ones checked)\n", accepted, checked);
    return checked > 1000 ? 0 : fail("too few accepted calls", checked);
}

// Host side of skinny_linear_bf16, _fp8 and _int8 (include/skinny_ops.h): the choice
// of kernel, and the element-wise kernel for what the vector paths do not take.
#include "ops_host.hpp"

#include <cmath>
#include <cstdint>

#include "linear.hpp"
#include "validate_ops.hpp"

namespace skg {

// Any alignment, stride and K: 16 x 16 outputs per block of 256 threads, K in parts of
// 64 columns through LDS as floats (64 divides a 128-column block of scales), or as integers
// where x and W are. One multiply-add for two reads of LDS, which bound it: bfloat16 1 x 4096 x 4100 151 us, 64 rows
// 205 us, 4096 rows 8.8 ms, where a K of 4096 takes 8, 10 and 96 us.
template <int MODE, bool GATED>
__global__ __launch_bounds__(256) void linear_any_kernel(LinArgs a, int64_t tiles, int nt)
{
    constexpr int MATS = GATED ? 2 : 1;
    using val = std::conditional_t<MODE == kInt8Row, int, float>;
    __shared__ val xl[16][65], wl[MATS][16][65];
    const int tn = threadIdx.x & 15, tm = threadIdx.x >> 4;
    const int64_t wld = (int64_t)a.K;
    auto at = [&](const uint8_t *p, int64_t i) {
        if constexpr (MODE == kBf16)
            return bf16_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
        else if constexpr (MODE == kInt8Row)
            return (int)reinterpret_cast<const int8_t *>(p)[i];
        else
            return __builtin_amdgcn_cvt_f32_fp8((int)p[i], 0);
    };
    const int64_t ldx = MODE == kBf16 ? a.ldx / 2 : a.ldx;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int n0 = (int)(tile % nt) * 16, m0 = (int)(tile / nt) * 16;
        val acc[MATS] = {};
        for (int k0 = 0; k0 < a.K; k0 += 64) {
            __syncthreads();
            for (int i = threadIdx.x; i < 16 * 64; i += 256) {
                const int r = i >> 6, k = i & 63;
                const bool kin = k < a.K - k0;
                xl[r][k] = kin && r < a.M - m0 ? at(a.x, (int64_t)(m0 + r) * ldx + k0 + k) : val(0);
#pragma unroll
                for (int t = 0; t < MATS; ++t)
                    wl[t][r][k] = kin && r < a.N - n0 ? at(a.w[t], (int64_t)(n0 + r) * wld + k0 + k) : val(0);
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < MATS; ++t) {
                val p = MODE == kE4m3Block ? val(0) : acc[t];
                for (int k = 0; k < 64; ++k) {
                    if constexpr (MODE == kInt8Row)
                        p += xl[tm][k] * wl[t][tn][k];
                    else
                        p = __builtin_fmaf(xl[tm][k], wl[t][tn][k], p);
                }
                if constexpr (MODE == kE4m3Block) {
                    const int b = k0 >> 7;
                    if (tm < a.M - m0 && tn < a.N - n0)
                        acc[t] = __builtin_fmaf(p, a.xs[(int64_t)(m0 + tm) * a.kb + b] *
                                                       a.ws[t][(int64_t)((n0 + tn) >> 7) * a.kb + b], acc[t]);
                } else {
                    acc[t] = p;
                }
            }
            if (k0 > 0x7FFFFFFF - 64)
                break;  // the next k0 would pass 32 bits
        }
        if (tm < a.M - m0 && tn < a.N - n0) {
            const int m = m0 + tm, n = n0 + tn;
            float v[2] = {0.0f, 0.0f};
#pragma unroll
            for (int t = 0; t < MATS; ++t) {
                v[t] = (float)acc[t];
                if constexpr (row_scaled(MODE))
                    if (a.K > 0)
                        v[t] *= a.xs[m] * a.ws[t][n];
            }
            put(a, finish<GATED>(a, v[0], v[1], m, n), m, n);
        }
    }
}

}  // namespace skg

namespace skg_host {
namespace {

const void *any_fn(int mode, bool gated)
{
    using namespace skg;
    static const void *const fn[4][2] = {
        {(const void *)&linear_any_kernel<0, false>, (const void *)&linear_any_kernel<0, true>},
        {(const void *)&linear_any_kernel<1, false>, (const void *)&linear_any_kernel<1, true>},
        {(const void *)&linear_any_kernel<2, false>, (const void *)&linear_any_kernel<2, true>},
        {(const void *)&linear_any_kernel<3, false>, (const void *)&linear_any_kernel<3, true>}};
    return fn[mode][gated];
}

// A launch holds fewer than 2^32 threads; blocks here have at most 512.
constexpr int64_t kMaxBlocks = 1 << 22;

struct Choice {
    const void *fn;
    int64_t nt, mt;  // blocks along N and M
    int waves;
    skinny_linear_plan_t plan;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The kernel whose estimated time, in microseconds, is least. The estimate of a streaming
// kernel has three parts: one for the bytes of W and x (22.5 MB/us is a coefficient of the
// fit, not a rate of the memory); the bytes that the fullest compute unit takes into LDS, at
// 97.5 KB/us; and the round trips of 0.93 us that its waves wait for one after another (a
// ring of two stages hides a part of them). A part of all three
// is paid beside the largest, since they overlap incompletely, and each turn of blocks
// adds its start and the sum of its waves. That of a tiled kernel is its time per stage
// and the bytes of its outputs, which all blocks store together.
// The constants were fitted to the times of some 80 kernels at 1228 sizes of each type (K
// 512 to 8192, N 256 to 12576, M 17 to 4096): the choice takes 2.0% longer than the best of
// all kernels on average and 7% at the 90th percentile.
Choice choose(int mode, bool gated, bool exact, int M, int N, int64_t kbytes, int cus)
{
    const int mats = gated ? 2 : 1;
    const double stages = (double)ceil_div(kbytes, 128);
    const double hbm = ((double)mats * N + M) * (double)kbytes / 22.5e6;
    const double out = (double)M * N * 2.0 / 14.6e6;
    Choice best{};
    double least = 0.0;
    auto offer = [&](const Choice &c, double us) {
        if (!best.fn || us < least) {
            best = c;
            least = us;
        }
    };
    StreamKernel s[kStreamMost];
    const int ns = mode == 0   ? stream_kernels_bf16(M, gated, exact, s)
                   : mode == 1 ? stream_kernels_row(M, gated, exact, s)
                   : mode == 2 ? stream_kernels_block(M, gated, exact, s)
                               : stream_kernels_int8(M, gated, s);
    for (int i = 0; i < ns; ++i) {
        const StreamKernel &k = s[i];
        const Choice c{k.fn, ceil_div(N, k.nb), ceil_div(M, k.bm), k.waves,
                       {SKINNY_LINEAR_STREAM, k.nb, k.bm, k.waves, k.ring, i, 0}};
        const double per_cu = (double)ceil_div(c.nt * c.mt, cus);
        double at_once = 163840 / k.lds < 32 / k.waves ? 163840 / k.lds : 32 / k.waves;
        const double turns = std::ceil((double)(c.nt * c.mt) / (cus * at_once));
        if (at_once > per_cu)
            at_once = per_cu;
        const double lds = per_cu * stages * k.stage / 97500.0;
        const double trips = 0.932 * std::ceil(stages * per_cu / (k.waves * at_once * (1.0 + 1.1 * (k.ring - 1))));
        double most = hbm > lds ? hbm : lds;
        most = most > trips ? most : trips;
        offer(c, 3.0 + most + 0.2 * (hbm + lds + trips) + turns * (0.344 + 0.0292 * k.waves * k.tiles));
    }
    best.plan.count = ns;
    if (M <= 16)  // W once: a tile of many rows only adds work
        return best;
    TileKernel t[kTileMost];
    const int ntk = mode == 0   ? tile_kernels_bf16(gated, exact, t)
                    : mode == 1 ? tile_kernels_row(gated, exact, t)
                    : mode == 2 ? tile_kernels_block(gated, exact, t)
                                : tile_kernels_int8(gated, t);
    for (int i = 0; i < ntk; ++i) {
        const TileKernel &k = t[i];
        const Choice c{k.fn, ceil_div(N, k.nb), ceil_div(M, k.bm), k.waves,
                       {SKINNY_LINEAR_TILE, k.nb, k.bm, k.waves, 0, ns + i, 0}};
        const double per_cu = (double)ceil_div(c.nt * c.mt, cus);
        offer(c, 5.5 + per_cu * (0.5 + stages * k.stage_us) + out);
    }
    best.plan.count = ns + ntk;
    return best;
}

// The type of x and W.
enum Type { kTypeBf16, kTypeE4m3, kTypeInt8 };

int validate(const skinny_linear_t *p, Type type)
{
    return type == kTypeInt8 ? validate_linear_int8(p) : validate_linear(p, type == kTypeE4m3);
}

int mode_of(const skinny_linear_t &p, Type type) { return type == kTypeInt8 ? (int)skg::kInt8Row : p.scales; }

// The kernel of a checked call with outputs; fn is null for the element-wise one.
Choice plan_of(const skinny_linear_t &p, Type type, int cus)
{
    const bool bytes = type != kTypeBf16;
    Choice c{};
    if (linear_vector_ok(p, bytes))
        c = choose(mode_of(p, type), p.W1 != nullptr, p.out_f32 != 0, p.M, p.N, (int64_t)p.K * (bytes ? 1 : 2), cus);
    if (!c.fn || c.nt * c.mt > kMaxBlocks)
        c = Choice{nullptr, 0, 0, 4, {SKINNY_LINEAR_ELEMENTS, 16, 16, 4, 0, -1, 0}};
    return c;
}

int run_linear(const skinny_linear_t *p, Type type, hipStream_t stream)
{
    int st = validate(p, type);
    if (st != SKINNY_OK || p->M == 0 || p->N == 0)
        return st;
    int cus = 0;
    st = ops_device(&cus);
    if (st != SKINNY_OK)
        return st;
    const int mode = mode_of(*p, type);
    const bool gated = p->W1 != nullptr;
    skg::LinArgs a{};
    a.x = static_cast<const uint8_t *>(p->x);
    a.w[0] = static_cast<const uint8_t *>(p->W0);
    a.w[1] = static_cast<const uint8_t *>(p->W1);
    a.xs = p->x_scale;
    a.ws[0] = p->w0_scale;
    a.ws[1] = p->w1_scale;
    a.bias[0] = static_cast<const uint16_t *>(p->bias0);
    a.bias[1] = static_cast<const uint16_t *>(p->bias1);
    a.res = static_cast<const uint16_t *>(p->residual);
    a.y = p->y;
    a.ldx = p->ldx * (type == kTypeBf16 ? 2 : 1);
    a.ldr = p->ldr;
    a.ldy = p->ldy;
    a.M = p->M;
    a.N = p->N;
    a.K = p->K;
    a.kb = (int)(((int64_t)p->K + 127) / 128);
    a.act = p->act;
    a.out_f32 = p->out_f32;

    const Choice c = plan_of(*p, type, cus);
    if (!c.fn) {  // the element-wise kernel loops over its tiles, so it takes any size
        int nt = (int)(((int64_t)a.N + 15) / 16);
        int64_t tiles = (((int64_t)a.M + 15) / 16) * nt;
        void *args[] = {&a, &tiles, &nt};
        return ops_launch(any_fn(mode, gated), dim3((unsigned)(tiles < (1 << 20) ? tiles : 1 << 20)), 256, args,
                          stream);
    }
    int nt = (int)c.nt, mt = (int)c.mt;
    void *args[] = {&a, &nt, &mt};
    return ops_launch(c.fn, dim3((unsigned)(c.nt * c.mt)), c.waves * 64, args, stream);
}

int default_plan(const skinny_linear_t *p, Type type, int32_t cus, skinny_linear_plan_t *out)
{
    const int st = validate(p, type);
    if (st != SKINNY_OK)
        return st;
    if (p->M == 0 || p->N == 0)
        return SKINNY_ERR_INVALID_ARG;
    *out = plan_of(*p, type, cus).plan;
    return SKINNY_OK;
}

}  // namespace
}  // namespace skg_host

extern "C" {

int skinny_linear_bf16(const skinny_linear_t *args, hipStream_t stream)
{
    return skg_host::run_linear(args, skg_host::kTypeBf16, stream);
}

int skinny_linear_fp8(const skinny_linear_t *args, hipStream_t stream)
{
    return skg_host::run_linear(args, skg_host::kTypeE4m3, stream);
}

int skinny_linear_int8(const skinny_linear_t *args, hipStream_t stream)
{
    return skg_host::run_linear(args, skg_host::kTypeInt8, stream);
}

int skinny_linear_default_plan(const skinny_linear_t *args, int32_t compute_units, skinny_linear_plan_t *out)
{
    if (!args || !out || compute_units < 1)
        return SKINNY_ERR_INVALID_ARG;
    return skg_host::default_plan(args, args->scales ? skg_host::kTypeE4m3 : skg_host::kTypeBf16, compute_units, out);
}

int skinny_linear_int8_default_plan(const skinny_linear_t *args, int32_t compute_units, skinny_linear_plan_t *out)
{
    if (!args || !out || compute_units < 1)
        return SKINNY_ERR_INVALID_ARG;
    return skg_host::default_plan(args, skg_host::kTypeInt8, compute_units, out);
}

}  // extern "C"

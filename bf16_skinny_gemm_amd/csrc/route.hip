// The router of a mixture-of-experts layer (include/skinny_moe.h): scores, the k best
// experts of each token, and their weights.
//
// One wave per token, lane l holding the experts l * V .. l * V + V - 1, so that of equal
// ranks the lowest lane has the lowest index. Ranks are turned into unsigned integers of the
// same order (NaN above everything, 0 for what is out), k times the wave's largest is found
// and taken out. Without a bias the rank is the logit itself: 32 bits, and no score but those
// of the chosen is computed. With one it is score + bias in float64, which is as good as
// exact: in float32 two experts whose scores lie within a rounding of each other would
// change places, and so the choice.
//
// A prompt is bound by instructions, one token by the launch: of 4.5 us for 1 x 288, k 8, the
// empty kernel is 2. 8191 x 256, sigmoid, k 8, calls back to back: the logits alone 7.9 us
// (1.1 TB/s), most of it the eight rounds, each a maximum over the wave for one token's four values a
// lane; with a bias 13.2, of which float64's exponentials and quotients are the 5; with four of
// eight groups 17.5 (one lane a group: a tenth more). A ranking in float32 that goes to float64
// only where two ranks lie close gained 8% and was not worth its second path. Several tokens
// a wave would share the rounds' steps; that is not built.
#include "ops_host.hpp"

#include <cstdint>
#include <type_traits>

#include "ops_device.hpp"
#include "validate_moe.hpp"

namespace skg {

struct RouteArgs {
    const float *logits, *bias;
    int32_t *ids;
    float *weights;
    int64_t ldl;
    int M, E, k, groups, kept, renormalize;
    float scale;
};

// Unsigned integers in the order of the values, NaN first; -0 is 0.
__device__ __forceinline__ unsigned order_of(float v)
{
    const unsigned b = __builtin_bit_cast(unsigned, v + 0.0f);
    return v != v ? ~0u : b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ unsigned long long order_of(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v + 0.0);
    return v != v ? ~0ull : b >> 63 ? ~b : b | 0x8000000000000000ull;
}

__device__ __forceinline__ float value_of(unsigned o)
{
    return __builtin_bit_cast(float, o >> 31 ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ double value_of(unsigned long long o)
{
    return __builtin_bit_cast(double, o >> 63 ? o & 0x7FFFFFFFFFFFFFFFull : ~o);
}

template <int CTRL>
__device__ __forceinline__ unsigned dpp_max(unsigned v)
{
    const unsigned o = (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
    return o > v ? o : v;
}

// The wave's largest, as a scalar. All lanes take part.
__device__ __forceinline__ unsigned wave_max(unsigned v)
{
    v = dpp_max<0xB1>(v);   // lane ^ 1
    v = dpp_max<0x4E>(v);   // lane ^ 2
    v = dpp_max<0x141>(v);  // the other quad of each 8 lanes
    v = dpp_max<0x140>(v);  // the other half of each 16 lanes
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 64; i += 16) {
        const unsigned o = (unsigned)__builtin_amdgcn_readlane((int)v, i);
        m = o > m ? o : m;
    }
    return m;
}

// The lanes that hold the wave's largest.
__device__ __forceinline__ unsigned long long holders(unsigned key) { return __ballot(key == wave_max(key)); }

__device__ __forceinline__ unsigned long long holders(unsigned long long key)
{
    const unsigned hi = (unsigned)(key >> 32);
    const bool in = hi == wave_max(hi);
    const unsigned long long b = __ballot(in);
    if (__popcll(b) == 1)
        return b;
    const unsigned lo = in ? (unsigned)key : 0;
    const unsigned most = wave_max(lo);  // by all lanes: not behind the && below
    return __ballot(in && lo == most);
}

template <typename T>
__device__ __forceinline__ T wave_add(T v)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        v += __shfl_xor(v, d, 64);
    return v;
}

__device__ __forceinline__ float wave_top(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        v = __builtin_fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}

constexpr int kRouteWaves = 4;

template <int V, bool SOFTMAX, bool BIAS>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteArgs a)
{
    using key_t = std::conditional_t<BIAS, unsigned long long, unsigned>;
    __shared__ key_t keys[kRouteWaves][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kRouteWaves + wave;
    if (row >= a.M)
        return;  // waves do not wait for one another below
    const float *logits = a.logits + row * a.ldl;
    const int e0 = lane * V;
    float x[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        x[v] = e0 + v < a.E ? logits[e0 + v] : -__builtin_inff();

    // softmax: the largest logit, and the sum where all of it is needed
    float top = 0.0f, sum = 1.0f;
    double sum64 = 1.0;
    if constexpr (SOFTMAX) {
        float t = x[0];
#pragma unroll
        for (int v = 1; v < V; ++v)
            t = __builtin_fmaxf(t, x[v]);
        top = wave_top(t);
        if (top == -__builtin_inff())
            top = 0.0f;  // every exponential is 0
        if constexpr (BIAS) {
            double s = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                s += exp((double)x[v] - (double)top);
            sum64 = wave_add(s);
            sum = (float)sum64;
        } else if (!a.renormalize) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v)
                s += expf(x[v] - top);
            sum = wave_add(s);
        }
    }

    key_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if constexpr (BIAS) {
            double s;
            if constexpr (SOFTMAX) {
                s = exp((double)x[v] - (double)top);
                s = s == 0.0 ? 0.0 : s / sum64;
            } else {
                s = 1.0 / (1.0 + exp(-(double)x[v]));
            }
            key[v] = e0 + v < a.E ? order_of(s + (double)a.bias[e0 + v < a.E ? e0 + v : 0]) : 0;
        } else {
            key[v] = e0 + v < a.E ? order_of(x[v]) : 0;
        }
    }

    if (a.groups > 1) {
        // `sub` lanes look through each group; then the groups are ranked against one another
        const int size = a.E / a.groups, shift = __builtin_clz((unsigned)a.groups - 1) - 26, sub = 1 << shift;
#pragma unroll
        for (int v = 0; v < V; ++v)
            keys[wave][e0 + v] = key[v];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
        const int group = lane >> shift;
        key_t best = 0, second = 0;  // of a group's ranks; the second only with a bias
        auto add = [&](key_t b, key_t s) {
            if constexpr (BIAS) {
                const key_t less = b < best ? b : best, more = s > second ? s : second;
                second = less > more ? less : more;
            }
            best = b > best ? b : best;
        };
        if (group < a.groups)
            for (int i = lane & (sub - 1); i < size; i += sub)
                add(keys[wave][group * size + i], 0);
        for (int d = 1; d < sub; d *= 2) {
            const key_t b = __shfl_xor(best, d, 64), s = BIAS ? __shfl_xor(second, d, 64) : 0;
            add(b, s);
        }
        if constexpr (BIAS)
            if (group < a.groups && size > 1)
                best = order_of(value_of(best) + value_of(second));
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
            key_t o;
            if constexpr (BIAS)
                o = (unsigned long long)(unsigned)__builtin_amdgcn_readlane((int)(best >> 32), g << shift) << 32 |
                    (unsigned)__builtin_amdgcn_readlane((int)best, g << shift);
            else
                o = (unsigned)__builtin_amdgcn_readlane((int)best, g << shift);
            before += o > best || (o == best && g < group);
        }
        const unsigned long long in = __ballot(group < a.groups && before < a.kept);  // a group's lanes alike
        // e / size without a division: e < 1024 and size <= 1024, so 2^20 / size rounded up
        // is close enough
        const unsigned inverse = ((1u << 20) + size - 1) / (unsigned)size;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (e0 + v < a.E && !(in >> (((unsigned)(e0 + v) * inverse >> 20) << shift) & 1))
                key[v] = 0;
    }

    int mine = 0;  // lane j: the j-th expert
    for (int j = 0; j < a.k; ++j) {
        key_t best = key[0];
        int at = 0;
#pragma unroll
        for (int v = 1; v < V; ++v)
            if (key[v] > best) {
                best = key[v];
                at = v;
            }
        const int from = __builtin_ctzll(holders(best));
        const int e = __builtin_amdgcn_readlane(e0 + at, from);
        mine = lane == j ? e : mine;
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = e0 + v == e ? 0 : key[v];
    }

    const float l = lane < a.k ? logits[mine] : 0.0f;
    if (a.renormalize) {
        // The chosen may all lie far below the row's largest (with a bias, or as sigmoids), where
        // float32 holds little or nothing of their scores: what these have in common, the
        // exponential of the largest chosen logit, leaves the quotients first. Below exp(-745),
        // the least of float64, scores are 0: masks of the lowest finite value leave nothing,
        // as those of -infinity.
        float most;
        if constexpr (BIAS)
            most = value_of(wave_max(lane < a.k ? order_of(l) : 0u));
        else  // the first choice
            most = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, l)));
        const float below = SOFTMAX ? most - top : most;
        if (below >= -745.0f && below <= 0.0f)
            top = most;
    }
    float w = 0.0f;
    if (lane < a.k) {
        if constexpr (SOFTMAX) {
            w = expf(l - top);
        } else {
            const float t = expf(-__builtin_fabsf(l));  // the other way round, exp(-l) overflows below -88
            w = (l < 0.0f ? expf(l - top) : 1.0f) / (1.0f + t);
        }
    }
    if (a.renormalize) {
        const float all = wave_add(w);
        w = all == 0.0f ? 0.0f : w / all;
        if constexpr (SOFTMAX && BIAS)  // NaN in the row, which need not be among the chosen
            w = sum != sum ? sum : w;
    } else if constexpr (SOFTMAX) {
        w = sum == 0.0f ? 0.0f : w / sum;
    }
    if (lane < a.k) {
        a.ids[row * a.k + lane] = mine;
        a.weights[row * a.k + lane] = w * a.scale;
    }
}

}  // namespace skg

namespace skg_host {
namespace {

template <int V>
const void *route_fn_of(int score, bool bias)
{
    using namespace skg;
    static const void *const fn[2][2] = {{(const void *)&route_kernel<V, true, false>, (const void *)&route_kernel<V, true, true>},
                                         {(const void *)&route_kernel<V, false, false>, (const void *)&route_kernel<V, false, true>}};
    return fn[score == SKINNY_SCORE_SIGMOID][bias];
}

const void *route_fn(int per_lane, int score, bool bias)
{
    return per_lane <= 1   ? route_fn_of<1>(score, bias)
           : per_lane <= 2 ? route_fn_of<2>(score, bias)
           : per_lane <= 3 ? route_fn_of<3>(score, bias)
           : per_lane <= 4 ? route_fn_of<4>(score, bias)
           : per_lane <= 6 ? route_fn_of<6>(score, bias)
           : per_lane <= 8 ? route_fn_of<8>(score, bias)
                           : route_fn_of<16>(score, bias);
}

}  // namespace
}  // namespace skg_host

extern "C" int skinny_route(const skinny_route_t *r, hipStream_t stream)
{
    using namespace skg_host;
    int st = validate_route(r);
    if (st != SKINNY_OK || r->M == 0)
        return st;
    int cus = 0;
    st = ops_device(&cus);
    if (st != SKINNY_OK)
        return st;
    skg::RouteArgs a{r->logits, r->bias, r->ids, r->weights, r->ldl, r->M, r->E, r->k, r->groups, r->kept, r->renormalize,
                     r->scale};
    void *args[] = {&a};
    const int64_t blocks = ((int64_t)r->M + skg::kRouteWaves - 1) / skg::kRouteWaves;
    const int64_t gx = blocks < (1 << 20) ? blocks : 1 << 20;
    return ops_launch(route_fn((r->E + 63) / 64, r->score, r->bias != nullptr),
                      dim3((unsigned)gx, (unsigned)((blocks + gx - 1) / gx)), skg::kRouteWaves * 64, args, stream);
}

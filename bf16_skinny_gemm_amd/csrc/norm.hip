// Root-mean-square norm with the residual's addition, to bfloat16 or to e4m3 with
// float32 scales (include/skinny_ops.h).
//
//   h = x + residual,   y = h * w / sqrt(mean(h^2) + eps)
//
// One pass over memory: a row's h and h * w stay in registers between the sum of
// squares and the store, so x, residual and w are read once and y (and h) written once,
// and HBM bounds the kernel. The scale needs no second reduction: the factor 1 / sqrt(..)
// is one positive number per row, so max |y| = max |h * w| times it, and the largest
// magnitude is found together with the sum. It is taken over the bit patterns of |h * w|
// as integers, whose order is that of the values with NaN above infinity: a NaN reaches
// the scale instead of being dropped by a float maximum.
#include "ops_host.hpp"

#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "ops_device.hpp"
#include "validate_ops.hpp"

namespace skg {

constexpr float kE4m3Max = 448.0f;
constexpr float kLeastAmax = 0x1p-100f;  // keeps 1 / scale finite for a row or group of zeros

struct NormArgs {
    const uint16_t *x, *r, *w;
    uint16_t *ro;
    void *y;
    float *scale;
    int64_t ldx, ldr, ldro, ldy;
    int M, D, groups;  // groups: scales per row
    float eps;
};

enum { kOutBf16 = 0, kOutRow = 1, kOutGroup = 2 };

template <int CTRL>
__device__ __forceinline__ unsigned dpp_umax(unsigned v)
{
    const unsigned o = (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
    return o > v ? o : v;
}

// Largest over each 16-lane row, in every lane of it.
__device__ __forceinline__ unsigned umax16(unsigned v)
{
    v = dpp_umax<0xB1>(v);   // lane ^ 1
    v = dpp_umax<0x4E>(v);   // lane ^ 2
    v = dpp_umax<0x141>(v);  // the other quad of each 8 lanes
    return dpp_umax<0x140>(v);
}

__device__ __forceinline__ float lane_f32(float v, int lane)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// The wave's sum, in every lane: 16-lane rows by DPP, then the four rows in fixed order.
__device__ __forceinline__ float wave_sum(float v)
{
    v = group_sum<16>(v);
    return (lane_f32(v, 0) + lane_f32(v, 16)) + (lane_f32(v, 32) + lane_f32(v, 48));
}

__device__ __forceinline__ unsigned wave_umax(unsigned v)
{
    v = umax16(v);
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 64; i += 16) {
        const unsigned o = (unsigned)__builtin_amdgcn_readlane((int)v, i);
        m = o > m ? o : m;
    }
    return m;
}

__device__ __forceinline__ unsigned abs_bits(float v) { return __builtin_bit_cast(unsigned, v) & 0x7FFFFFFFu; }

// scale of the largest |y| (amax >= 0, or NaN).
__device__ __forceinline__ float scale_of(float amax)
{
    const float a = amax < kLeastAmax ? kLeastAmax : amax;  // NaN stays
    return a / kE4m3Max;
}

// q = e4m3((hw * f) * (1 / scale)), f = 1 / rms. The factors stay apart: f / scale overflows
// for rows of rms below 2^-19 whose scale is the least one, and their zeros would turn into
// NaN; 1 / scale is at most 448 * 2^100. |q| <= 448 (1 + 2^-22) by the choice of the scale,
// which rounds to 448, so no clamp is needed. Against a division by the scale the product
// is off by at most 2 * 2^-24: a value on the border of two e4m3 ones may go to the other.
__device__ __forceinline__ unsigned pack_e4m3(float a, float b, float c, float d)
{
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
    return (unsigned)v;
}

// Eight bfloat16 values from p, of which `left` (> 0) exist: the others are 0. NT: with
// the non-temporal hint.
template <bool NT>
__device__ __forceinline__ u32x4 load8(const uint16_t *p, int left)
{
    if (left >= 8) {
        if constexpr (NT)
            return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p));
        else
            return *reinterpret_cast<const u32x4_any *>(p);
    }
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < left)
            v[e >> 1] |= (unsigned)p[e] << (16 * (e & 1));
    return v;
}

template <bool NT>
__device__ __forceinline__ void store8(uint16_t *p, const u32x4 &v, int left)
{
    if (left >= 8) {
        if constexpr (NT)
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any *>(p));
        else
            *reinterpret_cast<u32x4_any *>(p) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < left)
            p[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
}

template <bool NT>
__device__ __forceinline__ void store8(uint8_t *p, const u32x2 &v, int left)
{
    if (left >= 8) {
        if constexpr (NT)
            __builtin_nontemporal_store(v, reinterpret_cast<u32x2_any *>(p));
        else
            *reinterpret_cast<u32x2_any *>(p) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < left)
            p[e] = (uint8_t)(v[e >> 2] >> (8 * (e & 3)));
}

// WPR waves per row, P pieces of 8 columns per lane: covers D <= WPR * 64 * 8 * P. Piece p
// of a lane is p * WPR * 64 + lane, so a wave reads 1 KiB at a time and 16 neighbouring
// lanes hold 128 consecutive columns: a scale group is a 16-lane row. 1 x 4096 with residual
// takes 2.0 us, 8192 x 4096 with residual to e4m3 39.2 us: 6.0 TB/s.
template <int WPR, int P, bool RES, int OUT, bool NT>
__global__ __launch_bounds__(WPR >= 4 ? WPR * 64 : 256) void norm_kernel(NormArgs a)
{
    constexpr int ROWS = WPR >= 4 ? 1 : 4 / WPR;  // rows per block
    constexpr int LANES = WPR * 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int sub = wave / WPR;
    const int t = (wave % WPR) * 64 + lane;
    __shared__ float s_sum[WPR > 1 ? ROWS * WPR : 1];
    __shared__ unsigned s_max[WPR > 1 ? ROWS * WPR : 1];
    // 64-bit rows: M * ld passes 32 bits in a long prompt
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * ROWS + sub;
    const bool live = row < a.M;
    const int64_t rr = live ? row : 0;

    u32x4 xv[P], rv[RES ? P : 1], wv[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = (p * LANES + t) * 8;
        const bool in = live && c < a.D;
        xv[p] = in ? load8<NT>(a.x + rr * a.ldx + c, a.D - c) : u32x4{0, 0, 0, 0};
        if constexpr (RES)
            rv[p] = in ? load8<NT>(a.r + rr * a.ldr + c, a.D - c) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = (p * LANES + t) * 8;
        wv[p] = live && c < a.D ? load8<false>(a.w + c, a.D - c) : u32x4{0, 0, 0, 0};
    }

    float hw[P][8];
    float sum = 0.0f;
    unsigned top[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        top[p] = 0;
        u32x4 ho;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float h0 = lo_f32(xv[p][q]), h1 = hi_f32(xv[p][q]);
            if constexpr (RES) {
                h0 += lo_f32(rv[p][q]);
                h1 += hi_f32(rv[p][q]);
                ho[q] = pack_bf16(h0, h1);
            }
            sum = __builtin_fmaf(h0, h0, sum);
            sum = __builtin_fmaf(h1, h1, sum);
            hw[p][2 * q] = h0 * lo_f32(wv[p][q]);
            hw[p][2 * q + 1] = h1 * hi_f32(wv[p][q]);
            if constexpr (OUT != kOutBf16) {
                const unsigned b0 = abs_bits(hw[p][2 * q]), b1 = abs_bits(hw[p][2 * q + 1]);
                top[p] = b0 > top[p] ? b0 : top[p];
                top[p] = b1 > top[p] ? b1 : top[p];
            }
        }
        if constexpr (RES) {
            const int c = (p * LANES + t) * 8;
            // residual_out may be residual or x: every lane has read this row's pieces it
            // overwrites, and no other lane reads them
            if (live && c < a.D)
                store8<NT>(a.ro + rr * a.ldro + c, ho, a.D - c);
        }
    }
    sum = wave_sum(sum);
    unsigned most = 0;
    if constexpr (OUT == kOutRow) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            most = top[p] > most ? top[p] : most;
        most = wave_umax(most);
    }
    if constexpr (WPR > 1) {
        if (lane == 0) {
            s_sum[wave] = sum;
            if constexpr (OUT == kOutRow)
                s_max[wave] = most;
        }
        __syncthreads();
        sum = s_sum[sub * WPR];
        if constexpr (OUT == kOutRow)
            most = s_max[sub * WPR];
#pragma unroll
        for (int k = 1; k < WPR; ++k) {
            sum += s_sum[sub * WPR + k];
            if constexpr (OUT == kOutRow)
                most = s_max[sub * WPR + k] > most ? s_max[sub * WPR + k] : most;
        }
    }
    if (!live)
        return;
    const float f = 1.0f / __builtin_sqrtf(sum / (float)a.D + a.eps);
    if constexpr (OUT == kOutBf16) {
        uint16_t *y = static_cast<uint16_t *>(a.y) + rr * a.ldy;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = (p * LANES + t) * 8;
            u32x4 o;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                o[q] = pack_bf16(hw[p][2 * q] * f, hw[p][2 * q + 1] * f);
            if (c < a.D)
                store8<NT>(y + c, o, a.D - c);
        }
    } else {
        uint8_t *y = static_cast<uint8_t *>(a.y) + rr * a.ldy;
        float sc = 0.0f, g = 0.0f;
        if constexpr (OUT == kOutRow) {
            sc = scale_of(__builtin_bit_cast(float, most) * f);
            g = 1.0f / sc;
            if (t == 0)
                a.scale[row] = sc;
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = (p * LANES + t) * 8;
            if constexpr (OUT == kOutGroup) {
                sc = scale_of(__builtin_bit_cast(float, umax16(top[p])) * f);
                g = 1.0f / sc;
                if ((lane & 15) == 0 && c < a.D)
                    a.scale[rr * a.groups + (c >> 7)] = sc;
            }
            u32x2 o;
            o[0] = pack_e4m3(hw[p][0] * f * g, hw[p][1] * f * g, hw[p][2] * f * g, hw[p][3] * f * g);
            o[1] = pack_e4m3(hw[p][4] * f * g, hw[p][5] * f * g, hw[p][6] * f * g, hw[p][7] * f * g);
            if (c < a.D)
                store8<NT>(y + c, o, a.D - c);
        }
    }
}

// Rows wider than the registers of a block: one block of 256 threads per row.
// Every value is recomputed from x and residual in each pass, and all stores come in
// the last one, by the thread that alone reads those elements, so the accepted
// overlaps hold here too.
template <bool RES, int OUT>
__global__ __launch_bounds__(256) void norm_any_kernel(NormArgs a)
{
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (row >= a.M)
        return;
    const uint16_t *x = a.x + row * a.ldx;
    const uint16_t *r = RES ? a.r + row * a.ldr : nullptr;
    __shared__ float s_sum[4];
    __shared__ unsigned s_max[4];
    auto h_at = [&](int i) { return RES ? bf16_to_f32(x[i]) + bf16_to_f32(r[i]) : bf16_to_f32(x[i]); };
    float sum = 0.0f;
    unsigned most = 0;
    for (int64_t i = t; i < a.D; i += 256) {
        const float h = h_at((int)i);
        sum = __builtin_fmaf(h, h, sum);
        const unsigned b = abs_bits(h * bf16_to_f32(a.w[i]));
        most = b > most ? b : most;
    }
    sum = wave_sum(sum);
    most = wave_umax(most);
    if (lane == 0) {
        s_sum[wave] = sum;
        s_max[wave] = most;
    }
    __syncthreads();
    sum = ((s_sum[0] + s_sum[1]) + s_sum[2]) + s_sum[3];
    most = 0;
    for (int k = 0; k < 4; ++k)
        most = s_max[k] > most ? s_max[k] : most;
    const float f = 1.0f / __builtin_sqrtf(sum / (float)a.D + a.eps);
    auto store_h = [&](int i, float h) {
        if constexpr (RES)
            a.ro[row * a.ldro + i] = f32_to_bf16(h);
    };
    if constexpr (OUT == kOutBf16) {
        uint16_t *y = static_cast<uint16_t *>(a.y) + row * a.ldy;
        for (int64_t i = t; i < a.D; i += 256) {
            const float h = h_at((int)i);
            store_h((int)i, h);
            y[i] = f32_to_bf16(h * bf16_to_f32(a.w[i]) * f);
        }
    } else {
        uint8_t *y = static_cast<uint8_t *>(a.y) + row * a.ldy;
        if constexpr (OUT == kOutRow) {
            const float sc = scale_of(__builtin_bit_cast(float, most) * f), g = 1.0f / sc;
            if (t == 0)
                a.scale[row] = sc;
            for (int64_t i = t; i < a.D; i += 256) {
                const float h = h_at((int)i);
                store_h((int)i, h);
                y[i] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(h * bf16_to_f32(a.w[i]) * f * g, 0.0f, 0, false);
            }
        } else {
            // a wave takes a group of 128 columns, two per lane
            for (int64_t g0 = wave; g0 < a.groups; g0 += 4) {
                float h[2], v[2];
                unsigned top = 0;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int64_t i = g0 * 128 + k * 64 + lane;
                    h[k] = i < a.D ? h_at((int)i) : 0.0f;
                    v[k] = i < a.D ? h[k] * bf16_to_f32(a.w[i]) : 0.0f;
                    const unsigned b = abs_bits(v[k]);
                    top = b > top ? b : top;
                }
                const float sc = scale_of(__builtin_bit_cast(float, wave_umax(top)) * f), g = 1.0f / sc;
                if (lane == 0)
                    a.scale[row * a.groups + g0] = sc;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int64_t i = g0 * 128 + k * 64 + lane;
                    if (i < a.D) {
                        store_h((int)i, h[k]);
                        y[i] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[k] * f * g, 0.0f, 0, false);
                    }
                }
            }
        }
    }
}

}  // namespace skg

namespace skg_host {

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_mu;
std::atomic<int> g_state[kMaxDevices];  // 0: not asked; > 0: gfx950 with that many CUs; < 0: an error

template <int WPR, int P, bool NT>
const void *norm_fn_of(bool res, int out)
{
    using namespace skg;
    static const void *const fn[2][3] = {
        {(const void *)&norm_kernel<WPR, P, false, 0, NT>, (const void *)&norm_kernel<WPR, P, false, 1, NT>,
         (const void *)&norm_kernel<WPR, P, false, 2, NT>},
        {(const void *)&norm_kernel<WPR, P, true, 0, NT>, (const void *)&norm_kernel<WPR, P, true, 1, NT>,
         (const void *)&norm_kernel<WPR, P, true, 2, NT>}};
    return fn[res][out];
}

template <int WPR, int P>
const void *norm_fn(bool res, int out, bool nt)
{
    return nt ? norm_fn_of<WPR, P, true>(res, out) : norm_fn_of<WPR, P, false>(res, out);
}

const void *norm_any_fn(bool res, int out)
{
    using namespace skg;
    static const void *const fn[2][3] = {
        {(const void *)&norm_any_kernel<false, 0>, (const void *)&norm_any_kernel<false, 1>,
         (const void *)&norm_any_kernel<false, 2>},
        {(const void *)&norm_any_kernel<true, 0>, (const void *)&norm_any_kernel<true, 1>,
         (const void *)&norm_any_kernel<true, 2>}};
    return fn[res][out];
}

// One block per unit of rows, over two dimensions: a launch holds fewer than 2^32 threads
// along one.
dim3 row_grid(int64_t blocks)
{
    const int64_t x = blocks < (1 << 20) ? blocks : 1 << 20;
    return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}

int run_norm(const skinny_norm_t *n, bool fp8, hipStream_t stream)
{
    int st = validate_norm(n, fp8);
    if (st != SKINNY_OK || n->M == 0 || n->D == 0)
        return st;
    int cus = 0;
    st = ops_device(&cus);
    if (st != SKINNY_OK)
        return st;
    skg::NormArgs a{static_cast<const uint16_t *>(n->x), static_cast<const uint16_t *>(n->residual),
                    static_cast<const uint16_t *>(n->weight), static_cast<uint16_t *>(n->residual_out), n->y,
                    fp8 ? n->scale : nullptr, n->ldx, n->ldr, n->ldro, n->ldy, n->M, n->D,
                    n->group ? (n->D + 127) / 128 : 1, n->eps};
    void *args[] = {&a};
    const bool res = n->residual != nullptr;
    const int out = !fp8 ? skg::kOutBf16 : n->group ? skg::kOutGroup : skg::kOutRow;
    if (n->D > 32768)
        return ops_launch(norm_any_fn(res, out), row_grid(n->M), 256, args, stream);
    const void *fn;
    int wpr;
    const int D = n->D;
    // Beyond the 256 MB that the device's last cache holds, nothing read or written is
    // there for the next kernel: 8192 x 4096 with residual to e4m3 38.9 us with the
    // non-temporal hint on everything, 42.5 without.
    const int64_t bytes = (int64_t)n->M * D * ((res ? 6 : 2) + (fp8 ? 1 : 2));
    const bool nt = bytes > (INT64_C(192) << 20);
    if (D <= 8192 && n->M <= 1024) {
        // few rows: one piece a lane and more waves a row; M = 64 x 4096 3.0 us against 3.5,
        // 512 4.8 against 5, 2048 11.5 against 11.1. At most 1024 x 8192 x 8 bytes: never nt
        if (D <= 512)
            fn = norm_fn_of<1, 1, false>(res, out), wpr = 1;
        else if (D <= 1024)
            fn = norm_fn_of<2, 1, false>(res, out), wpr = 2;
        else if (D <= 2048)
            fn = norm_fn_of<4, 1, false>(res, out), wpr = 4;
        else if (D <= 4096)
            fn = norm_fn_of<8, 1, false>(res, out), wpr = 8;
        else
            fn = norm_fn_of<16, 1, false>(res, out), wpr = 16;
    } else if (D <= 512) {
        fn = norm_fn<1, 1>(res, out, nt), wpr = 1;
    } else if (D <= 1024) {
        fn = norm_fn<1, 2>(res, out, nt), wpr = 1;
    } else if (D <= 2048) {
        fn = norm_fn<2, 2>(res, out, nt), wpr = 2;
    } else if (D <= 4096) {
        fn = norm_fn<4, 2>(res, out, nt), wpr = 4;
    } else if (D <= 8192) {
        fn = norm_fn<8, 2>(res, out, nt), wpr = 8;
    } else if (D <= 16384) {
        fn = norm_fn<16, 2>(res, out, nt), wpr = 16;
    } else {
        fn = norm_fn<16, 4>(res, out, nt), wpr = 16;
    }
    const int rows = wpr >= 4 ? 1 : 4 / wpr;
    return ops_launch(fn, row_grid(((int64_t)n->M + rows - 1) / rows), wpr >= 4 ? wpr * 64 : 256, args, stream);
}

}  // namespace

int ops_device(int *cus)
{
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)hipGetLastError();
        return SKINNY_ERR_UNSUPPORTED;
    }
    int s = g_state[dev].load(std::memory_order_acquire);
    if (s == 0) {
        std::lock_guard<std::mutex> lk(g_mu);
        s = g_state[dev].load(std::memory_order_relaxed);
        if (s == 0) {
            hipDeviceProp_t prop;
            if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
                (void)hipGetLastError();
                return SKINNY_ERR_UNSUPPORTED;
            }
            s = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0
                    ? (prop.multiProcessorCount > 0 ? prop.multiProcessorCount : 1)
                    : SKINNY_ERR_UNSUPPORTED;
            g_state[dev].store(s, std::memory_order_release);
        }
    }
    if (s < 0)
        return s;
    *cus = s;
    return SKINNY_OK;
}

}  // namespace skg_host

extern "C" {

int skinny_rms_norm_bf16(const skinny_norm_t *args, hipStream_t stream)
{
    return skg_host::run_norm(args, false, stream);
}

int skinny_rms_norm_fp8(const skinny_norm_t *args, hipStream_t stream)
{
    return skg_host::run_norm(args, true, stream);
}

}  // extern "C"

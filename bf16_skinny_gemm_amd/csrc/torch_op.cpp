// torch.ops.skinny.linear with its GPU kernel registered in C++: the eager call
// goes from the dispatcher straight to the C ABI (include/skinny_gemm.h), with no
// Python frame in between. vLLM PR #65306 (SM90 skinny GEMM plans), section
// Details, puts the eager overhead of its custom op at 4-7 us per call; the C ABI
// call alone costs about 4 us here (almost all of it HIP's kernel launch), and
// this registration adds the dispatcher and the output allocation to it.
//
// Only argument marshalling lives here: shape, dtype and device checks, the
// output tensor, the current HIP stream. The product runs in the HIP kernels.
// The fake (meta) implementation used for tracing is registered from Python
// (bf16_skinny_gemm_amd/torch_op.py), which this library names as the op's
// Python module.
//
// The operators of include/skinny_ops.h (norms, projections with an epilogue) and
// include/skinny_moe.h (router, experts) are registered below in the same way.
#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/library.h>

#include <climits>

#include "skinny_gemm.h"
#include "skinny_moe.h"
#include "skinny_ops.h"

namespace {

// y[..., N] = x[..., K] . weight[N, K]^T for bfloat16 x with prod(leading dims) = M
// in 1..8 and a contiguous bfloat16 weight on the same GPU. Refusals raise
// ValueError (the calls a router should have sent elsewhere); a refusal by the
// library itself (not gfx950, launch failure) raises RuntimeError.
at::Tensor linear_gpu(const at::Tensor &x, const at::Tensor &weight)
{
    TORCH_CHECK_VALUE(x.scalar_type() == at::kBFloat16 && weight.scalar_type() == at::kBFloat16,
                      "skinny::linear: x and weight must be bfloat16, got ", x.scalar_type(), " and ",
                      weight.scalar_type());
    TORCH_CHECK_VALUE(x.device() == weight.device(), "skinny::linear: x on ", x.device(), ", weight on ",
                      weight.device());
    TORCH_CHECK_VALUE(weight.dim() == 2 && x.dim() >= 1 && x.size(-1) == weight.size(1),
                      "skinny::linear: shapes x ", x.sizes(), " and weight ", weight.sizes(), " do not match");
    TORCH_CHECK_VALUE(weight.is_contiguous(), "skinny::linear: weight must be contiguous");
    const int64_t K = x.size(-1), N = weight.size(0);
    const int64_t M = K > 0 ? x.numel() / K : 0;
    TORCH_CHECK_VALUE(M >= 1 && M <= 8 && x.numel() == M * K,
                      "skinny::linear: the token count prod(x.shape[:-1]) must be 1..8, got x ", x.sizes());
    TORCH_CHECK_VALUE(N <= INT_MAX && K <= INT_MAX, "skinny::linear: N and K must fit in 32 bits");

    c10::DeviceGuard guard(x.device());
    const at::Tensor x2 = x.reshape({M, K}).contiguous();
    std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = N;
    at::Tensor y = at::empty(shape, x.options());
    const hipStream_t stream = c10::hip::getCurrentHIPStream(x.device().index()).stream();
    const int st = skinny_gemm_bf16(x2.data_ptr(), weight.data_ptr(), y.data_ptr(), (int)M, (int)N, (int)K, stream);
    TORCH_CHECK(st == SKINNY_OK, "skinny::linear: skinny_gemm_bf16 returned ", st, " (",
                skinny_gemm_status_string(st), ")");
    return y;
}

at::Tensor linear_cpu(const at::Tensor &x, const at::Tensor &weight)
{
    TORCH_CHECK_VALUE(false, "skinny::linear: runs on gfx950 GPU tensors only, got x on ", x.device(),
                      ", weight on ", weight.device());
    return at::Tensor();
}

// ---- operators of skinny_ops.h ---------------------------------------------------

// The rows of a [..., width] tensor as one [M][width] matrix with a row stride: 2-D
// tensors with unit column stride are taken as they are, others made contiguous.
struct Rows {
    at::Tensor t;  // holds a copy, if one was made, until the launch
    const void *p;
    int64_t M, ld;
};

Rows rows_of(const at::Tensor &t, int64_t width)
{
    if (t.dim() == 2 && (t.stride(1) == 1 || width == 1) && (t.stride(0) >= width || t.size(0) == 1))
        return Rows{at::Tensor(), t.data_ptr(), t.size(0), t.size(0) == 1 ? width : t.stride(0)};
    int64_t M = 1;
    for (int64_t d = 0; d + 1 < t.dim(); ++d)
        M *= t.size(d);
    if (t.is_contiguous())
        return Rows{at::Tensor(), t.data_ptr(), M, width};
    at::Tensor c = t.contiguous();
    const void *p = c.data_ptr();
    return Rows{std::move(c), p, M, width};
}

// An output tensor straight from the caching allocator: the dispatcher's round for it
// took 0.4 us of an eager call's 5.4.
at::Tensor output(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &x)
{
    return at::Tensor(at::detail::empty_cuda(shape, type, x.device(), std::nullopt));
}

// Makes x's device current for the call where it is not.
struct OnDevice {
    std::optional<c10::DeviceGuard> guard;
    explicit OnDevice(const at::Tensor &x)
    {
        if (x.device().index() != c10::hip::current_device())
            guard.emplace(x.device());
    }
};

void check_gpu(const char *op, const at::Tensor &x, const at::Tensor &t, const char *name, at::ScalarType type)
{
    TORCH_CHECK_VALUE(t.scalar_type() == type, op, ": ", name, " must be ", type, ", got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.device() == x.device(), op, ": ", name, " must be on ", x.device(), ", got ", t.device());
}

void check_matrix(const char *op, const at::Tensor &x, at::ScalarType type)
{
    TORCH_CHECK_VALUE(x.scalar_type() == type, op, ": x must be ", type, ", got ", x.scalar_type());
    TORCH_CHECK_VALUE(x.dim() >= 1, op, ": x must have at least one dimension");
}

int32_t size32(const char *op, int64_t v, const char *name)
{
    TORCH_CHECK_VALUE(v <= INT_MAX, op, ": ", name, " must fit in 31 bits, got ", v);
    return (int32_t)v;
}

void check_status(const char *op, int st)
{
    TORCH_CHECK_VALUE(st != SKINNY_ERR_INVALID_ARG, op, ": ", skinny_gemm_status_string(st));
    TORCH_CHECK(st == SKINNY_OK, op, ": ", skinny_gemm_status_string(st));
}

c10::SmallVector<int64_t, 6> with_last(const at::Tensor &x, int64_t last)
{
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = last;
    return shape;
}

// What a norm's call gives: bfloat16, e4m3 with scales per row or per 128 columns, 8-bit
// integers with scales per row of the norm, or of x itself (no weight).
enum class Out { bf16, rows, groups, int8, plain_int8 };

// Outputs: y, scale, new residual (undefined where there is none).
std::tuple<at::Tensor, at::Tensor, at::Tensor> norm_gpu(const char *op, const at::Tensor &x,
                                                        const at::Tensor *residual, const at::Tensor *weight,
                                                        double eps, Out out)
{
    check_matrix(op, x, at::kBFloat16);
    const int64_t D = x.size(-1);
    TORCH_CHECK_VALUE(D > 0, op, ": the width must be above 0");
    if (weight) {
        check_gpu(op, x, *weight, "weight", at::kBFloat16);
        TORCH_CHECK_VALUE(weight->dim() == 1 && weight->size(0) == D && weight->is_contiguous(), op,
                          ": weight must be a contiguous [", D, "], got ", weight->sizes());
    }
    if (residual) {
        check_gpu(op, x, *residual, "residual", at::kBFloat16);
        TORCH_CHECK_VALUE(residual->sizes() == x.sizes(), op, ": residual must have x's shape ", x.sizes(), ", got ",
                          residual->sizes());
    }
    const OnDevice on(x);
    const Rows xr = rows_of(x, D);
    Rows rr{};
    at::Tensor h, scale;
    const at::ScalarType type = out == Out::bf16                       ? at::kBFloat16
                                : out == Out::rows || out == Out::groups ? at::kFloat8_e4m3fn
                                                                       : at::kChar;
    at::Tensor y = output(x.sizes(), type, x);
    skinny_norm_t n{};
    n.x = xr.p;
    n.ldx = xr.ld;
    if (residual) {
        rr = rows_of(*residual, D);
        h = output(x.sizes(), at::kBFloat16, x);
        n.residual = rr.p;
        n.ldr = rr.ld;
        n.residual_out = h.data_ptr();
        n.ldro = D;
    }
    n.weight = weight ? weight->data_ptr() : nullptr;
    n.y = y.data_ptr();
    n.ldy = D;
    n.M = size32(op, xr.M, "the number of rows");
    n.D = size32(op, D, "the width");
    n.eps = (float)eps;
    if (out != Out::bf16) {
        c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end() - 1);
        n.group = out == Out::groups ? 128 : 0;
        if (n.group)
            shape.push_back((D + n.group - 1) / n.group);
        scale = output(shape, at::kFloat, x);
        n.scale = scale.data_ptr<float>();
    }
    const hipStream_t stream = c10::hip::getCurrentHIPStream(x.device().index()).stream();
    check_status(op, out == Out::bf16         ? skinny_rms_norm_bf16(&n, stream)
                     : out == Out::int8       ? skinny_rms_norm_int8(&n, stream)
                     : out == Out::plain_int8 ? skinny_quantize_int8(&n, stream)
                                              : skinny_rms_norm_fp8(&n, stream));
    return {y, scale, h};
}

Out fp8_out(const char *op, int64_t group)
{
    TORCH_CHECK_VALUE(group == 0 || group == 128, op, ": group must be 0 (per row) or 128, got ", group);
    return group ? Out::groups : Out::rows;
}

at::Tensor rms_norm_gpu(const at::Tensor &x, const at::Tensor &weight, double eps)
{
    return std::get<0>(norm_gpu("skinny::rms_norm", x, nullptr, &weight, eps, Out::bf16));
}

std::tuple<at::Tensor, at::Tensor> add_rms_norm_gpu(const at::Tensor &x, const at::Tensor &residual,
                                                    const at::Tensor &weight, double eps)
{
    auto r = norm_gpu("skinny::add_rms_norm", x, &residual, &weight, eps, Out::bf16);
    return {std::get<0>(r), std::get<2>(r)};
}

std::tuple<at::Tensor, at::Tensor> rms_norm_fp8_gpu(const at::Tensor &x, const at::Tensor &weight, double eps,
                                                    int64_t group)
{
    const char *op = "skinny::rms_norm_fp8";
    auto r = norm_gpu(op, x, nullptr, &weight, eps, fp8_out(op, group));
    return {std::get<0>(r), std::get<1>(r)};
}

std::tuple<at::Tensor, at::Tensor, at::Tensor> add_rms_norm_fp8_gpu(const at::Tensor &x, const at::Tensor &residual,
                                                                    const at::Tensor &weight, double eps,
                                                                    int64_t group)
{
    const char *op = "skinny::add_rms_norm_fp8";
    return norm_gpu(op, x, &residual, &weight, eps, fp8_out(op, group));
}

std::tuple<at::Tensor, at::Tensor> quantize_int8_gpu(const at::Tensor &x)
{
    auto r = norm_gpu("skinny::quantize_int8", x, nullptr, nullptr, 0.0, Out::plain_int8);
    return {std::get<0>(r), std::get<1>(r)};
}

std::tuple<at::Tensor, at::Tensor> rms_norm_int8_gpu(const at::Tensor &x, const at::Tensor &weight, double eps)
{
    auto r = norm_gpu("skinny::rms_norm_int8", x, nullptr, &weight, eps, Out::int8);
    return {std::get<0>(r), std::get<1>(r)};
}

std::tuple<at::Tensor, at::Tensor, at::Tensor> add_rms_norm_int8_gpu(const at::Tensor &x, const at::Tensor &residual,
                                                                     const at::Tensor &weight, double eps)
{
    return norm_gpu("skinny::add_rms_norm_int8", x, &residual, &weight, eps, Out::int8);
}

using Opt = std::optional<at::Tensor>;

int32_t act_of(const char *op, c10::string_view act)
{
    if (act == "none")
        return SKINNY_ACT_NONE;
    if (act == "relu")
        return SKINNY_ACT_RELU;
    if (act == "gelu")
        return SKINNY_ACT_GELU;
    if (act == "gelu_tanh")
        return SKINNY_ACT_GELU_TANH;
    if (act == "silu")
        return SKINNY_ACT_SILU;
    TORCH_CHECK_VALUE(false, op, ": act must be none, relu, gelu, gelu_tanh or silu, got ", act);
    return -1;
}

struct Side {  // one weight with what belongs to it
    const at::Tensor &w;
    const at::Tensor *scale;
    const Opt &bias;
};

// The scales of x and of one weight: 1-D w_scale = per row, 2-D = per 128 x 128 block.
void check_scales(const char *op, const at::Tensor &x, const at::Tensor &xs, const at::Tensor &ws, int64_t M,
                  int64_t N, int64_t K, bool blocks)
{
    check_gpu(op, x, xs, "x_scale", at::kFloat);
    check_gpu(op, x, ws, "the weight's scale", at::kFloat);
    TORCH_CHECK_VALUE(xs.is_contiguous() && ws.is_contiguous(), op, ": scales must be contiguous");
    const int64_t kb = (K + 127) / 128, nb = (N + 127) / 128;
    if (blocks) {
        TORCH_CHECK_VALUE(ws.dim() == 2 && ws.size(0) == nb && ws.size(1) == kb && xs.dim() >= 1 &&
                              xs.size(-1) == kb && xs.numel() == M * kb,
                          op, ": block scales must be [", M, ", ", kb, "] for x and [", nb, ", ", kb,
                          "] for the weight, got ", xs.sizes(), " and ", ws.sizes());
    } else {
        TORCH_CHECK_VALUE(ws.dim() == 1 && ws.numel() == N && xs.numel() == M, op, ": row scales must be [", M,
                          "] for x and [", N, "] for the weight, got ", xs.sizes(), " and ", ws.sizes());
    }
}

at::Tensor linear_any(const char *op, at::ScalarType type, const at::Tensor &x, const at::Tensor *xs,
                      const Side *sides, int mats, const Opt &residual, c10::string_view act, bool out_f32)
{
    check_matrix(op, x, type);
    const int64_t K = x.size(-1);
    const at::Tensor &w0 = sides[0].w;
    TORCH_CHECK_VALUE(w0.dim() == 2, op, ": the weight must be [N, K], got ", w0.sizes());
    const int64_t N = w0.size(0);
    const OnDevice on(x);
    const Rows xr = rows_of(x, K);
    skinny_linear_t a{};
    a.M = size32(op, xr.M, "the number of rows");
    a.N = size32(op, N, "N");
    a.K = size32(op, K, "K");
    a.act = act_of(op, act);
    a.x = xr.p;
    a.ldx = xr.ld;
    for (int i = 0; i < mats; ++i) {
        const Side &s = sides[i];
        check_gpu(op, x, s.w, "the weight", type);
        TORCH_CHECK_VALUE(s.w.dim() == 2 && s.w.size(0) == N && s.w.size(1) == K && s.w.is_contiguous(), op,
                          ": weights must be contiguous [", N, ", ", K, "], got ", s.w.sizes());
        (i ? a.W1 : a.W0) = s.w.data_ptr();
        if (xs) {
            const bool blocks = type == at::kFloat8_e4m3fn && sides[0].scale->dim() == 2;
            check_scales(op, x, *xs, *s.scale, xr.M, N, K, blocks);
            a.scales = blocks ? SKINNY_SCALES_BLOCK : SKINNY_SCALES_ROW;
            a.x_scale = xs->data_ptr<float>();
            (i ? a.w1_scale : a.w0_scale) = s.scale->data_ptr<float>();
        }
        if (s.bias) {
            check_gpu(op, x, *s.bias, "bias", at::kBFloat16);
            TORCH_CHECK_VALUE(s.bias->dim() == 1 && s.bias->size(0) == N && s.bias->is_contiguous(), op,
                              ": bias must be a contiguous [", N, "], got ", s.bias->sizes());
            (i ? a.bias1 : a.bias0) = s.bias->data_ptr();
        }
    }
    TORCH_CHECK_VALUE(mats == 1 || (N > 0 && K > 0) || xr.M == 0, op, ": the gated form needs N and K above 0");
    Rows rr{};
    const auto shape = with_last(x, N);
    if (residual) {
        check_gpu(op, x, *residual, "residual", at::kBFloat16);
        TORCH_CHECK_VALUE(residual->sizes() == at::IntArrayRef(shape), op, ": residual must be ", at::IntArrayRef(shape),
                          ", got ", residual->sizes());
        rr = rows_of(*residual, N);
        a.residual = rr.p;
        a.ldr = rr.ld;
    }
    at::Tensor y = output(shape, out_f32 ? at::kFloat : at::kBFloat16, x);
    a.y = y.data_ptr();
    a.ldy = N;
    a.out_f32 = out_f32;
    const hipStream_t stream = c10::hip::getCurrentHIPStream(x.device().index()).stream();
    check_status(op, type == at::kBFloat16 ? skinny_linear_bf16(&a, stream)
                     : type == at::kChar   ? skinny_linear_int8(&a, stream)
                                           : skinny_linear_fp8(&a, stream));
    return y;
}

at::Tensor linear_act_gpu(const at::Tensor &x, const at::Tensor &weight, const Opt &bias, const Opt &residual,
                          c10::string_view act, bool out_f32)
{
    const Side s[] = {{weight, nullptr, bias}};
    return linear_any("skinny::linear_act", at::kBFloat16, x, nullptr, s, 1, residual, act, out_f32);
}

at::Tensor linear_gated_gpu(const at::Tensor &x, const at::Tensor &w_gate, const at::Tensor &w_up, const Opt &b_gate,
                            const Opt &b_up, c10::string_view act, bool out_f32)
{
    const Side s[] = {{w_gate, nullptr, b_gate}, {w_up, nullptr, b_up}};
    return linear_any("skinny::linear_gated", at::kBFloat16, x, nullptr, s, 2, std::nullopt, act, out_f32);
}

at::Tensor linear_fp8_gpu(const at::Tensor &x, const at::Tensor &x_scale, const at::Tensor &weight,
                          const at::Tensor &w_scale, const Opt &bias, const Opt &residual, c10::string_view act,
                          bool out_f32)
{
    const Side s[] = {{weight, &w_scale, bias}};
    return linear_any("skinny::linear_fp8", at::kFloat8_e4m3fn, x, &x_scale, s, 1, residual, act, out_f32);
}

at::Tensor linear_gated_fp8_gpu(const at::Tensor &x, const at::Tensor &x_scale, const at::Tensor &w_gate,
                                const at::Tensor &gate_scale, const at::Tensor &w_up, const at::Tensor &up_scale,
                                const Opt &b_gate, const Opt &b_up, c10::string_view act, bool out_f32)
{
    const Side s[] = {{w_gate, &gate_scale, b_gate}, {w_up, &up_scale, b_up}};
    return linear_any("skinny::linear_gated_fp8", at::kFloat8_e4m3fn, x, &x_scale, s, 2, std::nullopt, act, out_f32);
}

at::Tensor linear_int8_gpu(const at::Tensor &x, const at::Tensor &x_scale, const at::Tensor &weight,
                           const at::Tensor &w_scale, const Opt &bias, const Opt &residual, c10::string_view act,
                           bool out_f32)
{
    const Side s[] = {{weight, &w_scale, bias}};
    return linear_any("skinny::linear_int8", at::kChar, x, &x_scale, s, 1, residual, act, out_f32);
}

at::Tensor linear_gated_int8_gpu(const at::Tensor &x, const at::Tensor &x_scale, const at::Tensor &w_gate,
                                 const at::Tensor &gate_scale, const at::Tensor &w_up, const at::Tensor &up_scale,
                                 const Opt &b_gate, const Opt &b_up, c10::string_view act, bool out_f32)
{
    const Side s[] = {{w_gate, &gate_scale, b_gate}, {w_up, &up_scale, b_up}};
    return linear_any("skinny::linear_gated_int8", at::kChar, x, &x_scale, s, 2, std::nullopt, act, out_f32);
}

// ---- operators of skinny_moe.h ---------------------------------------------------

std::tuple<at::Tensor, at::Tensor> route_gpu(const at::Tensor &logits, int64_t k, c10::string_view score, const Opt &bias,
                                             int64_t groups, int64_t kept, bool renormalize, double scale)
{
    const char *op = "skinny::route";
    TORCH_CHECK_VALUE(logits.scalar_type() == at::kFloat && logits.dim() >= 1, op,
                      ": logits must be float32 with at least one dimension, got ", logits.scalar_type(), " ", logits.sizes());
    const int64_t E = logits.size(-1);
    TORCH_CHECK_VALUE(E >= 1 && E <= 1024, op, ": the number of experts must be 1..1024, got ", E);
    TORCH_CHECK_VALUE(score == "softmax" || score == "sigmoid", op, ": score must be softmax or sigmoid, got ", score);
    TORCH_CHECK_VALUE(groups >= 1 && groups <= 64 && E % groups == 0 && kept >= 1 && kept <= groups, op,
                      ": groups must be 1..64 and divide ", E, ", and kept 1..groups, got ", groups, " and ", kept);
    TORCH_CHECK_VALUE(k >= 1 && k <= 64 && k <= kept * (E / groups), op, ": k must be 1..64 and at most ",
                      kept * (E / groups), ", got ", k);
    if (bias) {
        check_gpu(op, logits, *bias, "bias", at::kFloat);
        TORCH_CHECK_VALUE(bias->dim() == 1 && bias->size(0) == E && bias->is_contiguous(), op,
                          ": bias must be a contiguous [", E, "], got ", bias->sizes());
    }
    const OnDevice on(logits);
    const Rows r = rows_of(logits, E);
    const auto shape = with_last(logits, k);
    at::Tensor ids = output(shape, at::kInt, logits), weights = output(shape, at::kFloat, logits);
    skinny_route_t a{};
    a.logits = static_cast<const float *>(r.p);
    a.ldl = r.ld;
    a.bias = bias ? bias->data_ptr<float>() : nullptr;
    a.ids = ids.data_ptr<int32_t>();
    a.weights = weights.data_ptr<float>();
    a.M = size32(op, r.M, "the number of rows");
    a.E = (int32_t)E;
    a.k = (int32_t)k;
    a.score = score == "softmax" ? SKINNY_SCORE_SOFTMAX : SKINNY_SCORE_SIGMOID;
    a.groups = (int32_t)groups;
    a.kept = (int32_t)kept;
    a.renormalize = renormalize;
    a.scale = (float)scale;
    check_status(op, skinny_route(&a, c10::hip::getCurrentHIPStream(logits.device().index()).stream()));
    return {ids, weights};
}

// A stack of contiguous matrices or vectors, one per expert, any distance apart: the
// distance.
int64_t check_stack(const char *op, const at::Tensor &x, const at::Tensor &t, const char *name, at::ScalarType type,
                    at::IntArrayRef shape)
{
    check_gpu(op, x, t, name, type);
    bool inner = t.sizes() == shape;
    int64_t size = 1;
    for (int64_t d = t.dim() - 1; inner && d > 0; --d) {
        inner = t.size(d) == 1 || t.stride(d) == size;
        size *= t.size(d);
    }
    TORCH_CHECK_VALUE(inner, op, ": ", name, " must be ", shape, " with contiguous parts, got ", t.sizes(), " of strides ",
                      t.strides());
    return shape[0] > 1 ? t.stride(0) : size;
}

at::Tensor experts_gpu(const at::Tensor &x, const at::Tensor &ids, const at::Tensor &weights, const at::Tensor &w_gate,
                       const at::Tensor &w_up, const at::Tensor &w_down, const Opt &gate_scale, const Opt &up_scale,
                       const Opt &down_scale, const Opt &residual, c10::string_view act)
{
    const char *op = "skinny::experts";
    check_matrix(op, x, at::kBFloat16);
    const at::ScalarType type = w_gate.scalar_type();
    TORCH_CHECK_VALUE(type == at::kBFloat16 || type == at::kChar || type == at::kFloat8_e4m3fn, op,
                      ": w_gate must be bfloat16, int8 or float8_e4m3fn, got ", type);
    TORCH_CHECK_VALUE(w_gate.dim() == 3, op, ": w_gate must be [E, I, H], got ", w_gate.sizes());
    const int64_t H = x.size(-1), E = w_gate.size(0), I = w_gate.size(1);
    check_gpu(op, x, ids, "ids", at::kInt);
    check_gpu(op, x, weights, "weights", at::kFloat);
    TORCH_CHECK_VALUE(ids.dim() == x.dim() && ids.sizes() == weights.sizes() &&
                          ids.sizes().slice(0, ids.dim() - 1) == x.sizes().slice(0, x.dim() - 1),
                      op, ": ids and weights must be [..., k] beside x ", x.sizes(), ", got ", ids.sizes(), " and ",
                      weights.sizes());
    const int64_t k = ids.size(-1);
    TORCH_CHECK_VALUE(E >= 1 && E <= 1024 && k >= 1 && k <= 32 && H >= 1 && I >= 1, op,
                      ": E must be 1..1024, k 1..32, H and I above 0, got ", E, ", ", k, ", ", H, " and ", I);
    skinny_experts_t a{};
    a.up_stride = check_stack(op, x, w_gate, "w_gate", type, {E, I, H});
    TORCH_CHECK_VALUE(check_stack(op, x, w_up, "w_up", type, {E, I, H}) == a.up_stride, op,
                      ": w_gate and w_up must have the same strides");
    a.down_stride = check_stack(op, x, w_down, "w_down", type, {E, H, I});
    const bool scaled = type != at::kBFloat16;
    TORCH_CHECK_VALUE(gate_scale.has_value() == scaled && up_scale.has_value() == scaled && down_scale.has_value() == scaled,
                      op, ": float8_e4m3fn and int8 weights need a scale each, bfloat16 ones take none");
    a.type = SKINNY_WEIGHTS_BF16;
    if (scaled) {
        const bool blocks = type == at::kFloat8_e4m3fn && gate_scale->dim() == 3;
        const int64_t hb = (H + 127) / 128, ib = (I + 127) / 128;
        a.type = type == at::kChar ? SKINNY_WEIGHTS_INT8_ROW
                 : blocks          ? SKINNY_WEIGHTS_E4M3_BLOCK
                                   : SKINNY_WEIGHTS_E4M3_ROW;
        const c10::SmallVector<int64_t, 3> up = blocks ? c10::SmallVector<int64_t, 3>{E, ib, hb} : c10::SmallVector<int64_t, 3>{E, I};
        const c10::SmallVector<int64_t, 3> down =
            blocks ? c10::SmallVector<int64_t, 3>{E, hb, ib} : c10::SmallVector<int64_t, 3>{E, H};
        a.up_scale_stride = check_stack(op, x, *gate_scale, "gate_scale", at::kFloat, up);
        TORCH_CHECK_VALUE(check_stack(op, x, *up_scale, "up_scale", at::kFloat, up) == a.up_scale_stride, op,
                          ": gate_scale and up_scale must have the same strides");
        a.down_scale_stride = check_stack(op, x, *down_scale, "down_scale", at::kFloat, down);
        a.gate_scale = gate_scale->data_ptr<float>();
        a.up_scale = up_scale->data_ptr<float>();
        a.down_scale = down_scale->data_ptr<float>();
    }
    const OnDevice on(x);
    const Rows xr = rows_of(x, H);
    Rows rr{};
    a.x = xr.p;
    a.ldx = xr.ld;
    const at::Tensor ids_c = ids.contiguous(), weights_c = weights.contiguous();
    a.ids = ids_c.data_ptr<int32_t>();
    a.weights = weights_c.data_ptr<float>();
    a.w_gate = w_gate.data_ptr();
    a.w_up = w_up.data_ptr();
    a.w_down = w_down.data_ptr();
    a.M = size32(op, xr.M, "the number of rows");
    a.E = (int32_t)E;
    a.k = (int32_t)k;
    a.H = size32(op, H, "H");
    a.I = size32(op, I, "I");
    a.act = act_of(op, act);
    if (residual) {
        check_gpu(op, x, *residual, "residual", at::kBFloat16);
        TORCH_CHECK_VALUE(residual->sizes() == x.sizes(), op, ": residual must have x's shape ", x.sizes(), ", got ",
                          residual->sizes());
        rr = rows_of(*residual, H);
        a.residual = rr.p;
        a.ldr = rr.ld;
    }
    at::Tensor y = output(x.sizes(), at::kBFloat16, x);
    if (a.M == 0)
        return y;
    a.y = y.data_ptr();
    a.ldy = H;
    a.workspace_bytes = skinny_experts_workspace_bytes(a.M, a.k, a.E, a.I);
    // freed when the call returns, for later work on this stream only
    const at::Tensor workspace = output({(int64_t)a.workspace_bytes}, at::kByte, x);
    a.workspace = workspace.data_ptr();
    check_status(op, skinny_experts(&a, c10::hip::getCurrentHIPStream(x.device().index()).stream()));
    return y;
}

// CPU tensors: every operator refuses them by name.
void refuse_cpu(const c10::OperatorHandle &op, torch::jit::Stack *)
{
    TORCH_CHECK_VALUE(false, op.operator_name().name, ": runs on gfx950 GPU tensors only");
}

}  // namespace

TORCH_LIBRARY(skinny, m)
{
    m.set_python_module("bf16_skinny_gemm_amd.torch_op");
    m.def("linear(Tensor x, Tensor weight) -> Tensor");
    m.def("rms_norm(Tensor x, Tensor weight, float eps) -> Tensor");
    m.def("add_rms_norm(Tensor x, Tensor residual, Tensor weight, float eps) -> (Tensor, Tensor)");
    m.def("rms_norm_fp8(Tensor x, Tensor weight, float eps, int group) -> (Tensor, Tensor)");
    m.def("add_rms_norm_fp8(Tensor x, Tensor residual, Tensor weight, float eps, int group) "
          "-> (Tensor, Tensor, Tensor)");
    m.def("linear_act(Tensor x, Tensor weight, Tensor? bias=None, Tensor? residual=None, str act='none', "
          "bool out_f32=False) -> Tensor");
    m.def("linear_gated(Tensor x, Tensor w_gate, Tensor w_up, Tensor? b_gate=None, Tensor? b_up=None, "
          "str act='silu', bool out_f32=False) -> Tensor");
    m.def("linear_fp8(Tensor x, Tensor x_scale, Tensor weight, Tensor w_scale, Tensor? bias=None, "
          "Tensor? residual=None, str act='none', bool out_f32=False) -> Tensor");
    m.def("linear_gated_fp8(Tensor x, Tensor x_scale, Tensor w_gate, Tensor gate_scale, Tensor w_up, "
          "Tensor up_scale, Tensor? b_gate=None, Tensor? b_up=None, str act='silu', bool out_f32=False) -> Tensor");
    m.def("quantize_int8(Tensor x) -> (Tensor, Tensor)");
    m.def("rms_norm_int8(Tensor x, Tensor weight, float eps) -> (Tensor, Tensor)");
    m.def("add_rms_norm_int8(Tensor x, Tensor residual, Tensor weight, float eps) -> (Tensor, Tensor, Tensor)");
    m.def("linear_int8(Tensor x, Tensor x_scale, Tensor weight, Tensor w_scale, Tensor? bias=None, "
          "Tensor? residual=None, str act='none', bool out_f32=False) -> Tensor");
    m.def("linear_gated_int8(Tensor x, Tensor x_scale, Tensor w_gate, Tensor gate_scale, Tensor w_up, "
          "Tensor up_scale, Tensor? b_gate=None, Tensor? b_up=None, str act='silu', bool out_f32=False) -> Tensor");
    m.def("route(Tensor logits, int k, str score='softmax', Tensor? bias=None, int groups=1, int kept=1, "
          "bool renormalize=True, float scale=1.0) -> (Tensor, Tensor)");
    m.def("experts(Tensor x, Tensor ids, Tensor weights, Tensor w_gate, Tensor w_up, Tensor w_down, "
          "Tensor? gate_scale=None, Tensor? up_scale=None, Tensor? down_scale=None, Tensor? residual=None, "
          "str act='silu') -> Tensor");
}

TORCH_LIBRARY_IMPL(skinny, CUDA, m)
{
    m.impl("linear", &linear_gpu);
    m.impl("rms_norm", &rms_norm_gpu);
    m.impl("add_rms_norm", &add_rms_norm_gpu);
    m.impl("rms_norm_fp8", &rms_norm_fp8_gpu);
    m.impl("add_rms_norm_fp8", &add_rms_norm_fp8_gpu);
    m.impl("linear_act", &linear_act_gpu);
    m.impl("linear_gated", &linear_gated_gpu);
    m.impl("linear_fp8", &linear_fp8_gpu);
    m.impl("linear_gated_fp8", &linear_gated_fp8_gpu);
    m.impl("quantize_int8", &quantize_int8_gpu);
    m.impl("rms_norm_int8", &rms_norm_int8_gpu);
    m.impl("add_rms_norm_int8", &add_rms_norm_int8_gpu);
    m.impl("linear_int8", &linear_int8_gpu);
    m.impl("linear_gated_int8", &linear_gated_int8_gpu);
    m.impl("route", &route_gpu);
    m.impl("experts", &experts_gpu);
}

TORCH_LIBRARY_IMPL(skinny, CPU, m)
{
    m.impl("linear", &linear_cpu);
    for (const char *op : {"rms_norm", "add_rms_norm", "rms_norm_fp8", "add_rms_norm_fp8", "linear_act",
                           "linear_gated", "linear_fp8", "linear_gated_fp8", "quantize_int8", "rms_norm_int8",
                           "add_rms_norm_int8", "linear_int8", "linear_gated_int8", "route", "experts"})
        m.impl(op, torch::CppFunction::makeFromBoxedFunction<&refuse_cpu>());
}

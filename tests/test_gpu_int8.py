"""The 8-bit integer operators of include/skinny_ops.h against their definitions in 64 bits, on
the GPU.

Tolerances are counted from the roundings: the product's sum is exact, so a projection has the
rounding of the sum to float32, two of the scales, one of each further float32 operation, those
of the activation, and half a step of the output (2^-8 of a bfloat16 value, 2^-24 of a float32
one). An 8-bit value is off by half of its scale, and by the roundings of what it was made from.
"""
from __future__ import annotations

import math

import pytest
import torch

from .int8_choices import CHOICES
from .test_gpu_ops import (BF16, F32, LEAST, act_ref, bits, filled, gen, norm_ref, ops,  # noqa: F401
                           skg, walled, walls_hold)

pytestmark = pytest.mark.gpu

TOP = 127.0
MARK = 0x55


def marked(M, D, ld=None, shift=0):
    """An int8 [M, D] view of row stride ld inside a larger buffer that holds MARK elsewhere."""
    ld = ld or D
    flat = torch.full((M * ld + 64 + shift,), MARK, dtype=torch.int8, device="cuda")
    return flat, flat[32 + shift:32 + shift + M * ld].view(M, ld)[:, :D]


def marks_hold(flat, view):
    inside = torch.zeros(flat.shape, dtype=torch.bool, device="cuda")
    inside.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(True)
    return bool((flat[~inside] == MARK).all())


def ints(M, D, seed, ld=None, shift=0):
    """All values from -128 to 127."""
    view = marked(M, D, ld, shift)[1]
    view.copy_(torch.randint(-128, 128, (M, D), generator=gen(seed), device="cuda", dtype=torch.int8))
    return view


# ---- norm and rows to 8-bit integers -----------------------------------------

def check_norm(skg, M, D, residual=False, *, plain=False, ld=None, shift=0, seed=0, x=None):  # noqa: F811
    g = gen(seed)
    if x is None:
        x = torch.randn(M, D, generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn(M, D, generator=g, device="cuda").to(torch.bfloat16) if residual else None
    w = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    xv = filled(x, ld, shift)
    flat, out = marked(M, D, ld, shift)
    if plain:
        y, rel = x.double(), 4 * F32
        q, scale = skg.quantize_int8(xv, out=out)
    else:
        h, y = norm_ref(x, w, 1e-6, r)
        rel = (D / 2 + 16) * F32  # half the relative error of the sum of squares, and the factors
        hflat, hv = walled(M, D, ld, torch.bfloat16, shift)
        q, scale, *tail = skg.rms_norm(xv, filled(w[None], shift=shift)[0], 1e-6, quant="int8", out=out,
                                       residual=filled(r, ld, shift) if residual else None,
                                       residual_out=hv if residual else None)
        if residual:
            assert walls_hold(hflat, hv)
            assert ((tail[0].double() - h).abs() <= h.abs() * (BF16 + 2 * F32) + 1e-38).all()
    torch.cuda.synchronize()
    assert marks_hold(flat, out) and q.data_ptr() == out.data_ptr()
    s = y.abs().amax(dim=1).clamp_min(LEAST) / TOP
    assert ((scale.double() - s).abs() <= s * rel).all()
    s = scale.double()[:, None]
    # half a step, the roundings of y and those of the two factors of the quotient
    assert ((q.double() * s - y).abs() <= s * (0.5 + 130 * (rel + 4 * F32))).all()
    top = q.int().abs().amax(dim=1)
    assert ((top == 127) | (y.abs().amax(dim=1) < 2 * LEAST)).all()


@pytest.mark.parametrize("D", (1, 7, 8, 64, 127, 128, 512, 520, 1000, 1024, 1537, 2048, 4096, 5000, 8192, 16384, 16392,
                               32768, 33000))
def test_norm_widths(skg, D):  # noqa: F811
    for M in (1, 3, 17):
        for residual in (False, True):
            check_norm(skg, M, D, residual, seed=D + M)
        check_norm(skg, M, D, plain=True, seed=D + M)


@pytest.mark.parametrize("M,D,ld,shift", [(5, 512, 1024, 0), (3, 1000, 1003, 0), (6, 2048, 2048, 1), (2, 4096, 4100, 4),
                                          (9, 136, 137, 3), (1500, 4096, 4099, 0), (7001, 4091, 4091, 1)])
def test_norm_strides_and_alignment(skg, M, D, ld, shift):  # noqa: F811
    check_norm(skg, M, D, True, ld=ld, shift=shift, seed=ld)
    check_norm(skg, M, D, plain=True, ld=ld, shift=shift, seed=ld)


@pytest.mark.parametrize("D", (256, 4096, 999, 40000))
@pytest.mark.parametrize("plain", (False, True))
def test_special_rows(skg, D, plain):  # noqa: F811
    """Rows of zeros, tiny, large, infinite and NaN values; each row by itself."""
    x = torch.randn(8, D, generator=gen(3), device="cuda").to(torch.bfloat16)
    x[1] = 0.0
    x[2] *= 2.0 ** -60
    x[3] *= 2.0 ** 50
    x[4, 5] = float("nan")
    x[5, 5] = float("-inf")
    x[6] = 0.0
    x[6, D - 1] = -3.0
    w = torch.ones(D, device="cuda", dtype=torch.bfloat16)
    q, scale = skg.quantize_int8(x) if plain else skg.rms_norm(x, w, quant="int8")
    fine = [0, 1, 2, 3, 6, 7]
    if plain:
        check_norm(skg, len(fine), D, plain=True, x=x[fine])
    assert (q[1] == 0).all() and math.isclose(float(scale[1]) * TOP, LEAST, rel_tol=1e-6)
    assert int(q[6, D - 1]) == -127 and (q[6, :D - 1] == 0).all()
    assert (q[4:6] == 0).all() and (q[4:6].float() * scale[4:6, None]).isnan().all()
    assert scale[fine].isfinite().all()


def test_in_place(skg):  # noqa: F811
    x, r = (torch.randn(6, 4096, generator=gen(i), device="cuda").to(torch.bfloat16) for i in range(2))
    w = torch.randn(4096, generator=gen(2), device="cuda").to(torch.bfloat16)
    q0, s0, h0 = skg.rms_norm(x, w, residual=r, quant="int8")
    for over in ("residual", "x"):
        xc, rc = x.clone(), r.clone()
        q, s, h = skg.rms_norm(xc, w, residual=rc, quant="int8", residual_out=rc if over == "residual" else xc)
        assert torch.equal(q, q0) and torch.equal(s, s0) and torch.equal(bits(h), bits(h0))


def rows_of_every_value():
    """For each bfloat16 mantissa of the largest value a row of all the smaller ones of eight
    exponents, both signs: half of the largest is 63.5 steps, up to the scale's rounding."""
    m = torch.arange(128, 256, dtype=torch.float64)
    v = (m[:, None] * 2.0 ** -torch.arange(8)).flatten()
    v = torch.cat([v, -v]).expand(128, -1)
    return torch.where(v.abs() <= m[:, None], v, 0.0 * v).to(torch.bfloat16)


@pytest.mark.parametrize("D", (2048, 33000))
@pytest.mark.parametrize("power", (-107, -60, 0, 40, 120))
def test_rows_are_divided_by_their_scale(skg, power, D):  # noqa: F811
    """The quotient is float32's own, so that values half way between two integers go where a
    division puts them; no tolerance."""
    x = torch.zeros(128, D, dtype=torch.bfloat16)
    x[:, :2048] = rows_of_every_value() * 2.0 ** power
    q, scale = (t.cpu() for t in skg.quantize_int8(x.cuda()))
    assert torch.equal(scale, x.float().abs().amax(dim=1) / TOP)
    want = torch.round(x.float() / scale[:, None]).to(torch.int8)
    assert torch.equal(q, want), (int((q != want).sum()), (q != want).nonzero()[:4].tolist())


@pytest.mark.parametrize("D", (2048, 33000))
@pytest.mark.parametrize("residual", (False, True))
def test_norms_are_divided_by_their_scale(skg, residual, D):  # noqa: F811
    """The same of a norm: h is 1 or -1, so that its factor is 1 and y the weight's value."""
    x = torch.ones(3, D, dtype=torch.bfloat16, device="cuda")
    x[1] = -1.0
    x[2, ::2] = -1.0
    h = x.float().cpu()
    r = x * 0.5 if residual else None
    w = torch.zeros(128, D, dtype=torch.bfloat16)
    w[:, :2048] = rows_of_every_value()
    for row in w:
        q, scale = (t.cpu() for t in skg.rms_norm(x - r if residual else x, row.cuda(), 0.0, residual=r, quant="int8")[:2])
        assert torch.equal(scale, (row.float().abs().max() / TOP).expand(3))
        assert torch.equal(q, torch.round(row.float() * h / scale[:, None]).to(torch.int8))


# ---- projections -------------------------------------------------------------

def check_linear(skg, M, N, K, *, gated=False, act="none", bias=False, residual=False, f32=False, ld=None,  # noqa: F811
                 ldy=None, shift=0, seed=0, in_place=False, x=None):
    mats = 2 if gated else 1
    g = gen(seed + 1)
    x = ints(M, K, seed, ld, shift) if x is None else x
    w = [ints(N, K, seed + 2 + i, shift=shift) for i in range(mats)]
    xs = (torch.rand(M, generator=g, device="cuda") + 0.5) / 60
    ws = [(torch.rand(N, generator=g, device="cuda") + 0.5) / 60 / math.sqrt(max(K, 1)) for _ in range(mats)]
    b = [torch.randn(N, generator=g, device="cuda").to(torch.bfloat16) if bias else None for _ in range(mats)]
    r = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16) if residual else None
    odt = torch.float32 if f32 else torch.bfloat16
    oflat, ov = walled(M, N, ldy, odt, 0 if f32 or in_place else shift)
    rv = None
    if in_place:
        ov.copy_(r)
        rv = ov
    elif residual:
        rv = filled(r, ldy, shift)
    y = skg.linear(x, w[0], bias=b[0], residual=rv, act=act, W_up=w[1] if gated else None, bias_up=b[1] if gated else None,
                   x_scale=xs, w_scale=ws[0], w_up_scale=ws[1] if gated else None, out=ov, out_dtype=odt)
    torch.cuda.synchronize()
    assert walls_hold(oflat, ov)
    z, e = [], []
    for i in range(mats):
        v = (x.double() @ w[i].double().t().contiguous()) * xs.double()[:, None] * ws[i].double()
        err = 4 * F32 * v.abs()  # the sum to float32, and the two scales
        if bias:
            v = v + b[i].double()
            err = err + F32 * v.abs()
        z.append(v)
        e.append(err * 1.01 + 1e-30)
    ref = act_ref(z[0], act)
    err = 1.13 * e[0]
    if act != "none":
        # gelu is the widest: (32 + 3 z^2) roundings of its value; the others 32 of |z| or of the value
        err = err + (32 + (3 * z[0] ** 2 if act == "gelu" else 0)) * F32 * ref.abs()
        err = err + (32 * F32 * z[0].abs() if act in ("silu", "gelu_tanh") else 0)
    if gated:
        err = err * z[1].abs() + (ref.abs() + err) * e[1]
        ref = ref * z[1]
        err = err + 2 * F32 * ref.abs()
    if residual:
        ref = ref + r.double()
    err = err + ref.abs() * ((2 if f32 else 1) * F32 + (0 if f32 else BF16)) + 1e-38
    if not f32:
        err = err * (1 + 2 * BF16)  # the rounding is of the value reached, not of the exact one
    bad = ~((y.double() - ref).abs() <= err)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), y[bad][:4].tolist(), ref[bad][:4].tolist())


@pytest.mark.parametrize("M", (1, 2, 5, 8, 9, 16, 17, 32, 33, 48, 64, 65, 100, 129, 200, 300))
def test_rows(skg, M):  # noqa: F811
    check_linear(skg, M, 333, 1040, seed=M, f32=True)
    check_linear(skg, M, 256, 4096, act="silu", bias=True, residual=True, seed=M + 1)


@pytest.mark.parametrize("N", (1, 3, 15, 16, 17, 63, 65, 129, 255, 500, 1025))
def test_widths(skg, N):  # noqa: F811
    for M in (1, 6, 12, 40, 150, 600):
        check_linear(skg, M, N, 528, seed=N + M, bias=True)


@pytest.mark.parametrize("K", (0, 1, 5, 16, 24, 112, 127, 128, 136, 144, 1000, 2064, 8192, 20000, 131056, 131071))
def test_depths(skg, K):  # noqa: F811
    for M in (1, 5, 13, 30, 70, 260) if K < 20000 else (3, 20, 140):
        check_linear(skg, M, 144, K, seed=K + M, f32=M % 2 == 1, residual=True)


@pytest.mark.parametrize("M", (1, 4, 7, 16, 20, 33, 64, 128, 257, 700))
def test_gated(skg, M):  # noqa: F811
    check_linear(skg, M, 320, 1024, gated=True, act="silu", seed=M)
    check_linear(skg, M, 131, 272, gated=True, act="gelu", bias=True, f32=True, seed=M + 1)


@pytest.mark.parametrize("act", ("none", "relu", "gelu", "gelu_tanh", "silu"))
def test_activations(skg, act):  # noqa: F811
    for M in (3, 130):
        check_linear(skg, M, 200, 384, act=act, bias=True, residual=True, f32=True, seed=5)
        check_linear(skg, M, 200, 384, act=act, gated=True, bias=True, seed=6)


@pytest.mark.parametrize("M,N,K,ld,ldy,shift", [(3, 70, 256, 512, 96, 0), (40, 65, 256, 272, 66, 0), (7, 33, 250, 251, 40, 0),
                                               (150, 130, 384, 400, 131, 0), (5, 40, 128, 128, 40, 1), (90, 50, 77, 80, 50, 3)])
def test_strides_and_alignment(skg, M, N, K, ld, ldy, shift):  # noqa: F811
    check_linear(skg, M, N, K, bias=True, residual=True, ld=ld, ldy=ldy, shift=shift, seed=K)
    check_linear(skg, M, N, K, gated=True, act="silu", f32=True, ld=ld, ldy=ldy, shift=shift, seed=K)


@pytest.mark.parametrize("M", (1, 20, 100, 512))
def test_residual_in_place(skg, M):  # noqa: F811
    check_linear(skg, M, 264, 512, act="gelu_tanh", residual=True, in_place=True, ldy=270, seed=M)


@pytest.mark.parametrize("M,N,K", [(1024, 1024, 512), (2048, 1100, 640), (4100, 2048, 256), (1500, 1031, 384),
                                   (700, 2047, 4096)])
def test_large(skg, M, N, K):  # noqa: F811
    check_linear(skg, M, N, K, bias=True, residual=True, seed=M)
    check_linear(skg, M, N // 2, K, gated=True, act="silu", seed=M)


@pytest.mark.parametrize("M", (1, 12, 40, 300))
def test_the_largest_sums(skg, M):  # noqa: F811
    """131071 products of -128 and -128 fill the 32 bits of a sum."""
    K = 131056
    x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((20, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(max(M, 20), device="cuda")
    y = skg.linear(x, w, x_scale=one[:M], w_scale=one[:20], out_dtype=torch.float32)
    assert (y.double() == float(K * 2 ** 14)).all()


@pytest.mark.parametrize("M", (2, 60, 300))
def test_nan_scales_stay_in_their_row(skg, M):  # noqa: F811
    x, w = ints(M, 256, 1), ints(100, 256, 2)
    xs, ws = torch.full((M,), 0.01, device="cuda"), torch.full((100,), 0.01, device="cuda")
    clean = skg.linear(x, w, x_scale=xs, w_scale=ws)
    xs[M - 1] = float("nan")
    y = skg.linear(x, w, x_scale=xs, w_scale=ws)
    assert y[M - 1].isnan().all() and torch.equal(bits(y[:M - 1]), bits(clean[:M - 1]))


def test_long_outputs(skg):  # noqa: F811
    """More outputs than 31 bits hold: rows at both ends."""
    M, N, K = 70001, 32768, 64
    x, w = ints(M, K, 1), ints(N, K, 2)
    one = torch.ones(M, device="cuda")
    y = skg.linear(x, w, x_scale=one, w_scale=one[:N])
    for rows in (slice(0, 2), slice(M - 2, M)):
        ref = x[rows].double() @ w.double().t().contiguous()
        assert ((y[rows].double() - ref).abs() <= ref.abs() * BF16).all()


@pytest.mark.parametrize("kernel", [(key, i) for key in CHOICES for i in range(len(CHOICES[key]))], ids=str)
def test_kernel(skg, kernel):  # noqa: F811
    (gated, _), i = kernel
    M, N, K = CHOICES[kernel[0]][i]
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("the sizes are for 256 compute units")
    for f32 in (False, True):
        check_linear(skg, M, N, K, gated=bool(gated), act="silu" if gated else "gelu", bias=True, residual=not gated, f32=f32,
                     ld=K + 16, ldy=N + 3, seed=N + i)
    check_linear(skg, M, N, K, gated=bool(gated), seed=K + i)


# ---- as they are used ----------------------------------------------------------

def layer(ops, x, r, p):  # noqa: F811
    """Norm, gated projection, rows to 8 bits, projection back onto the residual stream."""
    q, s, h = ops.add_rms_norm_int8(x, r, p["norm"], 1e-6)
    g = ops.linear_gated_int8(q, s, *p["gate"], *p["up"])
    q, s = ops.quantize_int8(g)
    return ops.linear_int8(q, s, *p["down"], None, h)


def parameters(D, N):
    def weight(n, k, seed):
        w = torch.randn(n, k, generator=gen(seed), device="cuda") / math.sqrt(k)
        s = w.abs().amax(dim=1) / 127
        return torch.round(w / s[:, None]).to(torch.int8), s
    return {"norm": torch.ones(D, dtype=torch.bfloat16, device="cuda"), "gate": weight(N, D, 1), "up": weight(N, D, 2),
            "down": weight(D, N, 3)}


@pytest.mark.parametrize("M", (1, 5, 40))
def test_layer_is_near_the_unquantized_one(ops, M):  # noqa: F811
    """The whole chain against 64 bits on the dequantized weights. Each 8-bit rounding of x is half
    a step of amax / 127; rows of normal values have amax of 3 to 5 times their rms, so each of
    the two quantizations adds an error of about 4 / 127 / sqrt(12) = 0.9% of the norm of a product,
    and the three bfloat16 roundings 0.2% each: 5% is twice their sum on the layer's own part."""
    p = parameters(512, 384)
    x, r = (torch.randn(M, 512, generator=gen(9 + i), device="cuda").to(torch.bfloat16) for i in range(2))
    y = layer(ops, x, r, p).double()
    h, n = norm_ref(x, p["norm"], 1e-6, r)
    wide = {k: p[k][0].double() * p[k][1].double()[:, None] for k in ("gate", "up", "down")}
    g = n @ wide["gate"].t().contiguous()
    own = (torch.sigmoid(g) * g * (n @ wide["up"].t().contiguous())) @ wide["down"].t().contiguous()
    assert torch.linalg.norm(y - h - own) <= 0.05 * torch.linalg.norm(own) + BF16 * torch.linalg.norm(h)


def test_layer_replayed_from_a_graph(ops):  # noqa: F811
    """Captured once, replayed on new inputs with eager calls between the replays."""
    p = parameters(512, 384)
    x, r = (torch.randn(5, 512, generator=gen(i), device="cuda").to(torch.bfloat16) for i in range(2))
    layer(ops, x, r, p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        layer(ops, x, r, p)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        y = layer(ops, x, r, p)
    for i in range(4):
        x.copy_(torch.randn(5, 512, generator=gen(20 + i), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(layer(ops, x, r, p)))


def test_leading_shapes_and_strides(ops):  # noqa: F811
    """x of three dimensions, and rows inside a wider buffer; the Python kernels agree."""
    from bf16_skinny_gemm_amd import torch_op

    x = torch.randn(2, 3, 256, generator=gen(1), device="cuda").to(torch.bfloat16)
    w, ws = parameters(256, 96)["gate"]
    q, s = ops.quantize_int8(x)
    assert q.shape == x.shape and s.shape == (2, 3)
    y = ops.linear_int8(q, s, w, ws)
    assert y.shape == (2, 3, 96)
    flat = ops.linear_int8(q.view(6, 256), s.view(6), w, ws)
    assert torch.equal(bits(y.view(6, 96)), bits(flat))
    wide = torch.randn(6, 512, generator=gen(1), device="cuda").to(torch.bfloat16)
    q1, s1 = ops.quantize_int8(wide[:, 256:])
    q2, s2 = ops.quantize_int8(wide[:, 256:].contiguous())
    assert torch.equal(q1, q2) and torch.equal(s1, s2)
    n = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    for name, args in (("quantize_int8", (x,)), ("rms_norm_int8", (x, n, 1e-6)), ("add_rms_norm_int8", (x, x, n, 1e-6)),
                       ("linear_int8", (q, s, w, ws)), ("linear_gated_int8", (q, s, w, ws, w, ws))):
        got, want = torch_op._PY_KERNELS_MORE[name](*args), getattr(ops, name)(*args)
        for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
            assert a.shape == b.shape and torch.equal(bits(a), bits(b))


def test_empty(ops):  # noqa: F811
    w, ws = parameters(256, 96)["gate"]
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    q, s = ops.quantize_int8(x)
    assert q.shape == (0, 256) and s.shape == (0,) and ops.linear_int8(q, s, w, ws).shape == (0, 96)


def test_refusals(ops):  # noqa: F811
    x = torch.zeros(2, 256, dtype=torch.int8, device="cuda")
    s, w, ws = torch.ones(2, device="cuda"), torch.zeros(8, 256, dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda")
    for args in ((x.float(), s, w, ws), (x, s, w.float(), ws), (x, s[:1], w, ws), (x, s, w, ws[:7]), (x, s, w, ws[:, None]),
                 (x, s.double(), w, ws), (x[:, :128], s, w, ws), (x, s, w.t().contiguous().t(), ws), (x.cpu(), s, w, ws),
                 (x.to(torch.uint8), s, w, ws)):
        with pytest.raises((ValueError, NotImplementedError)):
            ops.linear_int8(*args)
    deep = torch.zeros(1, 131088, dtype=torch.int8, device="cuda")
    with pytest.raises(ValueError):
        ops.linear_int8(deep, s[:1], deep, ws[:1])
    with pytest.raises(ValueError):
        ops.quantize_int8(torch.zeros(2, 0, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        ops.quantize_int8(torch.zeros(2, 8, device="cuda"))

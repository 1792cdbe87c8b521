"""The operators of include/skinny_ops.h against their definitions in 64 bits, on the GPU.

Tolerances are counted from the roundings: the one of the output (half a step: 2^-8 of a
bfloat16 value, 2^-24 of a float32 one, 2^-4 of an e4m3 one or half of its smallest step),
the float32 sums (at most one rounding of the running magnitude per term), and the
activations (a few roundings, carried by a slope of at most 1.13).
"""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = 2.0 ** -8, 2.0 ** -24
TOP, LEAST = 448.0, 2.0 ** -100


@pytest.fixture(scope="module")
def skg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bf16_skinny_gemm_amd

    return bf16_skinny_gemm_amd


@pytest.fixture(scope="module")
def ops(skg):
    from bf16_skinny_gemm_amd import torch_op

    assert torch_op.CPP_OP
    return torch_op


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def walled(M, D, ld=None, dtype=torch.bfloat16, shift=0):
    """An [M, D] view of row stride ld inside a larger buffer whose other elements are NaN."""
    ld = ld or D
    flat = torch.full((M * ld + 64 + shift,), float("nan"), device="cuda").to(dtype)
    return flat, flat[32 + shift:32 + shift + M * ld].view(M, ld)[:, :D]


def filled(values, ld=None, shift=0):
    flat, view = walled(*values.shape, ld, values.dtype, shift)
    view.copy_(values)
    return view


def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32)


def walls_hold(flat, view):
    """Every element of the buffer outside the view still has its first bits."""
    probe = torch.full_like(bits(flat), 0)
    ref = torch.full((1,), float("nan"), device="cuda").to(flat.dtype)
    inside = torch.zeros(flat.shape, dtype=torch.bool, device="cuda")
    inside.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(True)
    probe = torch.where(inside, bits(ref).expand_as(inside), bits(flat))
    return bool((probe == bits(ref)).all())


# ---- norm -------------------------------------------------------------------

def norm_ref(x, w, eps, r):
    h = x.double() + (r.double() if r is not None else 0.0)
    f = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + eps)
    return h, h * w.double() * f


def check_norm(skg, M, D, quant, residual, *, ld=None, shift=0, eps=1e-6, seed=0, x=None, r=None):
    g = gen(seed)
    if x is None:
        x = torch.randn(M, D, generator=g, device="cuda").to(torch.bfloat16)
        r = torch.randn(M, D, generator=g, device="cuda").to(torch.bfloat16)
    r = r if residual else None
    w = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    h, y = norm_ref(x, w, eps, r)
    xv = filled(x, ld, shift)
    rv = filled(r, ld, shift) if residual else None
    wv = filled(w[None], shift=shift)[0]
    odt = torch.bfloat16 if quant is None else torch.float8_e4m3fn
    oflat, ov = walled(M, D, ld, odt, shift)
    hflat, hv = walled(M, D, ld, torch.bfloat16, shift)
    got = skg.rms_norm(xv, wv, eps, residual=rv, quant=quant, out=ov, residual_out=hv if residual else None)
    torch.cuda.synchronize()
    assert walls_hold(oflat, ov) and (not residual or walls_hold(hflat, hv))
    if residual:
        # one float32 addition, then one rounding
        tol = h.abs() * (BF16 + 2 * F32) + 1e-38
        assert ((got[-1].double() - h).abs() <= tol).all()
    rel = (D / 2 + 16) * F32  # half the relative error of the sum, and the factors
    if quant is None:
        y_got = got[0] if residual else got
        assert ((y_got.double() - y).abs() <= y.abs() * (BF16 + rel) + 1e-38).all()
        return
    q, scale = got[0], got[1]
    width = D if quant == "row" else 128
    pad = torch.nn.functional.pad(y, (0, -D % width)).view(M, -1, width)
    s = pad.abs().amax(dim=2).clamp_min(LEAST) / TOP
    assert ((scale.double().view(M, -1) - s).abs() <= s * rel).all()
    s = scale.double().view(M, -1).repeat_interleave(width, dim=1)[:, :D]
    err = (q.double() * s - y).abs()
    assert (err <= y.abs() * (2.0 ** -4 + 2 * rel) + s * (2.0 ** -10 + 2 * rel)).all()
    # the scale is the smallest that holds the row: its largest value is 448 itself
    top = torch.nn.functional.pad(q.double().abs(), (0, -D % width)).view(M, -1, width).amax(dim=2)
    assert ((top == TOP) | (pad.abs().amax(dim=2) < 2 * LEAST)).all()


NORM_D = (1, 7, 8, 64, 120, 127, 128, 512, 520, 1000, 1024, 1537, 2048, 4096, 5000, 8192, 16384, 16392, 32768,
          33000)


@pytest.mark.parametrize("quant", [None, "row", "group"])
@pytest.mark.parametrize("D", NORM_D)
def test_norm_widths(skg, D, quant):
    for M in (1, 3, 17):
        for residual in (False, True):
            check_norm(skg, M, D, quant, residual, seed=D + M)


@pytest.mark.parametrize("quant", [None, "row", "group"])
@pytest.mark.parametrize("M,D,ld,shift", [(5, 512, 1024, 0), (4, 1024, 1032, 0), (3, 1000, 1003, 0), (6, 2048, 2048, 1),
                                          (2, 4096, 4100, 4), (9, 136, 137, 3)])
def test_norm_strides_and_alignment(skg, M, D, ld, shift, quant):
    for residual in (False, True):
        check_norm(skg, M, D, quant, residual, ld=ld, shift=shift, seed=ld)


@pytest.mark.parametrize("D", [96, 4096, 1001])
def test_norm_in_place(skg, D):
    """residual_out over the residual or over x, and y over x."""
    g = gen(D)
    x = torch.randn(6, D, generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn(6, D, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(D, generator=g, device="cuda").to(torch.bfloat16)
    y0, h0 = skg.rms_norm(x, w, residual=r)
    for over in ("residual", "x"):
        xc, rc = x.clone(), r.clone()
        y, h = skg.rms_norm(xc, w, residual=rc, residual_out=rc if over == "residual" else xc)
        assert torch.equal(bits(y), bits(y0)) and torch.equal(bits(h), bits(h0))
        q0, s0, _ = skg.rms_norm(x, w, residual=r, quant="group")
        xc, rc = x.clone(), r.clone()
        q, s, h = skg.rms_norm(xc, w, residual=rc, quant="group", residual_out=rc if over == "residual" else xc)
        assert torch.equal(bits(q), bits(q0)) and torch.equal(s, s0) and torch.equal(bits(h), bits(h0))
    xc = x.clone()
    assert torch.equal(bits(skg.rms_norm(xc, w, out=xc)), bits(skg.rms_norm(x, w)))
    xc, rc = x.clone(), r.clone()
    y, h = skg.rms_norm(xc, w, residual=rc, out=xc, residual_out=rc)
    assert torch.equal(bits(xc), bits(y0)) and torch.equal(bits(rc), bits(h0))


@pytest.mark.parametrize("D", [256, 4096, 999])
@pytest.mark.parametrize("quant", [None, "row", "group"])
def test_norm_special_rows(skg, D, quant):
    """Rows of zeros, tiny, large, infinite and NaN values; each row by itself."""
    x = torch.randn(8, D, generator=gen(3), device="cuda").to(torch.bfloat16)
    x[1] = 0.0
    x[2] *= 2.0 ** -60
    x[3] *= 2.0 ** 50
    x[4, 5] = float("nan")
    x[5, 5] = float("inf")
    x[6] = 0.0
    x[6, D - 1] = -3.0
    w = torch.ones(D, device="cuda", dtype=torch.bfloat16)
    got = skg.rms_norm(x, w, 1e-6, quant=quant)
    y = got if quant is None else got[0]
    fine = [0, 1, 2, 3, 6, 7]
    check_norm(skg, len(fine), D, quant, False, x=x[fine], seed=4)
    yf = y.float()
    assert (yf[1] == 0).all()
    assert yf[4].isnan().all()
    if quant is None:
        assert yf[5, 5].isnan() and (torch.cat([yf[5, :5], yf[5, 6:]]) == 0).all()
    elif quant == "row":
        assert yf[5].isnan().all() and got[1][4:6].isnan().all()
        assert math.isclose(float(got[1][1]) * TOP, LEAST, rel_tol=1e-6)
    else:
        assert yf[5, :128].isnan().all() and got[1][5, 0].isnan()
        assert (yf[5, 128:] == 0).all() and got[1][5, 1:].isfinite().all() and got[1][4].isnan().all()


def test_norm_long(skg):
    """More elements than 31 bits hold: the last rows are right."""
    M, D = 65537 * 4, 8192
    x = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
    x.random_(-8, 9, generator=gen(1))
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    y = skg.rms_norm(x, w, out=x.clone())
    for rows in (slice(0, 3), slice(M - 3, M)):
        _, ref = norm_ref(x[rows], w, 1e-6, None)
        assert ((y[rows].double() - ref).abs() <= ref.abs() * (BF16 + (D / 2 + 16) * F32)).all()


@pytest.mark.parametrize("quant", [None, "row", "group"])
def test_norm_beyond_the_cache(skg, quant):
    """More bytes than the last cache holds, where the kernels use the non-temporal hint."""
    for D in (4096, 4091):
        check_norm(skg, 7001, D, quant, True, seed=D)


# ---- projections ------------------------------------------------------------

def act_ref(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def blocks_of(scale, rows, N, K):
    full = scale.double().repeat_interleave(128, dim=1)[:, :K]
    return full.repeat_interleave(rows, dim=0)[:N]


def make_linear(M, N, K, mode, mats, seed, ld=None, shift=0):
    """x and weights (wide double copies and the stored ones) with their scales."""
    g = gen(seed)
    x = torch.randn(M, K, generator=g, device="cuda")
    w = [torch.randn(N, K, generator=g, device="cuda") / math.sqrt(max(K, 1)) for _ in range(mats)]
    if mode == "bf16":
        xq, wq = x.to(torch.bfloat16), [v.to(torch.bfloat16) for v in w]
        xs = ws = None
        xd, wd = xq.double(), [v.double() for v in wq]
    else:
        # stored values over the whole e4m3 range, and scales apart from them
        xq = (x * 60).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
        wq = [(v * math.sqrt(max(K, 1)) * 60).clamp(-TOP, TOP).to(torch.float8_e4m3fn) for v in w]
        kb, nb = -(-K // 128), -(-N // 128)
        sh = ((M,), (N,)) if mode == "row" else ((M, kb), (nb, kb))
        xs = (torch.rand(sh[0], generator=g, device="cuda") + 0.5) / 60
        ws = [(torch.rand(sh[1], generator=g, device="cuda") + 0.5) / 60 / math.sqrt(max(K, 1)) for _ in range(mats)]
        if mode == "row":
            xd, wd = xq.double() * xs.double()[:, None], [q.double() * s.double()[:, None] for q, s in zip(wq, ws)]
        else:
            xd = xq.double() * blocks_of(xs, 1, M, K)
            wd = [q.double() * blocks_of(s, 128, N, K) for q, s in zip(wq, ws)]
    xv = filled(xq, ld, shift)
    wv = [filled(q, shift=shift) for q in wq]
    return xv, wv, xs, ws, xd, wd


def check_linear(skg, M, N, K, mode, *, gated=False, act="none", bias=False, residual=False, f32=False, ld=None,
                 ldy=None, shift=0, seed=0, in_place=False):
    mats = 2 if gated else 1
    xv, wv, xs, ws, xd, wd = make_linear(M, N, K, mode, mats, seed, ld, shift)
    g = gen(seed + 1)
    b = [torch.randn(N, generator=g, device="cuda").to(torch.bfloat16) if bias else None for _ in range(mats)]
    r = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16) if residual else None
    odt = torch.float32 if f32 else torch.bfloat16
    if in_place:
        oflat, ov = walled(M, N, ldy, odt)
        ov.copy_(r)
        rv = ov
    else:
        oflat, ov = walled(M, N, ldy, odt, 0 if f32 else shift)
        rv = None if r is None else filled(r, ldy, shift)
    y = skg.linear(xv, wv[0], bias=b[0], residual=rv, act=act, W_up=wv[1] if gated else None,
                   bias_up=b[1] if gated else None, x_scale=xs, w_scale=ws[0] if ws else None,
                   w_up_scale=ws[1] if ws and gated else None, out=ov, out_dtype=odt)
    torch.cuda.synchronize()
    assert walls_hold(oflat, ov)
    z, e = [], []
    for i in range(mats):
        v = xd @ wd[i].t().contiguous()
        mag = xd.abs() @ wd[i].abs().t().contiguous()
        if bias:
            v, mag = v + b[i].double(), mag + b[i].double().abs()
        z.append(v)
        per_mag = (2 * K + 64) * F32  # a product and an addition per term
        if mode != "bf16" and M > 16 and not f32:
            # the 8-bit matrix instruction cuts the products of each group of eight off at
            # 2^-13 of the largest, which the group's magnitude is at least: 7 * 2^-13 of it
            per_mag += 7 * 2.0 ** -13
        e.append(per_mag * mag + 1e-30)
    ref, err = act_ref(z[0], act), 1.13 * e[0]
    err = err + 32 * F32 * (ref.abs() + z[0].abs() * (0 if act in ("none", "relu") else 1))
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


MODES = ("bf16", "row", "block")


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 9, 16, 17, 32, 33, 48, 64, 65, 100, 128, 129, 200, 300])
def test_linear_rows(skg, M, mode):
    check_linear(skg, M, 333, 1040, mode, seed=M, f32=True)
    check_linear(skg, M, 256, 4096, mode, act="silu", bias=True, residual=True, seed=M + 1)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("N", [1, 3, 15, 16, 17, 63, 64, 65, 127, 129, 255, 500, 1025])
def test_linear_widths(skg, N, mode):
    for M in (1, 6, 12, 40, 150, 600):
        check_linear(skg, M, N, 528, mode, seed=N + M, bias=True)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("K", [1, 5, 8, 16, 24, 112, 120, 128, 136, 144, 256, 1000, 1536, 2064, 8192])
def test_linear_depths(skg, K, mode):
    for M in (1, 5, 13, 30, 70, 260):
        check_linear(skg, M, 144, K, mode, seed=K + M, f32=M % 2 == 1, residual=True)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M", [1, 4, 7, 16, 20, 32, 33, 64, 65, 128, 257, 700])
def test_linear_gated(skg, M, mode):
    check_linear(skg, M, 320, 1024, mode, gated=True, act="silu", seed=M)
    check_linear(skg, M, 131, 272, mode, gated=True, act="gelu", bias=True, f32=True, seed=M + 1)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("mode", MODES)
def test_linear_activations(skg, act, mode):
    for M in (3, 130):
        check_linear(skg, M, 200, 384, mode, act=act, bias=True, residual=True, f32=True, seed=5)
        check_linear(skg, M, 200, 384, mode, act=act, gated=True, bias=True, seed=6)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M,N,K,ld,ldy,shift", [(3, 70, 256, 512, 96, 0), (40, 65, 256, 272, 66, 0), (7, 33, 250, 251, 40, 0),
                                               (150, 130, 384, 400, 131, 0), (5, 40, 128, 128, 40, 1), (90, 50, 77, 80, 50, 3)])
def test_linear_strides_and_alignment(skg, M, N, K, ld, ldy, shift, mode):
    check_linear(skg, M, N, K, mode, bias=True, residual=True, ld=ld, ldy=ldy, shift=shift, seed=K)
    check_linear(skg, M, N, K, mode, gated=True, act="silu", f32=True, ld=ld, ldy=ldy, shift=shift, seed=K)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M", [1, 20, 100, 512])
def test_linear_residual_in_place(skg, M, mode):
    check_linear(skg, M, 264, 512, mode, act="gelu_tanh", residual=True, in_place=True, ldy=270, seed=M)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M,N,K", [(1024, 1024, 512), (2048, 1100, 640), (4100, 2048, 256)])
def test_linear_large(skg, M, N, K, mode):
    check_linear(skg, M, N, K, mode, bias=True, residual=True, seed=M)
    check_linear(skg, M, N // 2, K, mode, gated=True, act="silu", seed=M)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M,N,ldy", [(1500, 1031, 1031), (2100, 516, 523), (700, 2047, 2048), (1025, 769, 771)])
def test_linear_rows_that_end_inside_a_store(skg, M, N, ldy, mode):
    check_linear(skg, M, N, 384, mode, act="gelu", bias=True, residual=True, ldy=ldy, seed=N)
    check_linear(skg, M, N, 256, mode, residual=True, in_place=True, ldy=ldy, seed=N + 1)
    check_linear(skg, M, N, 256, mode, bias=True, residual=True, f32=True, ldy=ldy, seed=N + 2)
    check_linear(skg, M, N, 384, mode, gated=True, act="silu", bias=True, ldy=ldy, seed=N + 3)


def test_linear_long_outputs(skg):
    """More outputs than 31 bits hold: rows at both ends."""
    M, N, K = 70001, 32768, 64
    x = torch.randn(M, K, generator=gen(1), device="cuda").to(torch.bfloat16)
    w = torch.randn(N, K, generator=gen(2), device="cuda").to(torch.bfloat16)
    y = skg.linear(x, w)
    for rows in (slice(0, 2), slice(M - 2, M)):
        ref = x[rows].double() @ w.double().t().contiguous()
        mag = x[rows].double().abs() @ w.double().abs().t().contiguous()
        assert ((y[rows].double() - ref).abs() <= ref.abs() * BF16 + 2 * (2 * K + 64) * F32 * mag).all()


@pytest.mark.parametrize("M", [2, 40])
def test_linear_long_weight(skg, M):
    """A weight of more than 2^31 elements: its first and last features."""
    N, K = 530000, 4096
    w = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    w.random_(-4, 5, generator=gen(3))
    x = torch.randn(M, K, generator=gen(4), device="cuda").to(torch.bfloat16)
    y = skg.linear(x, w, out_dtype=torch.float32)
    for part in (slice(0, 70), slice(N - 70, N)):
        ref = x.double() @ w[part].double().t().contiguous()
        mag = x.double().abs() @ w[part].double().abs().t().contiguous()
        assert ((y[:, part].double() - ref).abs() <= (2 * K + 64) * F32 * mag).all()


@pytest.mark.parametrize("mode", MODES)
def test_linear_empty_depth(skg, mode):
    """K = 0: the empty sum, so act(bias) + residual."""
    check_linear(skg, 5, 40, 0, mode, bias=True, residual=True, act="silu", seed=1)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M", [2, 60, 300])
def test_linear_nan_stays_in_its_row(skg, M, mode):
    """A NaN in one row of x reaches that row of y alone, one in a row of W that column."""
    xv, wv, xs, ws, _, _ = make_linear(M, 100, 256, mode, 1, 9)
    kw = dict(x_scale=xs, w_scale=ws[0] if ws else None)
    clean = skg.linear(xv, wv[0], **kw)
    xn, wn = xv.clone(), wv[0].clone()
    nan = torch.full((1,), float("nan"), device="cuda").to(xv.dtype)
    bits(xn)[M - 1, 130] = bits(nan)[0]
    y = skg.linear(xn, wv[0], **kw)
    assert y[M - 1].isnan().all() and torch.equal(bits(y[:M - 1]), bits(clean[:M - 1]))
    bits(wn)[37, 3] = bits(nan)[0]
    y = skg.linear(xv, wn, **kw)
    assert y[:, 37].isnan().all()
    keep = [i for i in range(100) if i != 37]
    assert torch.equal(bits(y[:, keep].contiguous()), bits(clean[:, keep].contiguous()))


def test_empty_calls(ops, skg):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.randn(32, 64, device="cuda").to(torch.bfloat16)
    assert skg.linear(x, w).shape == (0, 32)
    assert ops.linear_act(x, w).shape == (0, 32)
    assert ops.linear_act(x.view(0, 3, 64), w).shape == (0, 3, 32)
    assert skg.rms_norm(x, w[0].contiguous()).shape == (0, 64)
    q, s = ops.rms_norm_fp8(x, w[0].contiguous(), 1e-6, 128)
    assert q.shape == (0, 64) and s.shape == (0, 1)


# ---- as they are used -------------------------------------------------------

def mlp_ref(x, r, nw, wg, wu, wd, group):
    """A layer's MLP in 64 bits from the stored values."""
    h = x.double() + r.double()
    y = h * nw.double() / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)
    z = act_ref(y @ wg.t(), "silu") * (y @ wu.t())
    return h, z @ wd.t() + h


@pytest.mark.parametrize("M", [1, 7, 40, 257])
@pytest.mark.parametrize("fp8", [False, True])
def test_mlp_run(ops, M, fp8):
    """norm with residual -> gated projection -> down projection added to the new residual,
    as one layer's MLP runs them; eagerly and as a replayed graph, on a side stream."""
    D, F = 1024, 640
    g = gen(M)
    x, r = (torch.randn(M, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    nw = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    wg, wu = (torch.randn(F, D, generator=g, device="cuda") / 32 for _ in range(2))
    wd = (torch.randn(D, F, generator=g, device="cuda") / math.sqrt(F)).to(torch.bfloat16)
    if fp8:
        def quantised(w):
            b = w.view(F // 128, 128, D // 128, 128)
            s = b.abs().amax(dim=(1, 3)) / TOP
            q = (b / s[:, None, :, None]).view(F, D).to(torch.float8_e4m3fn)
            return q, s, q.double() * blocks_of(s, 128, F, D)
        (qg, sg, dg), (qu, su, du) = quantised(wg), quantised(wu)
    else:
        wg, wu = wg.to(torch.bfloat16), wu.to(torch.bfloat16)
        dg, du = wg.double(), wu.double()

    def step(xi, ri):
        if fp8:
            q, s, h = ops.add_rms_norm_fp8(xi, ri, nw, 1e-6, 128)
            z = ops.linear_gated_fp8(q, s, qg, sg, qu, su)
        else:
            y, h = ops.add_rms_norm(xi, ri, nw, 1e-6)
            z = ops.linear_gated(y, wg, wu)
        return h, ops.linear_act(z, wd, None, h)

    h, y = step(x, r)
    hr, yr = mlp_ref(x, r, nw, dg, du, wd.double(), 128)
    # three roundings of the hidden values (2^-4 each element in 8 bits, averaged over the sum)
    assert torch.linalg.norm(y.double() - yr) <= (0.04 if fp8 else 0.01) * torch.linalg.norm(yr)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    xs, rs = x.clone(), r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        step(xs, rs)
        with torch.cuda.graph(graph, stream=stream):
            hg, yg = step(xs, rs)
    torch.cuda.current_stream().wait_stream(stream)
    for i in range(4):
        xi = torch.randn(M, D, generator=g, device="cuda").to(torch.bfloat16)
        he, ye = step(xi, r)
        xs.copy_(xi)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(hg), bits(he)) and torch.equal(bits(yg), bits(ye)), i


def test_streams_overlap(ops):
    """Calls on two streams at once, with nothing shared: the same bits as one after another."""
    g = gen(0)
    cases = []
    for M, N, K in ((4, 2048, 4096), (300, 1024, 1024), (40, 999, 1536)):
        x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
        w = torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16)
        cases.append((x, w, ops.linear_act(x, w)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(12):
        x, w, _ = cases[i % 3]
        with torch.cuda.stream(streams[i % 2 if i % 3 else 2]):
            got.append(ops.linear_act(x, w))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(bits(y), bits(cases[i % 3][2])), i


def test_op_shapes_and_layouts(ops, skg):
    """Leading dimensions, non-contiguous inputs and scales from the norm."""
    g = gen(2)
    x = torch.randn(2, 3, 256, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(96, 256, generator=g, device="cuda").to(torch.bfloat16)
    nw = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    flat = x.reshape(6, 256)
    assert torch.equal(ops.linear_act(x, w), skg.linear(flat, w).view(2, 3, 96))
    assert torch.equal(ops.rms_norm(x, nw, 1e-6), skg.rms_norm(flat, nw).view(2, 3, 256))
    assert torch.equal(ops.rms_norm(x[0, 0], nw, 1e-6), skg.rms_norm(flat[:1], nw)[0])
    t = x.transpose(0, 1)
    assert torch.equal(ops.linear_act(t, w), skg.linear(t.reshape(6, 256), w).view(3, 2, 96))
    wide = torch.randn(6, 512, generator=g, device="cuda").to(torch.bfloat16)
    assert torch.equal(ops.linear_act(wide[:, 256:], w), skg.linear(wide[:, 256:].contiguous(), w))
    e = flat[:1].expand(6, 256)
    assert torch.equal(ops.linear_act(e, w), skg.linear(e.contiguous(), w))
    for group in (0, 128):
        q, s = ops.rms_norm_fp8(x, nw, 1e-6, group)
        assert s.shape == ((2, 3, 2) if group else (2, 3))
        wq = w.clamp(-4, 4).to(torch.float8_e4m3fn)
        ws = torch.ones((1, 2) if group else (96,), device="cuda")
        y = ops.linear_fp8(q, s, wq, ws, None, None, "relu", True)
        ref = skg.linear(q.view(6, 256), wq, act="relu", x_scale=s.view(6, 2) if group else s.view(6), w_scale=ws,
                         out_dtype=torch.float32)
        assert torch.equal(y.view(6, 96), ref)


def test_ops_compile(ops):
    def f(x, r, nw, w, u):
        q, s, h = torch.ops.skinny.add_rms_norm_fp8(x, r, nw, 1e-6, 0)
        y, _ = torch.ops.skinny.add_rms_norm(x, r, nw, 1e-6)
        z = torch.ops.skinny.linear_gated(y, w, u)
        return q, s, h, torch.ops.skinny.linear_act(z, w[:, :64].t().contiguous(), None, None, "gelu", True)

    g = gen(8)
    x, r = (torch.randn(3, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    nw = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    w, u = (torch.randn(64, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    for a, b in zip(torch.compile(f, backend="aot_eager", fullgraph=True)(x, r, nw, w, u), f(x, r, nw, w, u)):
        assert torch.equal(bits(a), bits(b))


def test_install_fused(ops):
    """Biased layers and norms of a model run on the operators, and on the standard path
    where a gradient is asked for or a call does not qualify."""
    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.RMSNorm(256), torch.nn.Linear(256, 128, bias=True),
                                torch.nn.Linear(128, 64, bias=False), torch.nn.RMSNorm(64, eps=1e-5))
    model = model.cuda().to(torch.bfloat16)
    x = torch.randn(3, 5, 256, device="cuda").to(torch.bfloat16)
    plain = model(x)
    assert ops.install(model, fused=True) == 4 and ops.install(model, fused=True) == 0
    norm0, lin0, lin1, norm1 = model
    with torch.no_grad():
        a = ops.rms_norm(x, norm0.weight, torch.finfo(torch.float32).eps)
        b = ops.linear_act(a, lin0.weight, lin0.bias)
        c = torch.nn.functional.linear(b, lin1.weight)  # 15 rows: not the skinny product's
        assert torch.equal(model(x), ops.rms_norm(c, norm1.weight, 1e-5))
        # three roundings of values of size one, the last through a norm
        assert (model(x).float() - plain.float()).abs().max() <= 0.1
        many = torch.randn(65, 256, device="cuda").to(torch.bfloat16)
        assert torch.equal(lin0(many), torch.nn.functional.linear(many, lin0.weight, lin0.bias))
        f = norm0.float()
        xf = x.float()
        assert torch.equal(f(xf), torch.nn.functional.rms_norm(xf, (256,), f.weight, None))
        norm0.to(torch.bfloat16)
    y = model(x)
    y.float().sum().backward()
    assert lin0.weight.grad is not None and norm0.weight.grad is not None and lin0.bias.grad is not None


def test_install_fused_default_eps(ops):
    """A module without an eps, on rows small enough for it to count: both paths agree."""
    norm = torch.nn.RMSNorm(256).cuda().to(torch.bfloat16)
    x = torch.cat([torch.randn(4, 256, generator=gen(1), device="cuda") * s for s in (1.0, 0.05, 1e-3, 1e-4)])
    x = x.to(torch.bfloat16)
    with torch.no_grad():
        plain = norm(x).double()
        assert ops.install(norm, fused=True) == 1
        got = norm(x).double()
    # one rounding to bfloat16 each of values that float32 holds to (D / 2 + 16) of its steps
    assert ((got - plain).abs() <= plain.abs() * (2 * BF16 + 2 * (128 + 16) * F32)).all()


def test_install_fused_twice_and_own_forward(ops):
    class OnePlus(torch.nn.RMSNorm):
        def forward(self, x):
            return torch.nn.functional.rms_norm(x, (64,), 1 + self.weight, 1e-6)

    class Doubled(torch.nn.Linear):
        def forward(self, x):
            return 2 * super().forward(x)

    model = torch.nn.Sequential(torch.nn.Linear(128, 64), OnePlus(64), Doubled(64, 64)).cuda().to(torch.bfloat16)
    assert ops.install(model) == 2 and ops.install(model, fused=True) == 0
    x = torch.randn(20, 128, generator=gen(2), device="cuda").to(torch.bfloat16)
    with torch.no_grad():
        y = model[0](x)
        assert torch.equal(y, ops.linear_act(x, model[0].weight, model[0].bias, None, "none", False))
        assert torch.equal(model[1](y), torch.nn.functional.rms_norm(y, (64,), 1 + model[1].weight, 1e-6))


@pytest.mark.parametrize("quant", [None, "row", "group"])
def test_norm_in_place_beyond_the_registers(skg, quant):
    D = 33000
    x = torch.randn(3, D, generator=gen(5), device="cuda").to(torch.bfloat16)
    r = torch.randn(3, D, generator=gen(6), device="cuda").to(torch.bfloat16)
    w = torch.randn(D, generator=gen(7), device="cuda").to(torch.bfloat16)
    want = skg.rms_norm(x, w, residual=r, quant=quant)
    for over in ("residual", "x"):
        xc, rc = x.clone(), r.clone()
        got = skg.rms_norm(xc, w, residual=rc, quant=quant, residual_out=rc if over == "residual" else xc)
        assert all(torch.equal(bits(a) if a.dtype != torch.float32 else a, bits(b) if b.dtype != torch.float32 else b)
                   for a, b in zip(got, want))


@pytest.mark.parametrize("lead", [(5,), (2, 3)])
def test_python_kernels_agree(ops, lead):
    """The Python kernels of the operators, registered where the C++ ones are not built."""
    g, K, N = gen(11), 256, 130
    bf = torch.bfloat16
    x, r = (torch.randn(*lead, K, generator=g, device="cuda").to(bf) for _ in range(2))
    w, b, u = (torch.randn(*s, generator=g, device="cuda").to(bf) for s in ((K,), (N,), (N,)))
    wg, wu = (torch.randn(N, K, generator=g, device="cuda").to(bf) for _ in range(2))
    res = torch.randn(*lead, N, generator=g, device="cuda").to(bf)
    qg, qu = (t.float().to(torch.float8_e4m3fn) for t in (wg, wu))
    rows, blocks = torch.rand(N, generator=g, device="cuda"), torch.rand(2, 2, generator=g, device="cuda")
    q0, s0 = ops.rms_norm_fp8(x, w, 1e-6, 0)
    q1, s1 = ops.rms_norm_fp8(x, w, 1e-6, 128)
    calls = {
        "rms_norm": [(x, w, 1e-6)],
        "add_rms_norm": [(x, r, w, 1e-6)],
        "rms_norm_fp8": [(x, w, 1e-6, 0), (x, w, 1e-6, 128)],
        "add_rms_norm_fp8": [(x, r, w, 1e-6, 0), (x, r, w, 1e-6, 128)],
        "linear_act": [(x, wg), (x, wg, b, res, "gelu", True)],
        "linear_gated": [(x, wg, wu), (x, wg, wu, b, u, "relu", True)],
        "linear_fp8": [(q0, s0, qg, rows, b, res, "silu", False), (q1, s1, qg, blocks)],
        "linear_gated_fp8": [(q0, s0, qg, rows, qu, rows, b, u), (q1, s1, qg, blocks, qu, blocks)],
    }
    assert set(calls) == set(ops._PY_KERNELS)
    for name, several in calls.items():
        for args in several:
            want, got = getattr(ops, name)(*args), ops._PY_KERNELS[name](*args)
            want, got = (want, got) if isinstance(want, (tuple, list)) else ((want,), (got,))
            assert len(want) == len(got)
            for a, c in zip(want, got):
                assert a.dtype == c.dtype and a.shape == c.shape and torch.equal(bits(a), bits(c)), name


@pytest.mark.parametrize("eps", [1e-6, 1e-12, 1e-20, 1e-30])
@pytest.mark.parametrize("quant", ["row", "group"])
@pytest.mark.parametrize("D", [256, 999, 4096, 20000, 33000])
def test_norm_fp8_zeros_and_small_rows_at_any_eps(skg, D, quant, eps):
    """Rows and groups of zeros stay zeros beside values of any size, at every eps above 0."""
    x = torch.randn(9, D, generator=gen(D), device="cuda")
    x[0] = 0.0
    x[1] *= 1e-3
    x[2:5] *= 1e-7
    x[3, :128] = 0.0          # a group of zeros in a small row
    x[4, 5:] = 0.0
    x[5] *= 2.0 ** -60
    x[6] *= 2.0 ** -115       # y below the least scale's at the larger eps
    x[7, 128:] = 0.0
    x = x.to(torch.bfloat16)
    check_norm(skg, 9, D, quant, False, x=x, eps=eps, seed=D)
    check_norm(skg, 9, D, quant, True, x=x, r=torch.zeros_like(x), eps=eps, seed=D)


# rows, inputs and element types that take the streaming, the tiled and the element-wise kernel
EPILOGUE_PATHS = [(3, 64, "bf16"), (5, 128, "row"), (40, 128, "block"), (600, 128, "bf16"), (600, 128, "row"),
                  (600, 128, "block"), (3, 0, "bf16"), (6, 63, "row")]


def act_of_values(skg, values, act, M, K, mode, f32):
    """act of given bfloat16 values (the bias) through a product of zeros, [M, len(values)]."""
    N = values.numel()
    xv, wv, xs, ws, _, _ = make_linear(M, N, K, mode, 1, 1)
    y = skg.linear(torch.zeros_like(xv.contiguous()), wv[0], bias=values, act=act, x_scale=xs,
                   w_scale=ws[0] if ws else None, out_dtype=torch.float32 if f32 else torch.bfloat16)
    assert torch.equal(bits(y), bits(y[:1].expand(M, N).contiguous()))
    return y[0].double()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,K,mode", EPILOGUE_PATHS)
def test_activations_of_infinite_large_and_nan_values(skg, M, K, mode, act):
    inf = float("inf")
    v = torch.tensor([inf, 3e38, 1e30, 1e10, 300.0, 0.0, -300.0, -1e10, -1e30, -3e38, float("nan"), -inf, 1.0],
                     device="cuda").to(torch.bfloat16)
    for f32 in (False, True):
        y = act_of_values(skg, v, act, M, K, mode, f32)
        assert torch.equal(y[:6], v[:6].double())  # act(z) = z to the last bit for large z
        assert y[10].isnan()
        if act == "none":
            assert torch.equal(y[6:10], v[6:10].double()) and y[11] == -inf
        else:
            assert (y[6:10] == 0).all()
            # -inf times the 0 that it is weighted with, but relu's selects
            assert y[11] == 0 if act == "relu" else y[11].isnan()
        assert abs(y[12] - act_ref(torch.ones((), dtype=torch.float64), act)) <= BF16


@pytest.mark.parametrize("M,K,mode", EPILOGUE_PATHS)
def test_gelu_is_right_relative_to_its_value(skg, M, K, mode):
    """Far into the negative tail, too. Roundings counted for Phi: 2.2 * 2^-24 of the fit; 16 of
    the polynomial and its argument; z^2 / 2 in the exponent with 6 * 2^-24 of its own size (x,
    its square, the constants), which the exponential turns into as much of the value; 8 of the
    exponential and the products."""
    v = torch.linspace(-12, 12, 505, device="cuda").to(torch.bfloat16)
    z = v.double()
    ref = 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5))  # ndtr is 0 below -8.3
    rel = (32 + 3 * z * z) * F32
    for f32 in (False, True):
        y = act_of_values(skg, v, "gelu", M, K, mode, f32)
        assert ((y - ref).abs() <= ref.abs() * (rel + (F32 if f32 else BF16 * (1 + rel)))).all()


@pytest.mark.parametrize("shape,N", [((2, 3, 0), 40), ((5, 0), 40), ((0, 3, 64), 40), ((4, 64), 0), ((0, 0), 40)])
def test_python_kernels_agree_on_empty_sizes(ops, shape, N):
    g, bf, K = gen(12), torch.bfloat16, shape[-1]
    x = torch.randn(*shape, generator=g, device="cuda").to(bf)
    w, b = torch.randn(N, K, generator=g, device="cuda").to(bf), torch.randn(N, generator=g, device="cuda").to(bf)
    r = torch.randn(*shape[:-1], N, generator=g, device="cuda").to(bf)
    e4 = torch.float8_e4m3fn
    kb, nb = -(-K // 128), -(-N // 128)
    rows = (torch.ones(shape[:-1], device="cuda"), torch.ones(N, device="cuda"))
    blocks = (torch.ones(*shape[:-1], kb, device="cuda"), torch.ones(nb, kb, device="cuda"))
    calls = [("linear_act", (x, w, b, r, "silu", True))]
    calls += [("linear_fp8", (x.to(e4), xs, w.to(e4), ws, b, r, "silu", True)) for xs, ws in (rows, blocks)]
    for name, args in calls:
        want, got = getattr(ops, name)(*args), ops._PY_KERNELS[name](*args)
        assert want.shape == got.shape == (*shape[:-1], N) and torch.equal(bits(want), bits(got))
        if K == 0:
            ref = act_ref(b.double(), "silu") + r.double()
            assert ((want.double() - ref).abs() <= 32 * F32 * (ref.abs() + b.double().abs())).all()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M,N,K", [(700, 1031, 8208), (2100, 1100, 4112), (260, 8200, 5136)])
def test_linear_deep_tiles(skg, M, N, K, mode):
    """Many stages of the tiled kernels; the block scales of neighbouring stages differ."""
    check_linear(skg, M, N, K, mode, bias=True, residual=True, seed=K)
    check_linear(skg, M, N // 2, K, mode, gated=True, act="silu", seed=K)
    x, w, xs, ws, _, _ = make_linear(M, N, K, mode, 1, K + 1)
    kw = dict(x_scale=xs, w_scale=ws[0] if ws else None)
    first = skg.linear(x, w[0], **kw)
    for _ in range(5):
        assert torch.equal(bits(skg.linear(x, w[0], **kw)), bits(first))

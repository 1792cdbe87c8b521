"""Argument checks of the 8-bit integer operators, with no kernel run: validation comes before
any device work, so fake (never dereferenced) pointers serve."""
from __future__ import annotations

import ctypes

import pytest
import torch

from .int8_choices import CHOICES
from .test_ops_abi import BAD, OK, R, RO, S, UNSUPPORTED, W, X, Y, needs_no_gpu, skg  # noqa: F401


def norm(skg, plain=False, **kw):  # noqa: F811
    M, D = kw.get("M", 4), kw.get("D", 256)
    a = dict(x=X, y=Y, scale=S, ldx=D, ldy=D, M=M, D=D, group=0, eps=0.0)
    if not plain:
        a.update(weight=W)
    a.update(kw)
    if a.pop("res", False):
        a = {**dict(residual=R, residual_out=RO, ldr=D, ldro=D), **a}
    fn = skg.lib().skinny_quantize_int8 if plain else skg.lib().skinny_rms_norm_int8
    return fn(skg.NormArgs(**a), None)


def linear(skg, fn="skinny_linear_int8", **kw):  # noqa: F811
    M, N, K = kw.get("M", 4), kw.get("N", 64), kw.get("K", 256)
    a = dict(x=X, W0=W, y=Y, ldx=K, ldy=N, M=M, N=N, K=K, act=0, out_f32=0, scales=1, x_scale=S, w0_scale=S + 0x100000)
    a.update(kw)
    return getattr(skg.lib(), fn)(skg.LinearArgs(**a), None)


@needs_no_gpu
def test_accepted_arguments_reach_the_device_check(skg):  # noqa: F811
    """Without a GPU an accepted call ends at the device check, a refused one before it."""
    for kw in ({}, dict(res=True), dict(res=True, residual_out=R), dict(res=True, residual_out=X), dict(x=X + 2), dict(ldy=300)):
        assert norm(skg, **kw) == UNSUPPORTED
    for kw in ({}, dict(ldx=300, ldy=300), dict(x=X + 2, y=Y + 1), dict(M=1, ldx=256)):
        assert norm(skg, True, **kw) == UNSUPPORTED
    for kw in ({}, dict(bias0=R, residual=RO, ldr=64), dict(residual=Y, ldr=64), dict(K=131071, ldx=131071),
               dict(W1=R, bias1=RO, w1_scale=S + 0x200000), dict(ldx=300, ldy=70, out_f32=1),
               dict(K=0, ldx=0, x=None, W0=None, x_scale=None, w0_scale=None)):
        assert linear(skg, **kw) == UNSUPPORTED, kw


def test_empty_calls_are_noops(skg):  # noqa: F811
    assert norm(skg, M=0, x=None, y=None) == norm(skg, D=0) == norm(skg, True, M=0, x=None) == norm(skg, True, D=0) == OK
    assert linear(skg, M=0, x=None, y=None) == linear(skg, N=0) == OK


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(D=-1), dict(x=None), dict(y=None), dict(scale=None), dict(scale=S + 2), dict(group=128), dict(group=1),
    dict(ldx=255), dict(ldy=255), dict(x=X + 1), dict(y=X), dict(y=X + 8), dict(scale=Y), dict(scale=X), dict(scale=Y + 1020),
    dict(ldx=1 << 50), dict(M=1 << 30, ldx=1 << 35), dict(eps=-1.0), dict(eps=float("nan"))])
def test_norm_refusals(skg, kw):  # noqa: F811
    assert norm(skg, **kw) == norm(skg, True, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(weight=None), dict(weight=W + 1), dict(residual=R), dict(res=True, scale=RO),
                                dict(res=True, residual_out=Y), dict(y=W)])
def test_norm_refusals_of_its_own(skg, kw):  # noqa: F811
    assert norm(skg, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(weight=W), dict(eps=1e-6), dict(res=True), dict(residual=R), dict(residual_out=RO)])
def test_quantize_takes_no_norm(skg, kw):  # noqa: F811
    assert norm(skg, True, **kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(x=None), dict(W0=None), dict(y=None), dict(act=-1), dict(act=5),
    dict(out_f32=2), dict(ldx=255), dict(ldy=63), dict(residual=R, ldr=63), dict(bias0=R + 1), dict(y=Y + 1), dict(bias1=R),
    dict(out_f32=1, y=Y + 2), dict(y=X), dict(y=W), dict(residual=Y + 2, ldr=64), dict(residual=Y, ldr=64, out_f32=1),
    dict(scales=0), dict(scales=2), dict(scales=3), dict(x_scale=None), dict(w0_scale=None), dict(x_scale=S + 2),
    dict(y=S), dict(w0_scale=Y + 256), dict(W1=R), dict(W1=R, w1_scale=S, residual=RO, ldr=64), dict(K=131072, ldx=131072)])
def test_linear_refusals(skg, kw):  # noqa: F811
    assert linear(skg, **kw) == BAD


def test_null_arguments(skg):  # noqa: F811
    L = skg.lib()
    for fn in (L.skinny_rms_norm_int8, L.skinny_quantize_int8, L.skinny_linear_int8):
        assert fn(None, None) == BAD
    p = skg.LinearPlan()
    assert L.skinny_linear_int8_default_plan(None, 256, ctypes.byref(p)) == BAD


def test_other_entry_points_take_no_int8(skg):  # noqa: F811
    """The scales value of another entry point is refused there, not read as this type."""
    assert linear(skg, "skinny_linear_fp8", scales=3) == linear(skg, "skinny_linear_bf16") == BAD


def test_plan(skg):  # noqa: F811
    def plan(**kw):
        a = dict(x=X, W0=W, y=Y, ldx=4096, ldy=4096, M=4, N=4096, K=4096, scales=1, x_scale=S, w0_scale=S + 0x100000)
        return skg.skinny_linear_int8_default_plan(skg.LinearArgs(**{**a, **kw}))
    assert plan().kind == plan(out_f32=1).kind == skg.SKINNY_LINEAR_STREAM
    big = dict(M=4096, x_scale=1 << 40)  # apart from the other operands
    assert plan(**big, y=1 << 41).kind == skg.SKINNY_LINEAR_TILE
    assert plan(ldx=4097).kind == plan(K=4095).kind == plan(x=X + 8).kind == skg.SKINNY_LINEAR_ELEMENTS
    for kw in (dict(M=0), dict(N=0), dict(scales=2), dict(K=131072, ldx=131072)):
        with pytest.raises(skg.SkinnyError):
            plan(**kw)


@pytest.mark.parametrize("key", CHOICES)
def test_every_offered_kernel_is_chosen_at_some_size(skg, key):  # noqa: F811
    gated, rows = key
    def plan(M, N, K, f32):
        return skg.skinny_linear_int8_default_plan(skg.LinearArgs(
            x=1 << 40, W0=1 << 41, W1=1 << 42 if gated else None, y=1 << 43, x_scale=1 << 44, w0_scale=1 << 45,
            w1_scale=1 << 46 if gated else None, ldx=K, ldy=N, M=M, N=N, K=K, scales=1, out_f32=f32))
    plans = [plan(M, N, K, 0) for M, N, K in CHOICES[key]]
    assert [p.index for p in plans] == list(range(plans[0].count))
    for p, (M, N, K) in zip(plans, CHOICES[key]):
        assert (M <= 8, M <= 16) == (rows == 0, rows <= 1)
        assert plan(M, N, K, 1).as_dict() == p.as_dict()  # float32 outputs take the same
        assert N > p.features and N % p.features and (M > p.rows or rows < 2) and M % p.rows
        assert -(-K // 128) > (p.waves * p.ring if p.kind == skg.SKINNY_LINEAR_STREAM else 8) and K % 128


def test_python_helpers_refuse(skg):  # noqa: F811
    x, w, s = torch.zeros(2, 16, dtype=torch.int8), torch.zeros(8, 16, dtype=torch.int8), torch.ones(8)
    with pytest.raises(ValueError, match="GPU"):
        skg.linear(x, w, x_scale=s[:2], w_scale=s)
    with pytest.raises(TypeError):
        skg.quantize_int8(x)
    with pytest.raises(ValueError, match="GPU"):
        skg.quantize_int8(x.to(torch.bfloat16))
    with pytest.raises(ValueError, match="quant"):
        from torch._subclasses.fake_tensor import FakeTensorMode

        with FakeTensorMode():
            skg.rms_norm(torch.empty(2, 16, dtype=torch.bfloat16, device="cuda"),
                         torch.empty(16, dtype=torch.bfloat16, device="cuda"), quant="int4")


def test_operators_refuse_cpu_tensors_and_give_shapes_to_a_tracer(skg):  # noqa: F811
    from bf16_skinny_gemm_amd import torch_op as t

    x, w = torch.zeros(2, 3, 32, dtype=torch.bfloat16), torch.zeros(40, 32, dtype=torch.int8)
    n, q, s, ws = torch.zeros(32, dtype=torch.bfloat16), torch.zeros(2, 3, 32, dtype=torch.int8), torch.ones(2, 3), torch.ones(40)
    calls = {"quantize_int8": (x,), "rms_norm_int8": (x, n, 1e-6), "add_rms_norm_int8": (x, x, n, 1e-6),
             "linear_int8": (q, s, w, ws), "linear_gated_int8": (q, s, w, ws, w, ws)}
    for name, args in calls.items():
        with pytest.raises(ValueError, match="skinny::" + name):
            getattr(t, name)(*args)
        got = getattr(t, name)(*(a.to("meta") if isinstance(a, torch.Tensor) else a for a in args))
        got = got if isinstance(got, tuple) else (got,)
        if name.startswith("linear"):
            assert [(tuple(g.shape), g.dtype) for g in got] == [((2, 3, 40), torch.bfloat16)]
            continue
        assert [(tuple(g.shape), g.dtype) for g in got] == [
            ((2, 3, 32), torch.int8), ((2, 3), torch.float32), ((2, 3, 32), torch.bfloat16)][:len(got)]


def test_python_kernels_take_their_own_type(skg):  # noqa: F811
    """Those of the e4m3 projections refuse 8-bit integers, and the other way round, as the C++ ones do."""
    from bf16_skinny_gemm_amd import torch_op as t

    s, ws = torch.ones(2), torch.ones(8)
    for kernels, name, other in ((t._PY_KERNELS, "fp8", torch.int8), (t._PY_KERNELS_MORE, "int8", torch.float8_e4m3fn)):
        for dtype in (other, torch.bfloat16):
            x, w = torch.zeros(2, 16, dtype=dtype), torch.zeros(8, 16, dtype=dtype)
            with pytest.raises(ValueError, match="x must be torch"):
                kernels["linear_" + name](x, s, w, ws)
            with pytest.raises(ValueError, match="x must be torch"):
                kernels["linear_gated_" + name](x, s, w, ws, w, ws)

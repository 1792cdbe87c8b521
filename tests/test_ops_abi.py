"""Argument checks of include/skinny_ops.h and of its Python layers, with no kernel run:
validation comes before any device work, so fake (never dereferenced) pointers serve."""
from __future__ import annotations

import os

import pytest
import torch

X, R, W, RO, Y, S = (0x10000000 * i for i in range(1, 7))
OK, BAD, UNSUPPORTED = 0, -1, -2


@pytest.fixture(scope="module")
def skg():
    from bf16_skinny_gemm_amd.build import LIB_PATH, TORCH_OP_PATH

    if not os.path.exists(LIB_PATH) or not os.path.exists(TORCH_OP_PATH):
        import __graft_entry__

        __graft_entry__.build()
    import bf16_skinny_gemm_amd

    bf16_skinny_gemm_amd.lib()
    return bf16_skinny_gemm_amd


def norm(skg, fp8=False, **kw):
    M, D = kw.get("M", 4), kw.get("D", 256)
    a = dict(x=X, weight=W, y=Y, ldx=D, ldy=D, M=M, D=D, group=0, eps=1e-6)
    if fp8:
        a.update(scale=S)
    a.update(kw)
    if a.pop("res", False):
        a = {**dict(residual=R, residual_out=RO, ldr=D, ldro=D), **a}
    fn = skg.lib().skinny_rms_norm_fp8 if fp8 else skg.lib().skinny_rms_norm_bf16
    return fn(skg.NormArgs(**a), None)


def linear(skg, fp8=False, **kw):
    M, N, K = kw.get("M", 4), kw.get("N", 64), kw.get("K", 256)
    a = dict(x=X, W0=W, y=Y, ldx=K, ldy=N, M=M, N=N, K=K, act=0, out_f32=0, scales=0)
    if fp8:
        a.update(x_scale=S, w0_scale=S + 0x100000, scales=1)
    a.update(kw)
    fn = skg.lib().skinny_linear_fp8 if fp8 else skg.lib().skinny_linear_bf16
    return fn(skg.LinearArgs(**a), None)


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls would launch")


@needs_no_gpu
def test_accepted_arguments_reach_the_device_check(skg):
    """Without a GPU an accepted call ends at the device check, a refused one before it."""
    for fp8 in (False, True):
        assert norm(skg, fp8) == UNSUPPORTED
        assert norm(skg, fp8, res=True) == UNSUPPORTED
        assert norm(skg, fp8, res=True, residual_out=R) == UNSUPPORTED
        assert norm(skg, fp8, res=True, residual_out=X) == UNSUPPORTED
        assert linear(skg, fp8) == UNSUPPORTED
        assert linear(skg, fp8, bias0=R, residual=RO, ldr=64) == UNSUPPORTED
        assert linear(skg, fp8, residual=Y, ldr=64) == UNSUPPORTED
        assert linear(skg, fp8, W1=R, bias1=RO, w1_scale=S + 0x200000 if fp8 else None) == UNSUPPORTED
        assert linear(skg, fp8, ldx=300, ldy=70, out_f32=1) == UNSUPPORTED
        assert linear(skg, fp8, K=0, ldx=0, x=None, W0=None) == UNSUPPORTED
    assert norm(skg, True, group=128) == UNSUPPORTED
    assert norm(skg, y=X) == UNSUPPORTED
    assert linear(skg, True, scales=2) == UNSUPPORTED
    # x and y as the two halves of one merged buffer
    assert norm(skg, ldx=512, ldy=512, y=X + 512) == UNSUPPORTED


def test_empty_calls_are_noops(skg):
    for fp8 in (False, True):
        assert norm(skg, fp8, M=0, x=None, y=None) == OK
        assert norm(skg, fp8, D=0) == OK
        assert linear(skg, fp8, M=0, x=None, y=None) == OK
        assert linear(skg, fp8, N=0) == OK


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(D=-1), dict(x=None), dict(weight=None), dict(y=None), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(ldx=255), dict(ldy=255), dict(x=X + 1),
    dict(weight=W + 1), dict(residual=R), dict(residual_out=RO), dict(res=True, ldr=255),
    dict(res=True, ldro=255), dict(res=True, residual=R + 1), dict(res=True, residual_out=RO + 1),
    dict(res=True, residual_out=Y), dict(res=True, residual_out=R + 2), dict(res=True, residual_out=X + 512),
    dict(res=True, residual_out=X, y=X), dict(res=True, y=R), dict(y=X + 2), dict(y=W), dict(res=True, residual_out=W),
    dict(ldx=512, y=X), dict(ldx=512, ldy=512, y=X + 510), dict(group=64), dict(ldx=1 << 50),
    dict(M=1 << 30, ldx=1 << 35)])
def test_norm_refusals(skg, kw):
    assert norm(skg, **kw) == BAD
    if kw.get("y") != X + 510:
        assert norm(skg, True, **kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(scale=None), dict(scale=S + 2), dict(group=1), dict(group=-128), dict(scale=Y), dict(scale=X),
    dict(scale=W), dict(y=X), dict(res=True, scale=RO), dict(res=True, scale=R + 512)])
def test_norm_fp8_refusals(skg, kw):
    assert norm(skg, True, **kw) == BAD


def test_norm_bf16_takes_no_group(skg):
    assert norm(skg, group=128) == BAD


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(x=None), dict(W0=None), dict(y=None), dict(act=-1), dict(act=5),
    dict(out_f32=2), dict(out_f32=-1), dict(ldx=255), dict(ldy=63), dict(residual=R, ldr=63), dict(bias0=R + 1),
    dict(residual=R + 1, ldr=64), dict(y=Y + 1), dict(out_f32=1, y=Y + 2), dict(bias1=R), dict(y=X), dict(y=W),
    dict(y=W + 64 * 256 - 2), dict(bias0=Y + 100), dict(residual=Y + 2, ldr=64), dict(residual=Y, ldr=65),
    dict(residual=Y, ldr=64, out_f32=1), dict(ldy=1 << 50), dict(M=1 << 30, ldx=1 << 35)])
def test_linear_refusals(skg, kw):
    assert linear(skg, **kw) == BAD
    assert linear(skg, True, **kw) == BAD


def test_linear_gated_refusals(skg):
    for fp8 in (False, True):
        more = dict(w1_scale=S + 0x200000) if fp8 else {}
        assert linear(skg, fp8, W1=R, residual=RO, ldr=64, **more) == BAD
        assert linear(skg, fp8, W1=Y, **more) == BAD
        assert linear(skg, fp8, W1=R, bias1=RO + 1, **more) == BAD
    assert linear(skg, True, W1=R) == BAD  # no scale for it


@pytest.mark.parametrize("kw", [
    dict(scales=0), dict(scales=3), dict(x_scale=None), dict(w0_scale=None), dict(x_scale=S + 2),
    dict(w0_scale=S + 1), dict(y=S), dict(y=S + 0x100000), dict(scales=2, y=S + 16), dict(w0_scale=Y + 256)])
def test_linear_fp8_refusals(skg, kw):
    assert linear(skg, True, **kw) == BAD


def test_linear_bf16_takes_no_scales(skg):
    assert linear(skg, scales=1) == BAD


def test_null_arguments(skg):
    L = skg.lib()
    for fn in (L.skinny_rms_norm_bf16, L.skinny_rms_norm_fp8, L.skinny_linear_bf16, L.skinny_linear_fp8):
        assert fn(None, None) == BAD


def test_python_helpers_refuse(skg):
    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    w = torch.zeros(8, 16, dtype=torch.bfloat16)
    for call in (lambda: skg.rms_norm(x, w[0]), lambda: skg.linear(x, w)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        skg.rms_norm(x.float(), w[0])
    with pytest.raises(TypeError):
        skg.linear(x.float(), w)
    with pytest.raises(TypeError):
        skg.linear(None, w)


def test_operators_refuse_cpu_tensors_by_name(skg):
    from bf16_skinny_gemm_amd import torch_op as t

    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    w = torch.zeros(8, 16, dtype=torch.bfloat16)
    q, s = x.to(torch.float8_e4m3fn), torch.ones(2)
    calls = {"rms_norm": (x, w[0], 1e-6), "add_rms_norm": (x, x, w[0], 1e-6), "rms_norm_fp8": (x, w[0], 1e-6, 0),
             "add_rms_norm_fp8": (x, x, w[0], 1e-6, 128), "linear_act": (x, w), "linear_gated": (x, w, w),
             "linear_fp8": (q, s, w.to(torch.float8_e4m3fn), torch.ones(8)),
             "linear_gated_fp8": (q, s, w.to(torch.float8_e4m3fn), torch.ones(8), w.to(torch.float8_e4m3fn),
                                  torch.ones(8))}
    for name, args in calls.items():
        with pytest.raises(ValueError, match="skinny::" + name):
            getattr(t, name)(*args)


def test_operators_give_shapes_to_a_tracer(skg):
    from bf16_skinny_gemm_amd import torch_op as t

    x = torch.empty(2, 3, 300, dtype=torch.bfloat16, device="meta")
    w = torch.empty(40, 300, dtype=torch.bfloat16, device="meta")
    n = torch.empty(300, dtype=torch.bfloat16, device="meta")
    assert t.rms_norm(x, n, 1e-6).shape == x.shape
    y, h = t.add_rms_norm(x, x, n, 1e-6)
    assert y.shape == h.shape == x.shape and h.dtype == torch.bfloat16
    for group, shape in ((0, (2, 3)), (128, (2, 3, 3))):
        q, s = t.rms_norm_fp8(x, n, 1e-6, group)
        assert q.dtype == torch.float8_e4m3fn and s.shape == shape and s.dtype == torch.float32
        q, s, h = t.add_rms_norm_fp8(x, x, n, 1e-6, group)
        assert q.shape == h.shape == x.shape and s.shape == shape
    assert t.linear_act(x, w).shape == (2, 3, 40)
    assert t.linear_gated(x, w, w, out_f32=True).dtype == torch.float32
    q, wq = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
    s, ws = torch.empty(2, 3, device="meta"), torch.empty(40, device="meta")
    assert t.linear_fp8(q, s, wq, ws).dtype == torch.bfloat16
    assert t.linear_gated_fp8(q, s, wq, ws, wq, ws).shape == (2, 3, 40)
    with pytest.raises(ValueError):
        t.rms_norm_fp8(x, n, 1e-6, 64)


def test_python_helpers_refuse_sizes_past_31_bits(skg):
    """The argument structures hold 32 bits and would cut them off without a word (tensors
    without memory: the sizes are refused before an address is asked for)."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    bf, big = torch.bfloat16, 2 ** 32 + 5
    with FakeTensorMode():
        one, tall, wide = (torch.empty(*s, dtype=bf, device="cuda") for s in ((1,), (big, 1), (1, big)))
        for call in (lambda: skg.rms_norm(tall, one), lambda: skg.rms_norm(wide, wide[0]),
                     lambda: skg.linear(tall, one[None]), lambda: skg.linear(one[None], tall),
                     lambda: skg.linear(wide, wide)):
            with pytest.raises(ValueError, match="31 bits"):
                call()

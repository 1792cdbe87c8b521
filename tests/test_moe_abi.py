"""Argument checks of include/skinny_moe.h and of its Python layers, with no kernel run:
validation comes before any device work, so fake (never dereferenced) pointers serve."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest
import torch

from .test_ops_abi import BAD, OK, UNSUPPORTED, needs_no_gpu, skg  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
X, IDS, WTS, GATE, UP, DOWN, GS, US, DS, RES, Y, WS = ((i + 1) << 36 for i in range(12))


def route(skg, **kw):  # noqa: F811
    a = dict(logits=X, ids=IDS, weights=WTS, ldl=96, M=4, E=96, k=8, score=0, groups=1, kept=1, renormalize=1, scale=1.0)
    a.update(kw)
    return skg.lib().skinny_route(skg.RouteArgs(**a), None)


def experts(skg, kind=0, **kw):  # noqa: F811
    M, E, k, H, I = (kw.get(n, v) for n, v in (("M", 4), ("E", 8), ("k", 2), ("H", 256), ("I", 128)))
    a = dict(x=X, ids=IDS, weights=WTS, w_gate=GATE, w_up=UP, w_down=DOWN, y=Y, workspace=WS, workspace_bytes=1 << 30,
             ldx=H, ldy=H, up_stride=H * I, down_stride=H * I, M=M, E=E, k=k, H=H, I=I, act=4, type=kind)
    if kind:
        a.update(gate_scale=GS, up_scale=US, down_scale=DS, up_scale_stride=I, down_scale_stride=H)
    a.update(kw)
    return skg.lib().skinny_experts(skg.ExpertsArgs(**a), None)


@needs_no_gpu
def test_accepted_arguments_reach_the_device_check(skg):  # noqa: F811
    """Without a GPU an accepted call ends at the device check, a refused one before it."""
    for kw in ({}, dict(bias=GATE), dict(ldl=100), dict(E=1, k=1, ldl=1), dict(E=1024, k=64, ldl=1024, groups=64, kept=4),
               dict(score=1, renormalize=0, scale=-2.5), dict(groups=8, kept=1, k=8)):
        assert route(skg, **kw) == UNSUPPORTED, kw
    for kind in range(4):
        for kw in ({}, dict(residual=RES, ldr=256), dict(residual=Y, ldr=256), dict(E=1, k=32), dict(E=1024), dict(M=1000),
                   dict(ldx=300, ldy=301), dict(H=3, I=5), dict(up_stride=256 * 128 + 7), dict(w_up=GATE + 256 * 128 * 2),
                   dict(act=0)):
            assert experts(skg, kind, **kw) == UNSUPPORTED, (kind, kw)
    need = skg.skinny_experts_workspace_bytes(4, 2, 8, 128)
    assert experts(skg, workspace_bytes=need) == UNSUPPORTED


def test_empty_calls_are_noops(skg):  # noqa: F811
    assert route(skg, M=0, logits=None, ids=None, weights=None) == OK
    assert experts(skg, M=0, x=None, y=None, workspace=None, workspace_bytes=0) == OK


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(E=0), dict(E=1025, ldl=1025), dict(k=0), dict(k=65), dict(k=97), dict(k=9, groups=12), dict(groups=0),
    dict(groups=5), dict(groups=96 * 2), dict(E=130, ldl=130, groups=65), dict(kept=0), dict(kept=2), dict(score=2), dict(score=-1),
    dict(renormalize=2), dict(scale=float("nan")), dict(scale=float("inf")), dict(logits=None), dict(ids=None),
    dict(weights=None), dict(ldl=95), dict(logits=X + 2), dict(ids=IDS + 1), dict(weights=WTS + 2), dict(bias=GATE + 2),
    dict(ids=X), dict(weights=X + 95 * 4), dict(ids=WTS + 4), dict(bias=IDS), dict(bias=WTS - 4), dict(ldl=1 << 50),
    dict(M=1 << 30, ldl=1 << 35)])
def test_route_refusals(skg, kw):  # noqa: F811
    assert route(skg, **kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(H=0), dict(I=0), dict(H=-1), dict(act=5), dict(act=-1),
    dict(x=None), dict(ids=None), dict(weights=None), dict(w_gate=None), dict(w_up=None), dict(w_down=None), dict(y=None),
    dict(workspace=None), dict(workspace_bytes=0), dict(ldx=255), dict(ldy=255), dict(residual=RES, ldr=255),
    dict(up_stride=256 * 128 - 1), dict(down_stride=256 * 128 - 1), dict(up_stride=-(1 << 40)), dict(up_stride=1 << 50),
    dict(x=X + 1), dict(y=Y + 1), dict(residual=RES + 1, ldr=256), dict(ids=IDS + 2), dict(weights=WTS + 1),
    dict(workspace=WS + 8), dict(y=X), dict(y=IDS), dict(y=WTS + 8), dict(y=GATE + 4096), dict(y=DOWN + 256 * 128 * 7),
    dict(y=WS + 64), dict(workspace=X), dict(workspace=GATE + 16), dict(workspace=RES + 16, residual=RES, ldr=256),
    dict(residual=Y + 2, ldr=256), dict(residual=Y, ldr=257), dict(ldx=1 << 50), dict(M=1 << 30, ldx=1 << 35)])
def test_experts_refusals(skg, kw):  # noqa: F811
    for kind in range(4):
        assert experts(skg, kind, **kw) == BAD, kind


@pytest.mark.parametrize("kw", [dict(gate_scale=None), dict(up_scale=None), dict(down_scale=None), dict(gate_scale=GS + 2),
                                dict(up_scale_stride=127), dict(down_scale_stride=255), dict(y=GS), dict(y=DS + 512),
                                dict(workspace=US)])
def test_experts_scale_refusals(skg, kw):  # noqa: F811
    for kind in (1, 3):
        assert experts(skg, kind, **kw) == BAD


def test_experts_types(skg):  # noqa: F811
    assert experts(skg, 4) == experts(skg, -1) == BAD
    assert experts(skg, 0, gate_scale=GS) == experts(skg, 0, down_scale=GS) == BAD
    assert experts(skg, 2, up_scale_stride=1) == BAD      # 1 x 2 blocks
    assert experts(skg, 0, w_gate=GATE + 1) == BAD


def test_workspace_bytes(skg):  # noqa: F811
    f = skg.skinny_experts_workspace_bytes
    assert f(0, 2, 8, 128) == f(4, 0, 8, 128) == f(4, 33, 8, 128) == f(4, 2, 0, 128) == f(4, 2, 8, 0) == f(-1, 2, 8, 128) == 0
    assert f(1, 1, 1, 1) >= 2 and f(4, 2, 8, 128) >= 4 * 2 * 128 * 2
    # one pass at a time: h, two sets of 16 outputs for 256 blocks and every row, and little more
    assert f(128, 8, 288, 1024) == f(10 ** 6, 8, 288, 1024) < 128 * 8 * 1024 * 4 + 2 * 256 * 128 * 64 + (1 << 16)
    sizes = [f(m, 4, 64, 96) for m in range(1, 200)]
    assert sizes == sorted(sizes)
    need = f(4, 2, 8, 128)
    assert experts(skg, workspace_bytes=need - 1) == BAD


def test_null_arguments(skg):  # noqa: F811
    assert skg.lib().skinny_route(None, None) == skg.lib().skinny_experts(None, None) == BAD


def test_python_helpers_refuse(skg):  # noqa: F811
    x, i, f = torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    w = torch.zeros(4, 8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        skg.route(f, 1)
    with pytest.raises(ValueError, match="GPU"):
        skg.experts(x, i, f, w, w, w)
    with pytest.raises(TypeError):
        skg.route(x, 1)
    with pytest.raises(skg.SkinnyError):
        skg.experts_workspace(4, 40, 8, 128, "cpu")
    assert skg.experts_workspace(4, 2, 8, 128, "cpu").numel() == skg.skinny_experts_workspace_bytes(4, 2, 8, 128)


def test_operators_refuse_cpu_tensors_and_give_shapes_to_a_tracer(skg):  # noqa: F811
    from bf16_skinny_gemm_amd import torch_op as t

    x, i, f = torch.zeros(2, 3, 16, dtype=torch.bfloat16), torch.zeros(2, 3, 2, dtype=torch.int32), torch.zeros(2, 3, 2)
    w, d = torch.zeros(4, 8, 16, dtype=torch.bfloat16), torch.zeros(4, 16, 8, dtype=torch.bfloat16)
    for name, args in (("route", (f, 2)), ("experts", (x, i, f, w, w, d))):
        with pytest.raises(ValueError, match="skinny::" + name):
            getattr(t, name)(*args)
    ids, weights = t.route(f.to("meta"), 1)
    assert ids.shape == weights.shape == (2, 3, 1) and ids.dtype == torch.int32 and weights.dtype == torch.float32
    y = t.experts(*(a.to("meta") for a in (x, i, f, w, w, d)))
    assert y.shape == x.shape and y.dtype == torch.bfloat16


def test_moe_validation_under_asan_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    exe = str(tmp_path / "moe_fuzz")
    build = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
             "-D__HIP_PLATFORM_AMD__=1", "-I", os.path.join(ROOT, "include"),
             "-I", "/opt/rocm/include", os.path.join(ROOT, "tests", "sanitize", "moe_fuzz.cpp"), "-o", exe]
    res = subprocess.run(build, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, (res.stdout + res.stderr)[-4000:]
    assert "moe validation: ok" in res.stdout

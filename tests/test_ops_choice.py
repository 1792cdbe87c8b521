"""The choice of a projection's kernel (skinny_linear_default_plan): no device is needed, and
the addresses are never followed."""
from __future__ import annotations

import ctypes

import pytest

from .linear_choices import CHOICES

X, W0, W1, Y, XS, WS0, WS1 = ((i + 1) << 40 for i in range(7))


@pytest.fixture(scope="module")
def skg():
    import os

    from bf16_skinny_gemm_amd.build import LIB_PATH

    if not os.path.exists(LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    import bf16_skinny_gemm_amd

    return bf16_skinny_gemm_amd


def call(skg, M, N, K, scales=0, gated=False, f32=False, **kw):
    a = dict(x=X, W0=W0, y=Y, ldx=K, ldy=N, M=M, N=N, K=K, act=0, out_f32=f32, scales=scales)
    if gated:
        a.update(W1=W1)
    if scales:
        a.update(x_scale=XS, w0_scale=WS0, w1_scale=WS1 if gated else None)
    a.update(kw)
    return skg.LinearArgs(**a)


@pytest.mark.parametrize("key", CHOICES)
def test_every_offered_kernel_is_chosen_at_some_size(skg, key):
    scales, gated, rows, f32 = key
    plans = [skg.skinny_linear_default_plan(call(skg, M, N, K, scales, gated, f32)) for M, N, K in CHOICES[key]]
    assert [p.index for p in plans] == list(range(plans[0].count))
    for p, (M, N, K) in zip(plans, CHOICES[key]):
        assert (M <= 8, M <= 16) == (rows == 0, rows <= 1)
        assert p.kind in (skg.SKINNY_LINEAR_STREAM, skg.SKINNY_LINEAR_TILE)
        stages = -(-K * (1 if scales else 2) // 128)
        assert N > p.features and N % p.features and (M > p.rows or rows < 2) and M % p.rows
        assert stages > (p.waves * p.ring if p.kind == skg.SKINNY_LINEAR_STREAM else 8)
        assert K * (1 if scales else 2) % 128


def test_the_sets_are_all_there(skg):
    """Float32 outputs are a set of their own for more than 16 rows of 8-bit x only."""
    assert set(CHOICES) == {(s, g, r, f) for s in range(3) for g in range(2) for r in range(3)
                            for f in range(2 if s and r == 2 else 1)}
    for (scales, gated, rows, f32), sizes in CHOICES.items():
        if (scales, gated, rows, 1) in CHOICES:
            continue
        for M, N, K in sizes:
            assert (skg.skinny_linear_default_plan(call(skg, M, N, K, scales, gated, True)).as_dict()
                    == skg.skinny_linear_default_plan(call(skg, M, N, K, scales, gated, False)).as_dict())


def test_plans_of_other_devices_and_alignments(skg):
    for cus in (1, 32, 304, 2 ** 31 - 1):
        p = skg.skinny_linear_default_plan(call(skg, 300, 1000, 1024), cus)
        assert 0 <= p.index < p.count
    for kw in (dict(x=X + 2), dict(W0=W0 + 8), dict(K=1023, ldx=1024), dict(ldx=1025)):
        p = skg.skinny_linear_default_plan(call(skg, **{**dict(M=300, N=1000, K=1024), **kw}))
        assert (p.kind, p.index, p.count) == (skg.SKINNY_LINEAR_ELEMENTS, -1, 0)
    assert "kind=0" in repr(p)


@pytest.mark.parametrize("kw", [dict(M=0), dict(N=0), dict(M=-1), dict(y=None), dict(scales=3), dict(scales=-1),
                                dict(scales=1, x_scale=None), dict(act=9), dict(ldx=8), dict(y=X), dict(y=Y + 1)])
def test_plan_refusals(skg, kw):
    with pytest.raises(skg.SkinnyError):
        skg.skinny_linear_default_plan(call(skg, **{**dict(M=4, N=64, K=256), **kw}))


def test_plan_refuses_no_device_and_no_arguments(skg):
    a, p = call(skg, 4, 64, 256), skg.LinearPlan()
    with pytest.raises(skg.SkinnyError):
        skg.skinny_linear_default_plan(a, 0)
    f = skg.lib().skinny_linear_default_plan
    assert f(None, 256, ctypes.byref(p)) == f(ctypes.byref(a), 256, None) == -1

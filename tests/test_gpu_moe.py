"""The router and the experts of include/skinny_moe.h against their definitions in 64 bits, on
the GPU.

Tolerances are counted from the roundings: half a step of the output (2^-8 of a bfloat16 value),
the same for h between the two projections, one rounding of the running magnitude per term of a
float32 sum, and the activations' (a few roundings, carried by a slope of at most 1.13). The
choice of experts has no tolerance.
"""
from __future__ import annotations

import math

import pytest
import torch

from .experts_choices import CHOICES
from .test_gpu_ops import BF16, F32, act_ref, bits, filled, gen, ops, skg, walled, walls_hold  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- router ------------------------------------------------------------------

def route_ref(logits, k, score, bias, groups, kept, renormalize, scale):
    """In 64 bits, one row after the other, on the CPU."""
    v = logits.double().cpu()
    M, E = v.shape
    ids, weights = torch.zeros(M, k, dtype=torch.int32), torch.zeros(M, k, dtype=torch.float64)
    for m in range(M):
        if score == "softmax":
            top = v[m].max()
            s = torch.exp(v[m] - top) if top > -math.inf else torch.zeros(E, dtype=torch.float64)
            s = s / s.sum() if s.sum() != 0 else s
        else:
            s = torch.sigmoid(v[m])
        rank = (v[m] if bias is None else s + bias.double().cpu()).tolist()
        rank = [math.inf if math.isnan(r) else r for r in rank]
        experts = list(range(E))
        if groups > 1:
            size = E // groups
            parts = [sorted(rank[g * size:(g + 1) * size], reverse=True) for g in range(groups)]
            best = [p[0] if bias is None else sum(p[:2]) for p in parts]
            left = sorted(range(groups), key=lambda g: (-best[g], g))[:kept]
            experts = [e for e in experts if e // size in left]
        chosen = sorted(experts, key=lambda e: (-rank[e], e))[:k]
        w = s[chosen]
        if renormalize:
            w = w / w.sum() if w.sum() != 0 else torch.zeros_like(w)
        ids[m], weights[m] = torch.tensor(chosen, dtype=torch.int32), w * scale
    return ids, weights


def check_route(skg, logits, k, score="softmax", bias=None, groups=1, kept=1, renormalize=True, scale=1.0):  # noqa: F811
    M, E = logits.shape
    ids, weights = skg.route(logits, k, score, bias, groups, kept, renormalize, scale)
    want, wref = route_ref(logits, k, score, bias, groups, kept, renormalize, scale)
    assert torch.equal(ids.cpu(), want), [(m, ids[m].tolist(), want[m].tolist()) for m in range(M)
                                          if not torch.equal(ids[m].cpu(), want[m])][:3]
    # exp: 2 roundings of its value and those of its argument (below 2^7 here); its sum one a term
    # and as much; a quotient, and the scale
    tol = (2 * 128 + 2 * (E if score == "softmax" and not renormalize else k) + 8) * F32
    assert ((weights.double().cpu() - wref).abs() <= tol * wref.abs() + 1e-37).all()


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("with_bias", (False, True))
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (5, 3), (63, 8), (64, 64), (65, 4), (128, 1), (129, 8), (192, 6), (193, 8),
                                 (288, 8), (300, 16), (384, 8), (385, 9), (512, 8), (513, 10), (1000, 8), (1024, 64)])
def test_route(skg, E, k, score, with_bias):  # noqa: F811
    for M in (1, 6, 33):
        logits = 2.0 * torch.randn(M, E, generator=gen(E + M), device="cuda")
        bias = 0.2 * torch.randn(E, generator=gen(E), device="cuda") if with_bias else None
        check_route(skg, logits, k, score, bias, renormalize=bool(M % 2), scale=2.5)


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("with_bias", (False, True))
@pytest.mark.parametrize("E,groups,kept,k", [(4, 2, 1, 2), (64, 64, 7, 7), (256, 8, 4, 8), (160, 8, 3, 6), (60, 4, 4, 16),
                                             (1024, 64, 10, 64), (999, 27, 5, 9), (12, 1, 1, 12)])
def test_route_by_groups(skg, E, groups, kept, k, score, with_bias):  # noqa: F811
    logits = 2.0 * torch.randn(29, E, generator=gen(E), device="cuda")
    bias = 0.2 * torch.randn(E, generator=gen(E + 1), device="cuda") if with_bias else None
    check_route(skg, logits, k, score, bias, groups, kept)


@pytest.mark.parametrize("groups", (1, 4))
@pytest.mark.parametrize("with_bias", (False, True))
def test_route_ties_go_to_the_lowest_index(skg, with_bias, groups):  # noqa: F811
    logits = torch.randint(-2, 3, (40, 96), generator=gen(1), device="cuda").float()
    logits[0] = 0.0
    logits[1] = -0.0
    logits[1, ::2] = 0.0
    bias = torch.zeros(96, device="cuda") if with_bias else None
    for score in ("softmax", "sigmoid"):
        check_route(skg, logits, 10, score, bias, groups, max(1, groups // 2))


def test_route_ranks_closer_than_float32(skg):  # noqa: F811
    """Scores + bias whose float32 sums are equal, or in the other order, are told apart."""
    logits = torch.zeros(4, 70, device="cuda")
    logits[:, 60:] = 1e-6 * torch.arange(10, device="cuda")
    logits[1, 3] = 2e-7
    logits[2] = 40.0 + torch.arange(70, device="cuda")
    bias = torch.full((70,), 8.0, device="cuda")
    for score in ("softmax", "sigmoid"):
        check_route(skg, logits[:3], 12, score, bias)
    check_route(skg, logits[2:3], 5, "sigmoid")  # no bias: by the logits, though every score is 1


def test_route_special_rows(skg):  # noqa: F811
    inf, nan = float("inf"), float("nan")
    x = torch.randn(7, 96, generator=gen(5), device="cuda")
    x[1] = -inf                    # nothing is left
    x[2] = -inf
    x[2, 50] = 1.0                 # one is left
    x[3, 9] = inf
    x[4, 77] = nan
    x[5, 10:] = -inf
    x[6] = torch.finfo(torch.float32).min
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            ids, w = skg.route(x, 4, score, renormalize=renormalize)
            assert ids[1].tolist() == [0, 1, 2, 3] and ids[6].tolist() == [0, 1, 2, 3]
            assert ids[2].tolist() == [50, 0, 1, 2] and int(ids[3, 0]) == 9 and int(ids[4, 0]) == 77
            assert (w[1] == 0).all() and (w[2, 1:] == 0).all()
            assert w[0].isfinite().all() and w[5].isfinite().all()
            if score == "softmax":
                assert float(w[2, 0]) == 1.0 and w[3].isnan().all() and w[4].isnan().all()
                assert ((w[6] - (1 / 4 if renormalize else 1 / 96)).abs() < 1e-7).all()
            else:
                assert w[4, 0].isnan() and (w[6] == 0).all()
    check_route(skg, x[[0, 2, 5]], 8)
    bias = 0.1 * torch.randn(96, generator=gen(6), device="cuda")
    for score in ("softmax", "sigmoid"):
        check_route(skg, x[[0, 1, 2, 5, 6]], 8, score, bias, 8, 3)
        ids, _ = skg.route(x[4:5], 4, "sigmoid", bias, 8, 3)
        assert int(ids[0, 0]) == 77
    bias[5] = -inf
    check_route(skg, x[:1, :64].contiguous(), 64, "sigmoid", bias[:64].contiguous())


def test_route_small_sigmoids(skg):  # noqa: F811
    """Scores below the normal float32 values keep what bits they have: here 2^-149 / exp(-95) of
    them, which is 2^-12, half of it for each of two scores and twice as much for their sum."""
    logits = -95.0 + torch.rand(9, 70, generator=gen(4), device="cuda")
    ids, w = skg.route(logits, 6, "sigmoid")
    want, wref = route_ref(logits, 6, "sigmoid", None, 1, 1, True, 1.0)
    assert torch.equal(ids.cpu(), want) and ((w.double().cpu() - wref).abs() <= 2.0 ** -11 * wref).all()


@pytest.mark.parametrize("depth", (85.0, 100.0, 120.0, 300.0, 600.0))
def test_route_weights_far_below_the_top(skg, depth):  # noqa: F811
    """Renormalized weights are quotients of the scores however small these are: float32 holds
    none of exp(-120)."""
    logits = -depth + torch.rand(9, 70, generator=gen(4), device="cuda")
    check_route(skg, logits, 6, "sigmoid", scale=2.5)
    logits[3:, 11] = -depth + 3.0
    logits[6:, 69] = 0.0                       # the softmax's top
    check_route(skg, logits, 6, "sigmoid")
    bias = torch.rand(70, generator=gen(5), device="cuda")
    bias[69] = -10.0                           # is not chosen
    for score in ("softmax", "sigmoid"):
        check_route(skg, logits, 6, score, bias)
        check_route(skg, logits, 6, score, bias, 7, 3)
    logits[:, :40] = -math.inf
    for score in ("softmax", "sigmoid"):
        check_route(skg, logits, 64, score, bias)


@pytest.mark.parametrize("mask", (-math.inf, torch.finfo(torch.float32).min, -1e4))
def test_route_of_masked_choices(skg, mask):  # noqa: F811
    """Where every chosen expert is masked the weights are 0, also below a finite top."""
    logits = torch.full((3, 32), mask, device="cuda")
    logits[1:, 31] = 4.0
    bias = torch.zeros(32, device="cuda")
    bias[31] = -20.0
    for score in ("softmax", "sigmoid"):
        ids, w = skg.route(logits, 5, score, bias)
        assert ids.tolist() == [[0, 1, 2, 3, 4]] * 3
        # the softmax of a row of one finite value is even
        assert (w[1:] == 0).all() and ((w[0] - 0.2).abs() < 1e-7 if score == "softmax" and mask > -math.inf else w[0] == 0).all()


@pytest.mark.parametrize("groups,kept", ((1, 1), (8, 3)))
@pytest.mark.parametrize("renormalize", (False, True))
def test_route_of_rows_with_nan_and_a_bias(skg, renormalize, groups, kept):  # noqa: F811
    """A NaN or +infinity anywhere in a row makes its softmax weights NaN, chosen or not."""
    logits = torch.randn(5, 96, generator=gen(3), device="cuda")
    logits[1, 95] = math.nan
    logits[2, 40] = math.inf
    logits[3] = -math.inf
    logits[3, 90] = math.nan
    bias = torch.linspace(1.0, -1.0, 96, device="cuda")
    _, w = skg.route(logits, 4, "softmax", bias, groups, kept, renormalize)
    assert w[1:4].isnan().all() and w[[0, 4]].isfinite().all()


def test_route_strides_and_shapes(skg, ops):  # noqa: F811
    flat, view = walled(7, 96, 131, torch.float32)
    view.copy_(torch.randn(7, 96, generator=gen(1), device="cuda"))
    a, b = ops.route(view, 6), ops.route(view.contiguous().view(7, 1, 96), 6)
    assert b[0].shape == b[1].shape == (7, 1, 6)
    assert torch.equal(a[0], b[0].view(7, 6)) and torch.equal(a[1], b[1].view(7, 6))
    check_route(skg, view, 6)
    got = ops.route(torch.empty(0, 96, device="cuda"), 6)
    assert got[0].shape == (0, 6)


def test_route_many_rows(skg):  # noqa: F811
    x = torch.randn(70000, 64, generator=gen(1), device="cuda")
    ids, w = skg.route(x, 4)
    assert torch.equal(ids.long(), torch.sort(x, dim=1, descending=True, stable=True).indices[:, :4])
    assert ((w.sum(dim=1) - 1).abs() < 1e-6).all()


# ---- experts -------------------------------------------------------------------

KINDS = ("bf16", "row", "block", "int8")


def stack(q, pad):
    """The stack [E, N, K] with `pad` values between its parts, which are NaN (or large)."""
    E, N, K = q.shape
    if q.dtype == torch.int8:
        flat = torch.full((E * (N * K + pad) + 64,), 0x55, dtype=torch.int8, device="cuda")
    else:
        flat = torch.full((E * (N * K + pad) + 64,), float("nan"), device="cuda").to(q.dtype)
    out = flat[32:32 + E * (N * K + pad)].view(E, N * K + pad)[:, :N * K].view(E, N, K) if E == 1 else \
        flat.as_strided((E, N, K), (N * K + pad, K, 1), 32)
    out.copy_(q)
    return out


def make_weight(g, E, N, K, kind, pad):
    """Stored weights, their scales, and both wide."""
    v = torch.randn(E, N, K, generator=g, device="cuda")
    if kind == "bf16":
        q = (v / math.sqrt(K)).to(torch.bfloat16)
        return stack(q, pad), None, q.double()
    q = (v * 40).clamp(-128, 127).round().to(torch.int8) if kind == "int8" else (v * 60).to(torch.float8_e4m3fn)
    nb, kb = -(-N // 128), -(-K // 128)
    s = (torch.rand(*((E, nb, kb) if kind == "block" else (E, N)), generator=g, device="cuda") + 0.5) / 50 / math.sqrt(K)
    if kind == "block":
        wide = s.double().repeat_interleave(128, dim=1)[:, :N].repeat_interleave(128, dim=2)[:, :, :K]
    else:
        wide = s.double()[:, :, None]
    return stack(q, pad), s, q.double() * wide


def check_experts(skg, M, E, k, H, I, kind, *, act="silu", residual=False, ids=None, ldx=None, ldy=None, pad=0, shift=0,  # noqa: F811
                  seed=0, in_place=False, merged=False, h_rounding=BF16):
    g = gen(seed)
    x = torch.randn(M, H, generator=g, device="cuda").to(torch.bfloat16)
    gate, gs, gw = make_weight(g, E, I, H, kind, pad)
    up, us, uw = make_weight(g, E, I, H, kind, pad)
    down, ds, dw = make_weight(g, E, H, I, kind, pad)
    if merged:
        both = torch.cat([gate, up], dim=1)
        gate, up = both[:, :I], both[:, I:]
        if kind != "bf16":
            scales = torch.cat([gs, us], dim=1)
            gs, us = scales[:, :gs.shape[1]], scales[:, gs.shape[1]:]
    if ids is None:
        ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(M)]).to(torch.int32)
    named = torch.zeros(E, dtype=torch.bool, device="cuda")
    inside = (ids >= 0) & (ids < E)
    named[ids[inside].long()] = True
    if kind != "int8":  # experts that nobody names are not read
        for w in (gate, up, down):
            w[~named] = torch.full((1,), float("nan"), device="cuda").to(w.dtype)
    weights = torch.rand(*ids.shape, generator=g, device="cuda") - 0.2
    r = torch.randn(M, H, generator=g, device="cuda").to(torch.bfloat16) if residual else None
    oflat, ov = walled(M, H, ldy, torch.bfloat16, shift)
    rv = None
    if in_place:
        ov.copy_(r)
        rv = ov
    elif residual:
        rv = filled(r, ldy, shift)
    space = skg.skinny_experts_workspace_bytes(M, k, E, I)
    work = torch.full((space + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read too early
    y = skg.experts(filled(x, ldx, shift), ids, weights, gate, up, down, gs, us, ds, rv, act, out=ov,
                    workspace=work[:space])
    torch.cuda.synchronize()
    assert walls_hold(oflat, ov) and (work[space:] == 0xFF).all()
    xd = x.double()
    ref = r.double() if residual else torch.zeros(M, H, dtype=torch.float64, device="cuda")
    err, mag = torch.zeros_like(ref), ref.abs()
    for e in named.nonzero().flatten().tolist():
        m, j = (ids == e).nonzero(as_tuple=True)
        z, u = xd[m] @ gw[e].t().contiguous(), xd[m] @ uw[e].t().contiguous()
        ez, eu = ((2 * H + 64) * F32 * (xd[m].abs() @ w[e].abs().t().contiguous()) for w in (gw, uw))
        a = act_ref(z, act)
        ea = 1.13 * ez + (32 + (3 * z ** 2 if act == "gelu" else 0)) * F32 * a.abs()
        ea = ea + (32 * F32 * z.abs() if act in ("silu", "gelu_tanh") else 0)
        h = a * u
        eh = ea * u.abs() + (a.abs() + ea) * eu
        eh = eh + (h.abs() + eh) * (h_rounding + 4 * F32)
        w = weights[m, j].double()[:, None]
        ref.index_add_(0, m, w * (h @ dw[e].t().contiguous()))
        down_abs = dw[e].abs().t().contiguous()
        err.index_add_(0, m, w.abs() * (eh @ down_abs))
        mag.index_add_(0, m, w.abs() * ((h.abs() + eh) @ down_abs))
    err = err + (2 * I + 2 * k + 80) * F32 * mag
    err = (err + ref.abs() * BF16 + 1e-38) * (1 + 2 * BF16)
    bad = ~((y.double() - ref).abs() <= err)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), y[bad][:4].tolist(), ref[bad][:4].tolist())
    return y


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", (1, 2, 3, 8, 9, 16, 17, 31, 40, 64, 65, 100, 128))
def test_experts_tokens(skg, M, kind):  # noqa: F811
    check_experts(skg, M, 16, 4, 512, 256, kind, seed=M)
    check_experts(skg, M, 67, 2, 272, 144, kind, act="gelu_tanh", residual=True, seed=M + 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,I", [(16, 16), (128, 128), (256, 48), (48, 400), (1024, 512), (2064, 144), (144, 2064), (4096, 128),
                                 (512, 1408)])
def test_experts_widths(skg, H, I, kind):  # noqa: F811
    for M in (1, 7, 33):
        check_experts(skg, M, 8, 3, H, I, kind, seed=H + M, residual=M == 7)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (3, 1), (32, 32), (64, 8), (65, 7), (300, 8), (1024, 3)])
def test_experts_counts(skg, E, k, kind):  # noqa: F811
    for M in (1, 5, 64, 128):
        check_experts(skg, M, E, k, 128, 96, kind, seed=E + M, act="gelu")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("act", ("none", "relu", "gelu", "gelu_tanh", "silu"))
def test_experts_activations(skg, act, kind):  # noqa: F811
    for M in (2, 50):
        check_experts(skg, M, 12, 3, 256, 128, kind, act=act, seed=7)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", (1, 6, 70, 128))
def test_experts_that_do_not_exist(skg, M, kind):  # noqa: F811
    """Ids outside the range add nothing, whole rows of them too."""
    ids = torch.randint(-2, 12, (M, 5), generator=gen(M), device="cuda", dtype=torch.int32)
    ids[:, 0] = torch.tensor([-2 ** 31, 2 ** 31 - 1, 8, -1, 3, 10 ** 6], device="cuda")[torch.arange(M, device="cuda") % 6].int()
    ids[M // 2] = -1
    check_experts(skg, M, 8, 5, 256, 128, kind, ids=ids, residual=True, seed=3)
    y = check_experts(skg, M, 8, 5, 256, 128, kind, ids=torch.full_like(ids, 9), seed=3)
    assert (y == 0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", (1, 4, 13, 60, 128))
def test_experts_named_twice(skg, M, kind):  # noqa: F811
    """One token may name an expert several times, and all tokens the same one."""
    ids = torch.randint(0, 3, (M, 6), generator=gen(M), device="cuda", dtype=torch.int32)
    check_experts(skg, M, 4, 6, 256, 128, kind, ids=ids, seed=2)
    check_experts(skg, M, 4, 6, 256, 128, kind, ids=torch.full_like(ids, 2), seed=2)
    check_experts(skg, M, 300, 6, 256, 128, kind, ids=ids + 290, seed=2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", (129, 300))
def test_experts_of_more_rows_than_one_pass(skg, M, kind):  # noqa: F811
    check_experts(skg, M, 16, 4, 256, 128, kind, residual=True, ldx=264, ldy=272, seed=M)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,I,ldx,ldy,pad,shift", [(128, 96, 136, 140, 16, 0), (256, 128, 264, 257, 48, 0), (250, 100, 251, 252, 5, 0),
                                                   (136, 40, 136, 136, 0, 0), (77, 33, 80, 78, 1, 1), (128, 96, 130, 129, 16, 1),
                                                   (1, 1, 1, 1, 0, 0), (128, 96, 128, 128, 3, 0)])
def test_experts_strides_and_alignment(skg, H, I, ldx, ldy, pad, shift, kind):  # noqa: F811
    for M in (1, 5, 40):
        check_experts(skg, M, 9, 3, H, I, kind, residual=True, ldx=ldx, ldy=ldy, pad=pad, shift=shift, seed=H + I)


@pytest.mark.parametrize("kind", KINDS)
def test_experts_merged_weights_and_residual_in_place(skg, kind):  # noqa: F811
    for M in (2, 30):
        check_experts(skg, M, 8, 2, 256, 128, kind, merged=True, residual=True, in_place=True, ldy=272, seed=4)


@pytest.mark.parametrize("kind", KINDS)
def test_experts_full_size(skg, kind):  # noqa: F811
    """Whole widths of a decode step, all compute units at work."""
    for M, E, k, H, I in ((1, 24, 8, 4096, 1024), (21, 24, 6, 2048, 1408), (48, 8, 2, 4096, 1536)):
        check_experts(skg, M, E, k, H, I, kind, seed=M)


# For each height of tiles (4, 8, 16 and 32 rows) calls of one wave of pairs and of more, for up to
# 16, 64 and 128 tokens, and widths whose rows of x leave LDS for 6, 4, 3 stages and none.
TILES = {4: (((1, 64, 4), (40, 64, 1), (100, 300, 1), (30, 300, 4), (10, 200, 8)), (512, 9008, 12000, 14000)),
         8: (((12, 16, 4), (50, 16, 1), (100, 32, 1), (16, 30, 6)), (520, 4000, 6000, 7200)),
         16: (((16, 7, 4), (60, 6, 1), (120, 13, 1), (16, 14, 8)), (528, 2000, 2800, 4000)),
         32: (((60, 2, 1), (100, 6, 2), (40, 2, 2)), (512, 1200, 1504, 2000)),
         "32 of 8 bits": (((70, 1, 1), (64, 1, 2)), (512, 1200, 1504, 2000)),
         "32 of 8 bits, wide": (((60, 2, 1), (100, 4, 1)), (2576,))}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", TILES)
def test_experts_tiles(skg, rows, kind):  # noqa: F811
    calls, widths = TILES[rows]
    for M, E, k in calls:
        ids = None
        if k > E:  # the only expert, named twice
            ids = torch.zeros(M, k, dtype=torch.int32, device="cuda")
        for H in widths:
            H = H // 16 * 16
            check_experts(skg, M, E, k, H, 64, kind, ids=ids, residual=True, seed=H + M)
            if H < 1000:
                check_experts(skg, M, E, k, 80, H, kind, ids=ids, seed=H + M)


@pytest.mark.parametrize("kind", range(4))
def test_experts_every_kernel(skg, kind):  # noqa: F811
    """Every kernel that calls choose among, first and second (which of them: test_experts_choice)."""
    for kinds, sizes in CHOICES.items():
        for i, (M, E, k, H) in enumerate(sizes if kind in kinds else ()):
            ids = torch.zeros(M, k, dtype=torch.int32, device="cuda") if k > E else None
            check_experts(skg, M, E, k, H, 80, KINDS[kind], ids=ids, residual=i % 2 == 0, seed=M + H)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", (4, 8))
def test_experts_of_few_rows_hold_h_in_two_parts(skg, rows, kind):  # noqa: F811
    """A bfloat16 value and what it leaves, rounded to bfloat16: off by 2^-16 of h at most."""
    for M, E, k in TILES[rows][0][:4]:
        check_experts(skg, M, E, k, 256, 144, kind, seed=M, h_rounding=BF16 ** 2)
    check_experts(skg, 3, 8, 2, 249, 135, kind, seed=9, h_rounding=BF16 ** 2)  # element by element: in float32


@pytest.mark.parametrize("M,E,H", [(2, 16, 64), (12, 16, 64), (40, 2, 64), (2, 16, 60)])
def test_experts_of_infinite_h(skg, M, E, H):  # noqa: F811
    """An infinite h makes its outputs infinite, not NaN, also where h is held in two parts."""
    I = 32
    x = torch.full((M, H), 2.0 ** 63, device="cuda").to(torch.bfloat16)
    gate, up = torch.zeros(E, I, H, device="cuda"), torch.zeros(E, I, H, device="cuda")
    gate[:, :, 0], up[:, :, 0] = 1.0, 2.0        # 2^63, 2^64: h is 2^127
    gate[:, 3, 0], up[:, 3, 0] = 1.5, 2.0 ** 30  # overflows
    down = torch.full((E, H, I), 1.0, device="cuda")
    down[:, 1] = -1.0
    down[:, 2:, 3] = 0.0
    down[:, 2:] *= 2.0 ** -10
    ids = torch.arange(M, device="cuda").remainder(E).to(torch.int32)[:, None]
    w = [v.to(torch.bfloat16) for v in (gate, up, down)]
    y = skg.experts(x, ids, torch.ones(M, 1, device="cuda"), *w, act="none").float()
    assert (y[:, 0] == math.inf).all() and (y[:, 1] == -math.inf).all()
    assert y[:, 2:].isnan().all()  # infinity times zero


@pytest.mark.parametrize("M,E,H", [(2, 16, 64), (12, 16, 64), (30, 6, 64), (40, 2, 64), (100, 16, 64), (2, 16, 60)])
def test_experts_of_infinite_weights(skg, M, E, H):  # noqa: F811
    """An infinite weight makes its output infinite whatever is left of h behind its first part: nothing
    (the even features), as much as the sign of h, and of the other sign."""
    I = 32
    x = torch.zeros(M, H, device="cuda")
    x[:, :2] = 1.0
    gate, up = torch.zeros(E, I, H, device="cuda"), torch.zeros(E, I, H, device="cuda")
    gate[:, :, 0] = 1.0
    up[:, :, 0] = 1.0
    up[:, 1::4, 1], up[:, 3::4, 1] = 2.0 ** -10, -2.0 ** -10
    up[:, 31] = 0.0                              # h is 0
    down = torch.full((E, H, I), 0.5, device="cuda")
    for n in range(H):
        down[:, n, n % I] = math.inf if n < I else -math.inf
    ids = torch.arange(M, device="cuda").remainder(E).to(torch.int32)[:, None]
    w = [v.to(torch.bfloat16) for v in (gate, up, down)]
    y = skg.experts(x.to(torch.bfloat16), ids, torch.ones(M, 1, device="cuda"), *w, act="none").float()
    n = torch.arange(H, device="cuda")
    assert y[:, n % I == 31].isnan().all()       # 0 times infinity
    assert (y[:, (n % I < 31) & (n < I)] == math.inf).all() and (y[:, (n % I < 31) & (n >= I)] == -math.inf).all()


@pytest.mark.parametrize("kind", KINDS)
def test_experts_outputs_of_several_blocks(skg, kind):  # noqa: F811
    """Sets of outputs that two and many blocks share, and blocks of several sets."""
    for M, E, k, H, I in ((24, 40, 4, 16, 2048), (24, 40, 4, 64, 1024), (9, 12, 4, 1000 // 16 * 16, 640), (70, 30, 4, 144, 1280),
                          (24, 24, 8, 4112, 256), (16, 16, 4, 8192, 128), (2, 8, 2, 5120, 2048)):
        check_experts(skg, M, E, k, H, I, kind, residual=True, seed=H)


@pytest.mark.parametrize("kind", KINDS)
def test_experts_give_the_same_bits_and_rows_are_their_own(skg, kind):  # noqa: F811
    """NaN in one token stays there; the same call gives the same bits."""
    g = gen(8)
    gate, gs, _ = make_weight(g, 12, 128, 256, kind, 0)
    up, us, _ = make_weight(g, 12, 128, 256, kind, 0)
    down, ds, _ = make_weight(g, 12, 256, 128, kind, 0)
    for M in (3, 40, 120):
        x = torch.randn(M, 256, generator=g, device="cuda").to(torch.bfloat16)
        ids, w = skg.route(torch.randn(M, 12, generator=g, device="cuda"), 4)
        call = lambda: skg.experts(x, ids, w, gate, up, down, gs, us, ds)  # noqa: E731
        y = call()
        for _ in range(5):
            assert torch.equal(bits(call()), bits(y))
        x[M // 2, 7] = float("nan")
        z = call()
        keep = torch.arange(M, device="cuda") != M // 2
        assert z[M // 2].isnan().all() and torch.equal(bits(z[keep]), bits(y[keep]))


def test_experts_with_far_weights(skg):  # noqa: F811
    """Experts beyond 2^31 elements and beyond 4 GiB from the first."""
    E, H, I = 600, 2048, 2048
    w = torch.empty(3, E, H, I, dtype=torch.bfloat16, device="cuda")
    w.random_(-3, 4, generator=gen(1))
    x = torch.randn(2, H, generator=gen(2), device="cuda").to(torch.bfloat16)
    ids = torch.tensor([[599, 0], [598, 599]], dtype=torch.int32, device="cuda")
    one = torch.tensor([[2.0 ** -12, 2.0 ** -13]] * 2, device="cuda")
    y = skg.experts(x, ids, one, w[0], w[1], w[2], act="none").double()
    ref, size = torch.zeros_like(y), torch.zeros_like(y)
    for m in range(2):
        for j in range(2):
            g, u, d = (w[i, int(ids[m, j])].double() for i in range(3))
            h = (g @ x[m].double()) * (u @ x[m].double())
            ref[m] += float(one[m, j]) * (d @ h)
            size[m] += float(one[m, j]) * (d.abs() @ h.abs())
    # half a step of h and of y, and the sums: of 2048 terms in float32, h's twice
    assert ((y - ref).abs() <= (BF16 * 1.1 + 3 * 4200 * F32) * size + BF16 * ref.abs()).all()


# ---- as they are used ------------------------------------------------------------

def layer(ops, x, r, p):  # noqa: F811
    """Norm, router, experts onto the residual stream."""
    n, h = ops.add_rms_norm(x, r, p["norm"], 1e-6)
    logits = ops.linear_act(n, p["router"], None, None, "none", True)
    ids, w = ops.route(logits, 4, "sigmoid", p["bias"], 4, 2, True, 2.5)
    return ops.experts(n, ids, w, *p["w"], *p["s"], h), ids, w


def parameters(kind, E=32, H=256, I=128):
    g = gen(11)
    parts = [make_weight(g, E, *s, kind, 0) for s in ((I, H), (I, H), (H, I))]
    return {"norm": torch.ones(H, dtype=torch.bfloat16, device="cuda"),
            "router": torch.randn(E, H, generator=g, device="cuda").to(torch.bfloat16),
            "bias": 0.1 * torch.randn(E, generator=g, device="cuda"),
            "w": [p[0] for p in parts], "s": [p[1] for p in parts], "wide": [p[2] for p in parts]}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", (1, 24, 90))
def test_layer(ops, M, kind):  # noqa: F811
    """The chain on the ids and weights that its router gave; n is what the norm gave, so the
    error is that of the experts: both bfloat16 roundings of half a step and the float32 sums,
    5% of a step, in the norm of each row."""
    p = parameters(kind)
    x, r = (torch.randn(M, 256, generator=gen(9 + i), device="cuda").to(torch.bfloat16) for i in range(2))
    y, ids, w = layer(ops, x, r, p)
    n, h = ops.add_rms_norm(x, r, p["norm"], 1e-6)
    ref = h.double()
    for m in range(M):
        for j in range(4):
            g, u, d = (v[int(ids[m, j])] for v in p["wide"])
            t = (g @ n[m].double()), (u @ n[m].double())
            ref[m] += float(w[m, j]) * (d @ (t[0] * torch.sigmoid(t[0]) * t[1]))
    off = torch.linalg.norm(y.double() - ref, dim=1)
    # a rounding of h changes y by at most BF16 |w| |Wd| |h|: as norms, with room for a Wd whose
    # largest singular value is 3 times its rms one
    assert (off <= 4.2 * BF16 * (torch.linalg.norm(ref, dim=1) + torch.linalg.norm(ref - h.double(), dim=1))).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", (1, 24))
def test_two_graphs_of_the_layer(ops, M, kind):  # noqa: F811
    """Two graphs captured from the same call, replayed in turn with eager calls between."""
    p = parameters(kind)
    x, r = (torch.randn(M, 256, generator=gen(i), device="cuda").to(torch.bfloat16) for i in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(ops, x, r, p)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    got = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            got.append(layer(ops, x, r, p))
    for i in range(4):
        x.copy_(torch.randn(M, 256, generator=gen(20 + i), device="cuda"))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = layer(ops, x, r, p)
        for out in got:
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(out, want))


def test_two_streams_at_once(ops):  # noqa: F811
    """Calls of the operator on two streams have workspaces of their own."""
    p = parameters("bf16", E=64, H=1024, I=512)
    inputs = [[torch.randn(20, 1024, generator=gen(10 * s + i), device="cuda").to(torch.bfloat16) for i in range(2)]
              for s in range(2)]
    want = [layer(ops, *t, p)[0] for t in inputs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(ops, *inputs[i], p)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(bits(y), bits(want[i])) for y in got[i])


def test_python_kernels_agree(ops):  # noqa: F811
    from bf16_skinny_gemm_amd import torch_op

    for kind in KINDS:
        p = parameters(kind)
        x = torch.randn(2, 3, 256, generator=gen(1), device="cuda").to(torch.bfloat16)
        logits = torch.randn(2, 3, 32, generator=gen(2), device="cuda")
        a, b = ops.route(logits, 5), torch_op._PY_KERNELS_MORE["route"](logits, 5)
        assert all(torch.equal(bits(u), bits(v)) and u.shape == (2, 3, 5) for u, v in zip(a, b))
        args = (x, *a, *p["w"], *p["s"], x, "gelu")
        y, z = ops.experts(*args), torch_op._PY_KERNELS_MORE["experts"](*args)
        assert y.shape == z.shape == x.shape and torch.equal(bits(y), bits(z))
    empty = ops.experts(x[:0], a[0][:0], a[1][:0], *p["w"], *p["s"])
    assert empty.shape == (0, 3, 256)


def test_refusals(skg, ops):  # noqa: F811
    p = parameters("int8")
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    ids, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    g, u, d = p["w"]
    s = p["s"]
    ops.experts(x, ids, w, g, u, d, *s)
    for args in ((x.float(), ids, w, g, u, d, *s), (x, ids.long(), w, g, u, d, *s), (x, ids, w.double(), g, u, d, *s),
                 (x, ids[:3], w[:3], g, u, d, *s), (x, ids, w[:, :1], g, u, d, *s), (x, ids, w, g[:, :64], u, d, *s),
                 (x, ids, w, g, u, d), (x, ids, w, g, u, d, s[0], s[1], None), (x, ids, w, g, u, u, *s),
                 (x, ids, w, g.float(), u, d, *s), (x, ids, w, g, u.to(torch.bfloat16), d, *s),
                 (x, ids, w, g, u, d, s[0][:, :5], s[1], s[2]), (x, ids, w, g.transpose(1, 2), u, d, *s),
                 (x, ids, w, g, torch.cat([u, u], dim=1)[:, :128], d, *s), (x, ids, w, g, u, d, *s, x[:2]),
                 (x, ids[:, :0], w[:, :0], g, u, d, *s), (x, ids, w, g, u, d, *s, None, "tanh"),
                 (x, ids.repeat(1, 17), w.repeat(1, 17), g, u, d, *s), (x.cpu(), ids, w, g, u, d, *s)):
        with pytest.raises((ValueError, NotImplementedError)):
            ops.experts(*args)
    with pytest.raises(ValueError):  # scales that belong to no bfloat16 weight
        ops.experts(x, ids, w, *(t.to(torch.bfloat16) for t in (g, u, d)), *s)
    need = skg.skinny_experts_workspace_bytes(4, 2, 32, 128)
    with pytest.raises(skg.SkinnyError):
        skg.experts(x, ids, w, g, u, d, *s, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    logits = torch.zeros(4, 32, device="cuda")
    for args in ((logits.double(), 4), (logits, 0), (logits, 33), (logits, 4, "tanh"), (logits, 4, "softmax", logits[0, :5]),
                 (logits, 4, "softmax", None, 5), (logits, 4, "softmax", None, 8, 9), (logits, 5, "softmax", None, 8, 1),
                 (logits, 4, "softmax", None, 8, 0), (torch.zeros(1, 1025, device="cuda"), 4), (logits.cpu(), 4),
                 (logits, 4, "softmax", None, 1, 1, True, float("inf"))):
        with pytest.raises((ValueError, NotImplementedError)):
            ops.route(*args)

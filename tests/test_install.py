"""What install() leaves as it was: classes with a forward of their own, and calls that ask
for derivatives. On the CPU every product takes the standard path, so the results of a hooked
module are those of the module before, and the routing is seen by its calls."""
from __future__ import annotations

import copy

import pytest
import torch


@pytest.fixture(scope="module")
def op():
    from bf16_skinny_gemm_amd import torch_op

    return torch_op


class Doubled(torch.nn.Linear):
    def forward(self, x):
        return 2 * super().forward(x)


class Adapted(torch.nn.Linear):
    """A low-rank update beside the product, and an argument that nn.Linear does not have."""

    def __init__(self, *args, **kwargs):
        super().__init__(*args, **kwargs)
        self.down = torch.nn.Parameter(torch.randn(4, self.in_features))
        self.up = torch.nn.Parameter(torch.randn(self.out_features, 4))

    def forward(self, x, *, update=True):
        y = torch.nn.functional.linear(x, self.weight, self.bias)
        return y + (x @ self.down.t()) @ self.up.t() if update else y


class Masked(torch.nn.Linear):
    """A product with another matrix than the weight."""

    def forward(self, x):
        return torch.nn.functional.linear(x, self.weight.tril(), self.bias)


class Renamed(torch.nn.Linear):
    """No forward of its own."""


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("cls", [Doubled, Adapted, Masked, Renamed])
def test_a_linear_class_keeps_its_own_forward(op, cls, bias, fused):
    torch.manual_seed(0)
    layer = cls(24, 16, bias=bias)
    x = torch.randn(3, 24)
    want = layer(x)
    model = torch.nn.Sequential(layer)
    assert op.install(model, fused=fused) == 1 and op.install(model, fused=fused) == 0
    assert torch.equal(layer(x), want)
    assert torch.equal(copy.deepcopy(model)(x), want)
    if cls is Adapted:
        assert torch.equal(layer(x, update=False), torch.nn.functional.linear(x, layer.weight, layer.bias))
    layer(x).sum().backward()
    assert layer.weight.grad is not None


@pytest.mark.parametrize("cls,calls", [(Doubled, 1), (Adapted, 1), (Masked, 0), (Renamed, 1)])
def test_the_product_by_the_weight_is_routed(op, monkeypatch, cls, calls):
    seen = []
    plain = op.skinny_linear

    def routed(x, weight, bias=None, fallback=True):
        seen.append((weight, fallback))
        return plain(x, weight, bias, fallback)

    monkeypatch.setattr(op, "skinny_linear", routed)
    layer = cls(8, 8, bias=False)
    op.install(torch.nn.Sequential(layer), fallback=True)
    layer(torch.randn(2, 8))
    assert len(seen) == calls and all(w is layer.weight and f for w, f in seen)
    torch.nn.functional.linear(torch.randn(2, 8), layer.weight)  # outside of the layer
    assert len(seen) == calls


def test_own_forward_without_fallback_refuses_what_does_not_qualify(op):
    layer = Doubled(8, 8, bias=False)
    op.install(torch.nn.Sequential(layer), fallback=False)
    with pytest.raises(ValueError):
        layer(torch.randn(2, 8))


def test_own_forward_compiles(op):
    torch.manual_seed(0)
    model = torch.nn.Sequential(Doubled(8, 8, bias=False), torch.nn.Linear(8, 8))
    x = torch.randn(2, 8)
    want = model(x)
    op.install(model)
    with torch.no_grad():
        assert torch.equal(torch.compile(model, backend="aot_eager")(x), want)


@pytest.mark.gpu
def test_own_forward_on_the_kernels(op):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.manual_seed(0)
    layer = Doubled(256, 128, bias=False).cuda().to(torch.bfloat16)
    many, few = (torch.randn(m, 256, device="cuda").to(torch.bfloat16) for m in (20, 4))
    want = layer(many)
    assert op.install(torch.nn.Sequential(layer), fused=True) == 1
    with torch.no_grad():
        assert torch.equal(layer(many), want)
        assert torch.equal(layer(few), 2 * op.linear(few, layer.weight))


def derivatives(model, x, t):
    """The model's directional derivative, three ways."""
    import torch.autograd.forward_ad as fw

    with fw.dual_level():
        got = [fw.unpack_dual(model(fw.make_dual(x, t))).tangent]
    got.append(torch.func.jvp(model, (x,), (t,))[1])
    params = {k: v.detach() for k, v in model.named_parameters()}
    along = {k: torch.ones_like(v) for k, v in params.items()}
    got.append(torch.func.jvp(lambda p: torch.func.functional_call(model, p, (x,)), (params,), (along,))[1])
    return got


def test_derivatives_do_not_reach_the_operators(op, monkeypatch):
    """With every call taken for one that qualifies, those with a tangent or inside a transform
    still run on the standard path (the operator itself refuses CPU tensors)."""
    import torch.autograd.forward_ad as fw

    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.Linear(8, 8, bias=False), torch.nn.Tanh())
    x, t = torch.randn(2, 8), torch.randn(2, 8)
    want = derivatives(model, x, t)
    each = torch.vmap(model)(x)
    op.install(model)
    monkeypatch.setattr(op, "qualifies", lambda *args: True)
    with pytest.raises(ValueError, match="skinny::linear"):
        model(x)
    for a, b in zip(derivatives(model, x, t), want):
        assert torch.equal(a, b)
    assert torch.equal(torch.vmap(model)(x), each)
    model[0].forward.keywords["fallback"] = False
    with pytest.raises(ValueError, match="qualify"):
        torch.func.jvp(model, (x,), (t,))
    # the condition of the operators that fused takes
    seen = []
    torch.func.jvp(lambda a: (seen.append(op._inference(a, None)), a)[1], (x,), (t,))
    with fw.dual_level(), torch.no_grad():
        seen += [op._inference(None, fw.make_dual(x, t)), op._inference(x, None)]
    assert seen == [False, False, True] and op._inference(x)


@pytest.mark.gpu
def test_derivatives_through_a_fused_model(op):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.manual_seed(0)
    # apart: torch's own norm gives float32 under a tangent, which the next layer refuses
    models = [torch.nn.Sequential(m).cuda().to(torch.bfloat16).requires_grad_(False)
              for m in (torch.nn.RMSNorm(64), torch.nn.Linear(64, 32), torch.nn.Linear(64, 16, bias=False))]
    x, t = (torch.randn(4, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    for model in models:
        want = derivatives(model, x, t)
        assert all(bool(w.any()) for w in want)
        assert op.install(model, fused=True) == 1
        for a, b in zip(derivatives(model, x, t), want):
            assert torch.equal(a, b)
    (norm,), (lin,), (bare,) = models
    assert torch.equal(norm(x), op.rms_norm(x, norm.weight, torch.finfo(torch.float32).eps))
    assert torch.equal(lin(x), op.linear_act(x, lin.weight, lin.bias))
    assert torch.equal(bare(x), op.linear(x, bare.weight))


@pytest.mark.gpu
def test_a_fused_model_compiles(op):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.RMSNorm(64), torch.nn.Linear(64, 32), Doubled(32, 16, bias=False))
    model = model.cuda().to(torch.bfloat16)
    x = torch.randn(4, 64, device="cuda").to(torch.bfloat16)
    op.install(model, fused=True)
    with torch.no_grad():
        want = model(x)
        assert torch.equal(torch.compile(model, backend="aot_eager", fullgraph=True)(x), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_fused_under_autocast(op, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.RMSNorm(64), torch.nn.Linear(64, 32)).cuda().to(torch.bfloat16)
    x = torch.randn(4, 64, device="cuda").to(torch.bfloat16)
    with torch.no_grad(), torch.autocast("cuda", dtype=dtype):
        norm, want = model[0](x), model(x)
        op.install(model, fused=True)
        assert model[0](x).dtype == norm.dtype and model(x).dtype == want.dtype == dtype
        y = model[0](x)
        if dtype == torch.bfloat16:
            assert torch.equal(model[1](y), op.linear_act(y, model[1].weight, model[1].bias))
        else:
            assert torch.equal(model[1](y), torch.nn.functional.linear(y, model[1].weight, model[1].bias))


def test_fused_takes_layers_whose_rows_are_whole_pieces(op, monkeypatch):
    """Rows that do not start at multiples of 16 bytes would run element-wise."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    monkeypatch.setattr(op, "_device_is_gfx950", lambda device: True)
    with FakeTensorMode():
        def make(*shape):
            return torch.empty(*shape, dtype=torch.bfloat16, device="cuda")

        def takes(x, w):
            return op.qualifies_fused(x, w, make(w.shape[0]))

        w = make(32, 64)
        for x in (make(4, 64), make(64), make(2, 3, 64), make(2, 3, 64).transpose(0, 1), make(4, 72)[:, :64],
                  make(4, 80)[:, 8:72], make(64, 4).t(), make(5, 64)[1:]):
            assert takes(x, w)
        for x in (make(4, 65)[:, :64], make(4, 72)[:, 4:68], make(4 * 64 + 1)[1:].view(4, 64),
                  make(6 * 64 + 4)[4:].view(2, 3, 64), make(65, 64)):
            assert not takes(x, w)
        assert not takes(make(4, 60), make(32, 60)) and not takes(make(4, 1001), make(32, 1001))
        assert not takes(make(4, 64), make(32 * 64 + 1)[1:].view(32, 64))


@pytest.mark.gpu
def test_fused_leaves_odd_widths_to_the_standard_path(op):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    layer = torch.nn.Linear(1001, 64).cuda().to(torch.bfloat16)
    x = torch.randn(4, 1001, device="cuda").to(torch.bfloat16)
    with torch.no_grad():
        want = layer(x)
        op.install(torch.nn.Sequential(layer), fused=True)
        assert torch.equal(layer(x), want)
        y = layer(torch.randn(4, 1008, device="cuda").to(torch.bfloat16)[:, :1001])
        assert y.shape == (4, 64)


class Packed(torch.nn.Linear):
    """Its weight in another form, as quantised layers keep it."""

    def __init__(self, *args, **kwargs):
        super().__init__(*args, **kwargs)
        self.packed = torch.nn.Parameter(self.weight.detach() * 3)
        del self.weight

    def forward(self, x):
        return torch.nn.functional.linear(x, self.packed / 3, self.bias)


def test_a_linear_class_without_a_weight(op):
    torch.manual_seed(0)
    layer, x = Packed(8, 4), torch.randn(2, 8)
    want = layer(x)
    op.install(torch.nn.Sequential(layer))
    assert torch.equal(layer(x), want)


@pytest.mark.parametrize("call", [lambda f, x, s: f(x, s.weight) + s.bias, lambda f, x, s: f(x, s.weight, bias=s.bias),
                                  lambda f, x, s: f(x, s.weight, None) + s.bias])
def test_every_form_of_the_product_is_routed(op, monkeypatch, call):
    class Own(torch.nn.Linear):
        def forward(self, x):
            return call(torch.nn.functional.linear, x, self)

    torch.manual_seed(0)
    layer, x = Own(8, 4), torch.randn(2, 8)
    want, seen, plain = layer(x), [], op.skinny_linear
    op.install(torch.nn.Sequential(layer))
    monkeypatch.setattr(op, "skinny_linear", lambda *a, **k: (seen.append(a), plain(*a, **k))[1])
    assert torch.equal(layer(x), want) and len(seen) == 1

"""PyTorch operator and module hook for the skinny GEMM.

The routing follows the plan-table hook of vLLM PR #62949 (SM121 skinny GEMM
plans, sections Claims and Details) and vLLM PR #65306 (SM90 skinny GEMM plans,
section Details): a linear layer's apply path takes the skinny GEMM when the GPU
architecture, the dtype and the token count qualify, and keeps the standard
linear path otherwise. Here:

* ``torch.ops.skinny.linear(x, weight)`` is a custom operator (graph-capturable,
  with a fake implementation for tracing) that always runs the HIP kernel and
  raises if the call does not qualify. Its GPU and CPU implementations are
  registered in C++ (``libskinny_torch_op.so``, built from csrc/torch_op.cpp), so
  an eager call goes from the dispatcher to the C ABI with no Python frame; when
  that library has not been built, the same operator is registered from Python
  below (it calls the same C entry point through ctypes, at a few µs more per
  eager call);
* :func:`skinny_linear` routes: qualifying calls go to the op, others to
  ``torch.nn.functional.linear`` only when ``fallback=True`` (the default for the
  module hook), else they raise;
* :func:`install` swaps the forward of ``nn.Linear`` modules for the routed one;
* ``rms_norm``, ``add_rms_norm``, ``rms_norm_fp8``, ``add_rms_norm_fp8``, ``linear_act``,
  ``linear_gated``, ``linear_fp8`` and ``linear_gated_fp8`` (``torch.ops.skinny.*``, same
  registration) are the operators around the projection, for any number of rows;
  :func:`install` with ``fused=True`` routes biased ``nn.Linear`` layers and
  ``nn.RMSNorm`` modules to them.

A call qualifies when x and weight are bfloat16 CUDA tensors on a gfx950 device,
weight is [N, K] contiguous, x is [..., K] with 1 <= prod(leading dims) <= 8
(the token count M: the cited pages route 1..4; 5..8 is routed here too, since on
MI355X the kernels measured faster than F.linear there on the decode shapes), and
there is no bias. The kernel itself never falls back: a missing library or a
refused launch raises.
"""
from __future__ import annotations

import functools
import math
import os

import torch
from torch.autograd import forward_ad
from torch.overrides import TorchFunctionMode

from . import _on_device, _stream_handle, lib, skinny_gemm_bf16
from . import linear as _linear_call
from . import rms_norm as _norm_call
from .build import TORCH_OP_PATH

_ARCH_OK: dict[int, bool] = {}


def _device_is_gfx950(device: torch.device) -> bool:
    idx = device.index if device.index is not None else torch.cuda.current_device()
    if idx not in _ARCH_OK:
        props = torch.cuda.get_device_properties(idx)
        _ARCH_OK[idx] = str(getattr(props, "gcnArchName", "")).startswith("gfx950")
    return _ARCH_OK[idx]


def qualifies(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None) -> bool:
    """True when (x, weight, bias) can run on the skinny GEMM."""
    if bias is not None:
        return False
    if x.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        return False
    if x.device.type != "cuda" or weight.device != x.device:
        return False
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        return False
    if not weight.is_contiguous():
        # a strided weight would have to be copied whole on every call (634 MB for
        # the LM head): leave it to the standard path
        return False
    m = 1
    for d in x.shape[:-1]:
        m *= d
    if not (1 <= m <= 8):
        return False
    return _device_is_gfx950(x.device)


def _linear_gpu(x: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    """y = x @ weight.T on the HIP skinny GEMM; x [..., K] with M = prod(...) <= 8."""
    if not qualifies(x, weight):
        raise ValueError("skinny::linear: inputs do not qualify (bf16 on gfx950, no bias, "
                         f"M in 1..8): x {tuple(x.shape)} {x.dtype}, weight "
                         f"{tuple(weight.shape)} {weight.dtype}")
    K = x.shape[-1]
    N = weight.shape[0]
    x2 = x.reshape(-1, K)
    if not x2.is_contiguous():
        x2 = x2.contiguous()
    y = torch.empty((*x.shape[:-1], N), dtype=torch.bfloat16, device=x.device)
    # qualifies() has checked dtypes, devices and shapes: call the C entry point
    # directly (it raises if the library is missing or refuses the call)
    with _on_device(x.device):
        skinny_gemm_bf16(x2.data_ptr(), weight.data_ptr(), y.data_ptr(), x2.shape[0], N, K,
                         _stream_handle(x.device))
    return y


def _linear_other(x: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    raise ValueError("skinny::linear: runs on gfx950 GPU tensors only, got "
                     f"x on {x.device}, weight on {weight.device}")


def _linear_fake(x: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    return x.new_empty((*x.shape[:-1], weight.shape[0]))


if os.path.exists(TORCH_OP_PATH):
    # the C++ registration: schema and the CUDA / CPU kernels; the GEMM library it
    # links is the one the ctypes binding loads (same file, one copy in the process)
    lib()
    torch.ops.load_library(TORCH_OP_PATH)
    _LIB = torch.library.Library("skinny", "FRAGMENT")
    CPP_OP = True
else:
    # The Python registration goes through torch.library.Library rather than the
    # torch.library.custom_op decorator: the decorator's Python wrapping costs about
    # 10 us per eager call on its own, the plain registration about 3 us.
    _LIB = torch.library.Library("skinny", "DEF")
    _LIB.define("linear(Tensor x, Tensor weight) -> Tensor")
    _LIB.impl("linear", _linear_gpu, "CUDA")
    _LIB.impl("linear", _linear_other, "CPU")
    CPP_OP = False
torch.library.register_fake("skinny::linear", _linear_fake, lib=_LIB)
linear = torch.ops.skinny.linear


# ---- the operators around the projection ------------------------------------

_SCHEMAS = (
    "rms_norm(Tensor x, Tensor weight, float eps) -> Tensor",
    "add_rms_norm(Tensor x, Tensor residual, Tensor weight, float eps) -> (Tensor, Tensor)",
    "rms_norm_fp8(Tensor x, Tensor weight, float eps, int group) -> (Tensor, Tensor)",
    "add_rms_norm_fp8(Tensor x, Tensor residual, Tensor weight, float eps, int group) "
    "-> (Tensor, Tensor, Tensor)",
    "linear_act(Tensor x, Tensor weight, Tensor? bias=None, Tensor? residual=None, "
    "str act='none', bool out_f32=False) -> Tensor",
    "linear_gated(Tensor x, Tensor w_gate, Tensor w_up, Tensor? b_gate=None, Tensor? b_up=None, "
    "str act='silu', bool out_f32=False) -> Tensor",
    "linear_fp8(Tensor x, Tensor x_scale, Tensor weight, Tensor w_scale, Tensor? bias=None, "
    "Tensor? residual=None, str act='none', bool out_f32=False) -> Tensor",
    "linear_gated_fp8(Tensor x, Tensor x_scale, Tensor w_gate, Tensor gate_scale, Tensor w_up, "
    "Tensor up_scale, Tensor? b_gate=None, Tensor? b_up=None, str act='silu', "
    "bool out_f32=False) -> Tensor",
)


def _quant(group: int) -> str:
    if group not in (0, 128):
        raise ValueError(f"group must be 0 (per row) or 128, got {group}")
    return "group" if group else "row"


def _scale_shape(x: torch.Tensor, group: int) -> tuple:
    return (*x.shape[:-1], -(-x.shape[-1] // 128)) if group else tuple(x.shape[:-1])


def _norm_py(x, weight, eps, residual=None, quant=None):
    """Python kernels of the norms (used when the C++ operators are not built)."""
    D = x.shape[-1]
    got = _norm_call(x.reshape(-1, D), weight, eps,
                     residual=None if residual is None else residual.reshape(-1, D), quant=quant)
    got = got if isinstance(got, tuple) else (got,)
    shapes = [x.shape] + ([_scale_shape(x, quant == "group")] if quant else []) + [x.shape]
    got = tuple(g.reshape(s) for g, s in zip(got, shapes))
    return got[0] if len(got) == 1 else got


def _linear_py(x, weight, bias, residual, act, out_f32, W_up=None, bias_up=None, x_scale=None,
               w_scale=None, w_up_scale=None):
    """Python kernels of the projections (used when the C++ operators are not built)."""
    K, N, M = x.shape[-1], weight.shape[0], math.prod(x.shape[:-1])
    if x_scale is not None:
        x_scale = x_scale.reshape(M) if w_scale.dim() == 1 else x_scale.reshape(M, x_scale.shape[-1])
    y = _linear_call(x.reshape(M, K), weight, bias=bias, act=act, W_up=W_up, bias_up=bias_up,
                     residual=None if residual is None else residual.reshape(M, N),
                     x_scale=x_scale, w_scale=w_scale, w_up_scale=w_up_scale,
                     out_dtype=torch.float32 if out_f32 else torch.bfloat16)
    return y.reshape(*x.shape[:-1], N)


_PY_KERNELS = {
    "rms_norm": lambda x, w, eps: _norm_py(x, w, eps),
    "add_rms_norm": lambda x, r, w, eps: _norm_py(x, w, eps, r),
    "rms_norm_fp8": lambda x, w, eps, group: _norm_py(x, w, eps, None, _quant(group)),
    "add_rms_norm_fp8": lambda x, r, w, eps, group: _norm_py(x, w, eps, r, _quant(group)),
    "linear_act": lambda x, w, b=None, r=None, act="none", f32=False: _linear_py(x, w, b, r, act, f32),
    "linear_gated": lambda x, w, u, b=None, bu=None, act="silu", f32=False: _linear_py(
        x, w, b, None, act, f32, u, bu),
    "linear_fp8": lambda x, xs, w, ws, b=None, r=None, act="none", f32=False: _linear_py(
        x, w, b, r, act, f32, x_scale=xs, w_scale=ws),
    "linear_gated_fp8": lambda x, xs, w, ws, u, us, b=None, bu=None, act="silu", f32=False: _linear_py(
        x, w, b, None, act, f32, u, bu, xs, ws, us),
}


def _refuse_cpu(name):
    def refuse(*args, **kwargs):
        raise ValueError(f"skinny::{name}: runs on gfx950 GPU tensors only")
    return refuse


def _y_fake(x, n, f32):
    return x.new_empty((*x.shape[:-1], n), dtype=torch.float32 if f32 else torch.bfloat16)


def _q_fake(x, group):
    _quant(group)
    return (x.new_empty(x.shape, dtype=torch.float8_e4m3fn),
            x.new_empty(_scale_shape(x, group), dtype=torch.float32))


_FAKES = {
    "rms_norm": lambda x, weight, eps: x.new_empty(x.shape),
    "add_rms_norm": lambda x, residual, weight, eps: (x.new_empty(x.shape), x.new_empty(x.shape)),
    "rms_norm_fp8": lambda x, weight, eps, group: _q_fake(x, group),
    "add_rms_norm_fp8": lambda x, residual, weight, eps, group: (*_q_fake(x, group), x.new_empty(x.shape)),
    "linear_act": lambda x, weight, bias=None, residual=None, act="none", out_f32=False: _y_fake(
        x, weight.shape[0], out_f32),
    "linear_gated": lambda x, w_gate, w_up, b_gate=None, b_up=None, act="silu", out_f32=False: _y_fake(
        x, w_gate.shape[0], out_f32),
    "linear_fp8": lambda x, x_scale, weight, w_scale, bias=None, residual=None, act="none",
    out_f32=False: _y_fake(x, weight.shape[0], out_f32),
    "linear_gated_fp8": lambda x, x_scale, w_gate, gate_scale, w_up, up_scale, b_gate=None, b_up=None,
    act="silu", out_f32=False: _y_fake(x, w_gate.shape[0], out_f32),
}

for _schema in _SCHEMAS:
    _name = _schema.split("(")[0]
    if not CPP_OP:
        _LIB.define(_schema)
        _LIB.impl(_name, _PY_KERNELS[_name], "CUDA")
        _LIB.impl(_name, _refuse_cpu(_name), "CPU")
    torch.library.register_fake("skinny::" + _name, _FAKES[_name], lib=_LIB)
rms_norm = torch.ops.skinny.rms_norm.default
add_rms_norm = torch.ops.skinny.add_rms_norm.default
rms_norm_fp8 = torch.ops.skinny.rms_norm_fp8.default
add_rms_norm_fp8 = torch.ops.skinny.add_rms_norm_fp8.default
linear_act = torch.ops.skinny.linear_act.default
linear_gated = torch.ops.skinny.linear_gated.default
linear_fp8 = torch.ops.skinny.linear_fp8.default
linear_gated_fp8 = torch.ops.skinny.linear_gated_fp8.default


_func_level = torch._C._functorch.maybe_current_level


def _transformed(*tensors) -> bool:
    """A torch.func transform is at work, or a tensor carries a forward-mode tangent: the
    operators have rules for neither and would drop the derivative."""
    if _func_level() is not None:
        return True
    return forward_ad._current_level >= 0 and any(
        t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def skinny_linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                  fallback: bool = True) -> torch.Tensor:
    """F.linear semantics, routed: the skinny GEMM when the call qualifies,
    otherwise torch.nn.functional.linear if ``fallback`` (else ValueError). Calls inside a
    torch.func transform or with forward-mode tangents do not qualify."""
    if qualifies(x, weight, bias) and not _transformed(x, weight):
        return torch.ops.skinny.linear(x, weight)
    if not fallback:
        raise ValueError("skinny_linear: call does not qualify for the skinny GEMM")
    return torch.nn.functional.linear(x, weight, bias)


# Rows up to which a biased layer is routed: there linear_act reads each weight once, and
# the standard path is a library product that serves larger batches well (64 x 4096 x 4096
# 10.3 us against 13.5, 64 x 1024 x 4096 6.5 against 12.6, 64 x 12576 x 4096 28.7 against 26.1).
FUSED_ROWS = 64


def _inference(*tensors) -> bool:
    """No derivative is asked for: the operators record none."""
    return not (torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)) and (
        not _transformed(*tensors))


def _offset(t: torch.Tensor) -> int:
    # a tracer has no answer; views that start inside a piece are rare there
    return 0 if torch.compiler.is_compiling() else t.storage_offset()


def _pieces(x: torch.Tensor, weight: torch.Tensor) -> bool:
    """Rows of x and of the weight start at multiples of 16 bytes, as the fast kernels read
    them; other rows run element-wise, where the standard path is ahead: a layer of 4100 to
    4096 features 154 us against 19 for one row, 218 against 21 for 64."""
    if weight.shape[1] % 8 or _offset(weight) % 8:
        return False
    if x.dim() == 2 and x.stride(1) == 1:
        return _offset(x) % 8 == 0 and x.stride(0) % 8 == 0
    return not x.is_contiguous() or _offset(x) % 8 == 0  # others are copied


def qualifies_fused(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None) -> bool:
    """True when a layer with (weight, bias) should run on linear_act."""
    if x.dtype != torch.bfloat16 or x.device.type != "cuda" or x.dim() < 1 or x.numel() == 0:
        return False
    for t in (weight, bias):
        if t is not None and (t.dtype != torch.bfloat16 or t.device != x.device or not t.is_contiguous()):
            return False
    if x.shape[-1] != weight.shape[1] or x.numel() // x.shape[-1] > FUSED_ROWS:
        return False
    if not _pieces(x, weight):
        return False
    if torch.is_autocast_enabled("cuda") and torch.get_autocast_dtype("cuda") != torch.bfloat16:
        return False  # F.linear would compute in, and return, that type
    return _inference(x, weight, bias) and _device_is_gfx950(x.device)


def _norm_forward(self, x):
    """nn.RMSNorm.forward on the HIP norm where it qualifies."""
    w = self.weight
    if (w is not None and w.dim() == 1 and x.dim() >= 1 and x.shape[-1] == w.shape[0] and x.numel() > 0
            and x.dtype == w.dtype == torch.bfloat16 and x.device.type == "cuda" and w.device == x.device
            and w.is_contiguous() and _inference(x, w) and _device_is_gfx950(x.device)):
        # without an eps the module adds float32's, for bfloat16 inputs too
        eps = self.eps if self.eps is not None else torch.finfo(torch.float32).eps
        return rms_norm(x, w, eps)
    return type(self).forward(self, x)


class _RoutedProduct(TorchFunctionMode):
    """Within it, F.linear on the given weight, as nn.Linear.forward calls it, is routed."""

    def __init__(self, weight, fallback):
        super().__init__()
        self.weight, self.fallback = weight, fallback

    def __torch_function__(self, func, types, args=(), kwargs=None):
        kwargs = kwargs or {}
        if func is torch.nn.functional.linear and len(args) >= 2 and args[1] is self.weight:
            return skinny_linear(*args, **kwargs, fallback=self.fallback)
        return func(*args, **kwargs)


def _linear_forward(self, inp, fallback):
    """nn.Linear.forward, routed."""
    if getattr(self, "_skinny_fused", False) and self.bias is not None and qualifies_fused(inp, self.weight, self.bias):
        return linear_act(inp, self.weight, self.bias, None, "none", False)
    return skinny_linear(inp, self.weight, self.bias, fallback=fallback)


def _own_linear_forward(self, *args, _skinny_fallback, **kwargs):
    """The forward of a class derived from nn.Linear, with its weight's product routed."""
    with _RoutedProduct(getattr(self, "weight", None), _skinny_fallback):
        return type(self).forward(self, *args, **kwargs)


def install(module: torch.nn.Module, fallback: bool = True, fused: bool = False) -> int:
    """Route the forward of every nn.Linear inside ``module`` through
    :func:`skinny_linear`. A class derived from it that has a forward of its own keeps that:
    what it does with the product stays, and the product by its weight is routed where it
    calls nn.Linear's forward or F.linear for it. With ``fused``, nn.Linear layers with a
    bias and up to 64 rows of input run on linear_act and nn.RMSNorm modules on rms_norm,
    both where no derivative is asked for; classes with a forward of their own do not, and
    layers that an earlier call hooked without ``fused`` take it up. Returns the number of
    modules hooked."""
    count = 0
    for sub in module.modules():
        if fused and type(sub).forward is torch.nn.Linear.forward:
            sub._skinny_fused = True
        if getattr(sub, "_skinny_hooked", False):
            continue
        if type(sub).forward is torch.nn.Linear.forward:
            sub.forward = functools.partial(_linear_forward, sub, fallback=fallback)
        elif isinstance(sub, torch.nn.Linear):
            sub.forward = functools.partial(_own_linear_forward, sub, _skinny_fallback=fallback)
        elif fused and type(sub).forward is torch.nn.RMSNorm.forward:
            sub.forward = functools.partial(_norm_forward, sub)
        else:
            continue
        sub._skinny_hooked = True
        count += 1
    return count


__all__ = ["linear", "skinny_linear", "install", "qualifies", "qualifies_fused", "CPP_OP", "FUSED_ROWS",
           "rms_norm", "add_rms_norm", "rms_norm_fp8", "add_rms_norm_fp8", "linear_act", "linear_gated",
           "linear_fp8", "linear_gated_fp8"]

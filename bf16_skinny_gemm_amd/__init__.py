"""BF16 skinny GEMM for MI355X (gfx950): y[M,N] = x[M,K] . W[N,K]^T for M = 1..8.

Thin Python binding over the C ABI of ``libskinny_gemm_bf16.so``
(``include/skinny_gemm.h``). Every step of the computation runs in the HIP
kernels; this module only marshals arguments. PyTorch provides device memory
and the current stream. There is no fallback: if the library is missing, or the
device is not gfx950, calls raise.

Raw entry points (same names and arguments as the C functions; pointers as
Python ints; a non-zero status raises :class:`SkinnyError`):
    skinny_gemm_init, skinny_gemm_bf16, skinny_gemm_bf16_pair,
    skinny_gemm_bf16_ex, skinny_gemm_bf16_pair_ex, skinny_gemm_bf16_pair_strided,
    skinny_gemm_bf16_pair_strided_ex, skinny_gemm_bf16_f32out,
    skinny_gemm_bf16_f32out_ex, skinny_gemm_get_plan,
    skinny_gemm_num_variants, skinny_gemm_get_variant,
    skinny_gemm_status_string, skinny_gemm_version,
    skinny_gemm_split_k_workspace_bytes, skinny_gemm_bf16_split_k,
    skinny_gemm_bf16_split_k_noalloc, skinny_gemm_split_k_num_variants,
    skinny_gemm_split_k_get_variant, skinny_gemm_split_k_default_plan,
    skinny_rms_norm_bf16, skinny_rms_norm_fp8, skinny_linear_bf16, skinny_linear_fp8,
    skinny_linear_default_plan, skinny_rms_norm_int8, skinny_quantize_int8, skinny_linear_int8,
    skinny_linear_int8_default_plan, skinny_route, skinny_experts_workspace_bytes, skinny_experts

Tensor helpers: :func:`gemm`, :func:`gemm_pair`, :func:`gemm_pair_strided`,
:func:`split_k_workspace`, :func:`gemm_split_k` and :func:`gemm_split_k_noalloc`;
:func:`rms_norm`, :func:`quantize_int8` and :func:`linear` (any number of rows,
``include/skinny_ops.h``); :func:`route` and :func:`experts` (``include/skinny_moe.h``).
"""
from __future__ import annotations

import ctypes
import os
import threading

# torch first: its HIP runtime (soname libamdhip64.so.7) must be the one the
# library binds to, so that torch's stream handles are valid in it.
import torch

from .build import LIB_PATH

SKINNY_OK = 0
SKINNY_ERR_INVALID_ARG = -1
SKINNY_ERR_UNSUPPORTED = -2
SKINNY_ERR_NOT_INITIALIZED = -3
SKINNY_ERR_LAUNCH = -4

SKINNY_KIND_FIXED_K = 1
SKINNY_KIND_LOOP_K = 2
SKINNY_KIND_SCALAR = 3
SKINNY_KIND_MFMA = 4
SKINNY_KIND_SPLIT_K = 5

SKINNY_ACT_NONE = 0
SKINNY_ACT_RELU = 1
SKINNY_ACT_GELU = 2
SKINNY_ACT_GELU_TANH = 3
SKINNY_ACT_SILU = 4

SKINNY_SCALES_ROW = 1
SKINNY_SCALES_BLOCK = 2

SKINNY_LINEAR_ELEMENTS = 0
SKINNY_LINEAR_STREAM = 1
SKINNY_LINEAR_TILE = 2

SKINNY_SCORE_SOFTMAX = 0
SKINNY_SCORE_SIGMOID = 1

SKINNY_WEIGHTS_BF16 = 0
SKINNY_WEIGHTS_E4M3_ROW = 1
SKINNY_WEIGHTS_E4M3_BLOCK = 2
SKINNY_WEIGHTS_INT8_ROW = 3

SCORES = {"softmax": SKINNY_SCORE_SOFTMAX, "sigmoid": SKINNY_SCORE_SIGMOID}
ACTS = {"none": SKINNY_ACT_NONE, "relu": SKINNY_ACT_RELU, "gelu": SKINNY_ACT_GELU,
        "gelu_tanh": SKINNY_ACT_GELU_TANH, "silu": SKINNY_ACT_SILU}


class SkinnyError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_status_string(status)} (status {status})")


class Plan(ctypes.Structure):
    """skinny_plan_t."""

    _fields_ = [
        ("kind", ctypes.c_int32),
        ("threads_per_block", ctypes.c_int32),
        ("lanes_per_row", ctypes.c_int32),
        ("chunks", ctypes.c_int32),
        ("rows_per_wave", ctypes.c_int32),
        ("k_split", ctypes.c_int32),
        ("nontemporal", ctypes.c_int32),
        ("grid_blocks", ctypes.c_int32),
        ("x_in_lds", ctypes.c_int32),
        ("prefetch", ctypes.c_int32),
    ]

    def as_dict(self) -> dict:
        return {f: int(getattr(self, f)) for f, _ in self._fields_}

    @classmethod
    def from_dict(cls, d: dict) -> "Plan":
        return cls(**{f: int(d[f]) for f, _ in cls._fields_})

    def __repr__(self) -> str:
        return "Plan(" + ", ".join(f"{k}={v}" for k, v in self.as_dict().items()) + ")"


class NormArgs(ctypes.Structure):
    """skinny_norm_t."""

    _fields_ = [
        ("x", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("weight", ctypes.c_void_p),
        ("residual_out", ctypes.c_void_p), ("y", ctypes.c_void_p), ("scale", ctypes.c_void_p),
        ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64), ("ldro", ctypes.c_int64),
        ("ldy", ctypes.c_int64), ("M", ctypes.c_int32), ("D", ctypes.c_int32),
        ("group", ctypes.c_int32), ("eps", ctypes.c_float),
    ]


class LinearArgs(ctypes.Structure):
    """skinny_linear_t."""

    _fields_ = [
        ("x", ctypes.c_void_p), ("W0", ctypes.c_void_p), ("W1", ctypes.c_void_p),
        ("x_scale", ctypes.c_void_p), ("w0_scale", ctypes.c_void_p), ("w1_scale", ctypes.c_void_p),
        ("bias0", ctypes.c_void_p), ("bias1", ctypes.c_void_p), ("residual", ctypes.c_void_p),
        ("y", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64),
        ("ldy", ctypes.c_int64), ("M", ctypes.c_int32), ("N", ctypes.c_int32),
        ("K", ctypes.c_int32), ("act", ctypes.c_int32), ("out_f32", ctypes.c_int32),
        ("scales", ctypes.c_int32),
    ]


class LinearPlan(ctypes.Structure):
    """skinny_linear_plan_t."""

    _fields_ = [(name, ctypes.c_int32) for name in ("kind", "features", "rows", "waves", "ring", "index", "count")]

    def as_dict(self) -> dict:
        return {f[0]: int(getattr(self, f[0])) for f in self._fields_}

    def __repr__(self):
        return "LinearPlan(" + ", ".join(f"{k}={v}" for k, v in self.as_dict().items()) + ")"


class RouteArgs(ctypes.Structure):
    """skinny_route_t."""

    _fields_ = [
        ("logits", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("ids", ctypes.c_void_p),
        ("weights", ctypes.c_void_p), ("ldl", ctypes.c_int64), ("M", ctypes.c_int32),
        ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("score", ctypes.c_int32),
        ("groups", ctypes.c_int32), ("kept", ctypes.c_int32), ("renormalize", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class ExpertsArgs(ctypes.Structure):
    """skinny_experts_t."""

    _fields_ = [(name, ctypes.c_void_p) for name in (
        "x", "ids", "weights", "w_gate", "w_up", "w_down", "gate_scale", "up_scale", "down_scale",
        "residual", "y", "workspace")] + [("workspace_bytes", ctypes.c_size_t)] + [
        (name, ctypes.c_int64) for name in ("ldx", "ldr", "ldy", "up_stride", "down_stride",
                                            "up_scale_stride", "down_scale_stride")] + [
        (name, ctypes.c_int32) for name in ("M", "E", "k", "H", "I", "act", "type")]


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load the in-tree HIP library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it first (python -m bf16_skinny_gemm_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        vp = ctypes.c_void_p
        i = ctypes.c_int
        pp = ctypes.POINTER(Plan)
        L.skinny_gemm_init.argtypes = [i]
        L.skinny_gemm_bf16.argtypes = [vp, vp, vp, i, i, i, vp]
        L.skinny_gemm_bf16_pair.argtypes = [vp, vp, vp, vp, vp, i, i, i, vp]
        L.skinny_gemm_bf16_ex.argtypes = [vp, vp, vp, i, i, i, pp, vp]
        L.skinny_gemm_bf16_pair_ex.argtypes = [vp, vp, vp, vp, vp, i, i, i, pp, vp]
        L.skinny_gemm_bf16_f32out.argtypes = [vp, vp, vp, i, i, i, vp]
        L.skinny_gemm_bf16_pair_strided.argtypes = [vp, vp, i, vp, vp, vp, vp, i, i, i, i, vp]
        L.skinny_gemm_bf16_pair_strided_ex.argtypes = [vp, vp, i, vp, vp, vp, vp, i, i, i, i, pp, vp]
        L.skinny_gemm_bf16_f32out_ex.argtypes = [vp, vp, vp, i, i, i, pp, vp]
        L.skinny_gemm_get_plan.argtypes = [i, i, i, pp]
        L.skinny_gemm_num_variants.argtypes = []
        L.skinny_gemm_get_variant.argtypes = [i, pp]
        L.skinny_gemm_status_string.argtypes = [i]
        L.skinny_gemm_status_string.restype = ctypes.c_char_p
        L.skinny_gemm_version.argtypes = []
        L.skinny_gemm_split_k_workspace_bytes.argtypes = [i, i, i, pp]
        L.skinny_gemm_split_k_workspace_bytes.restype = ctypes.c_size_t
        L.skinny_gemm_bf16_split_k.argtypes = [vp, vp, vp, i, i, i, pp, vp, ctypes.c_size_t, vp]
        L.skinny_gemm_bf16_split_k_noalloc.argtypes = [vp, vp, vp, i, i, i, pp, vp]
        L.skinny_gemm_split_k_num_variants.argtypes = []
        L.skinny_gemm_split_k_get_variant.argtypes = [i, pp]
        L.skinny_gemm_split_k_default_plan.argtypes = [i, i, i, pp]
        for name, args in (("skinny_rms_norm_bf16", NormArgs), ("skinny_rms_norm_fp8", NormArgs),
                           ("skinny_rms_norm_int8", NormArgs), ("skinny_quantize_int8", NormArgs),
                           ("skinny_linear_bf16", LinearArgs), ("skinny_linear_fp8", LinearArgs),
                           ("skinny_linear_int8", LinearArgs), ("skinny_route", RouteArgs),
                           ("skinny_experts", ExpertsArgs)):
            getattr(L, name).argtypes = [ctypes.POINTER(args), vp]
            getattr(L, name).restype = ctypes.c_int
        L.skinny_experts_workspace_bytes.argtypes = [ctypes.c_int32] * 4
        L.skinny_experts_workspace_bytes.restype = ctypes.c_size_t
        for name in ("skinny_linear_default_plan", "skinny_linear_int8_default_plan"):
            getattr(L, name).argtypes = [ctypes.POINTER(LinearArgs), ctypes.c_int32, ctypes.POINTER(LinearPlan)]
            getattr(L, name).restype = ctypes.c_int
        for name in ("skinny_gemm_init", "skinny_gemm_bf16", "skinny_gemm_bf16_pair",
                     "skinny_gemm_bf16_ex", "skinny_gemm_bf16_pair_ex", "skinny_gemm_bf16_f32out",
                     "skinny_gemm_bf16_f32out_ex", "skinny_gemm_bf16_pair_strided",
                     "skinny_gemm_bf16_pair_strided_ex", "skinny_gemm_get_plan",
                     "skinny_gemm_num_variants", "skinny_gemm_get_variant", "skinny_gemm_version",
                     "skinny_gemm_bf16_split_k", "skinny_gemm_bf16_split_k_noalloc",
                     "skinny_gemm_split_k_num_variants", "skinny_gemm_split_k_get_variant",
                     "skinny_gemm_split_k_default_plan"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
        return L


def _status_string(status: int) -> str:
    try:
        return lib().skinny_gemm_status_string(int(status)).decode()
    except Exception:  # pragma: no cover - library not loadable
        return "unknown status"


def _check(status: int, where: str) -> int:
    if status < 0:
        raise SkinnyError(status, where)
    return status


# ---- raw entry points (same names as the C ABI) -----------------------------

def skinny_gemm_init(device: int) -> None:
    _check(lib().skinny_gemm_init(int(device)), "skinny_gemm_init")


def skinny_gemm_bf16(x: int, W: int, y: int, M: int, N: int, K: int, stream: int = 0) -> None:
    _check(lib().skinny_gemm_bf16(x, W, y, M, N, K, stream), "skinny_gemm_bf16")


def skinny_gemm_bf16_pair(x: int, W0: int, W1: int, y0: int, y1: int, M: int, N: int, K: int,
                          stream: int = 0) -> None:
    _check(lib().skinny_gemm_bf16_pair(x, W0, W1, y0, y1, M, N, K, stream), "skinny_gemm_bf16_pair")


def skinny_gemm_bf16_ex(x: int, W: int, y: int, M: int, N: int, K: int, plan: Plan,
                        stream: int = 0) -> None:
    _check(lib().skinny_gemm_bf16_ex(x, W, y, M, N, K, ctypes.byref(plan), stream),
           "skinny_gemm_bf16_ex")


def skinny_gemm_bf16_pair_ex(x: int, W0: int, W1: int, y0: int, y1: int, M: int, N: int, K: int,
                             plan: Plan, stream: int = 0) -> None:
    _check(lib().skinny_gemm_bf16_pair_ex(x, W0, W1, y0, y1, M, N, K, ctypes.byref(plan), stream),
           "skinny_gemm_bf16_pair_ex")


def skinny_gemm_bf16_pair_strided(x0: int, x1: int, ldx: int, W0: int, W1: int, y0: int, y1: int,
                                  ldy: int, M: int, N: int, K: int, stream: int = 0) -> None:
    _check(lib().skinny_gemm_bf16_pair_strided(x0, x1, ldx, W0, W1, y0, y1, ldy, M, N, K, stream),
           "skinny_gemm_bf16_pair_strided")


def skinny_gemm_bf16_pair_strided_ex(x0: int, x1: int, ldx: int, W0: int, W1: int, y0: int, y1: int,
                                     ldy: int, M: int, N: int, K: int, plan: Plan,
                                     stream: int = 0) -> None:
    _check(lib().skinny_gemm_bf16_pair_strided_ex(x0, x1, ldx, W0, W1, y0, y1, ldy, M, N, K,
                                                  ctypes.byref(plan), stream),
           "skinny_gemm_bf16_pair_strided_ex")


def skinny_gemm_bf16_f32out(x: int, W: int, y: int, M: int, N: int, K: int, stream: int = 0) -> None:
    _check(lib().skinny_gemm_bf16_f32out(x, W, y, M, N, K, stream), "skinny_gemm_bf16_f32out")


def skinny_gemm_bf16_f32out_ex(x: int, W: int, y: int, M: int, N: int, K: int, plan: Plan,
                               stream: int = 0) -> None:
    _check(lib().skinny_gemm_bf16_f32out_ex(x, W, y, M, N, K, ctypes.byref(plan), stream),
           "skinny_gemm_bf16_f32out_ex")


def skinny_gemm_get_plan(N: int, K: int, M: int) -> tuple[Plan, bool]:
    """(plan, tuned): the plan skinny_gemm_bf16 uses for (N, K, M)."""
    p = Plan()
    r = _check(lib().skinny_gemm_get_plan(N, K, M, ctypes.byref(p)), "skinny_gemm_get_plan")
    return p, bool(r == 1)


def skinny_gemm_num_variants() -> int:
    return lib().skinny_gemm_num_variants()


def skinny_gemm_get_variant(index: int) -> Plan:
    p = Plan()
    _check(lib().skinny_gemm_get_variant(index, ctypes.byref(p)), "skinny_gemm_get_variant")
    return p


def skinny_gemm_status_string(status: int) -> str:
    return _status_string(status)


def skinny_gemm_version() -> int:
    return lib().skinny_gemm_version()


def variants() -> list[Plan]:
    return [skinny_gemm_get_variant(i) for i in range(skinny_gemm_num_variants())]


def _plan_ref(plan: Plan | None):
    return ctypes.byref(plan) if plan is not None else None


def skinny_gemm_split_k_workspace_bytes(M: int, N: int, K: int, plan: Plan | None = None) -> int:
    """Workspace bytes of a split-K call (0: no call with these arguments is accepted)."""
    return int(lib().skinny_gemm_split_k_workspace_bytes(M, N, K, _plan_ref(plan)))


def skinny_gemm_bf16_split_k(x: int, W: int, y: int, M: int, N: int, K: int, plan: Plan | None,
                             workspace: int, workspace_bytes: int, stream: int = 0) -> None:
    _check(lib().skinny_gemm_bf16_split_k(x, W, y, M, N, K, _plan_ref(plan), workspace,
                                          workspace_bytes, stream), "skinny_gemm_bf16_split_k")


def skinny_gemm_bf16_split_k_noalloc(x: int, W: int, y: int, M: int, N: int, K: int,
                                     plan: Plan | None = None, stream: int = 0) -> None:
    _check(lib().skinny_gemm_bf16_split_k_noalloc(x, W, y, M, N, K, _plan_ref(plan), stream),
           "skinny_gemm_bf16_split_k_noalloc")


def skinny_gemm_split_k_num_variants() -> int:
    return lib().skinny_gemm_split_k_num_variants()


def skinny_gemm_split_k_get_variant(index: int) -> Plan:
    p = Plan()
    _check(lib().skinny_gemm_split_k_get_variant(index, ctypes.byref(p)),
           "skinny_gemm_split_k_get_variant")
    return p


def skinny_gemm_split_k_default_plan(M: int, N: int, K: int) -> Plan:
    p = Plan()
    _check(lib().skinny_gemm_split_k_default_plan(M, N, K, ctypes.byref(p)),
           "skinny_gemm_split_k_default_plan")
    return p


def split_k_variants() -> list[Plan]:
    return [skinny_gemm_split_k_get_variant(i) for i in range(skinny_gemm_split_k_num_variants())]


def skinny_rms_norm_bf16(args: NormArgs, stream: int = 0) -> None:
    _check(lib().skinny_rms_norm_bf16(ctypes.byref(args), stream), "skinny_rms_norm_bf16")


def skinny_rms_norm_fp8(args: NormArgs, stream: int = 0) -> None:
    _check(lib().skinny_rms_norm_fp8(ctypes.byref(args), stream), "skinny_rms_norm_fp8")


def skinny_rms_norm_int8(args: NormArgs, stream: int = 0) -> None:
    _check(lib().skinny_rms_norm_int8(ctypes.byref(args), stream), "skinny_rms_norm_int8")


def skinny_quantize_int8(args: NormArgs, stream: int = 0) -> None:
    _check(lib().skinny_quantize_int8(ctypes.byref(args), stream), "skinny_quantize_int8")


def skinny_linear_bf16(args: LinearArgs, stream: int = 0) -> None:
    _check(lib().skinny_linear_bf16(ctypes.byref(args), stream), "skinny_linear_bf16")


def skinny_linear_fp8(args: LinearArgs, stream: int = 0) -> None:
    _check(lib().skinny_linear_fp8(ctypes.byref(args), stream), "skinny_linear_fp8")


def skinny_linear_int8(args: LinearArgs, stream: int = 0) -> None:
    _check(lib().skinny_linear_int8(ctypes.byref(args), stream), "skinny_linear_int8")


def skinny_linear_default_plan(args: LinearArgs, compute_units: int = 256) -> LinearPlan:
    p = LinearPlan()
    _check(lib().skinny_linear_default_plan(ctypes.byref(args), compute_units, ctypes.byref(p)),
           "skinny_linear_default_plan")
    return p


def skinny_linear_int8_default_plan(args: LinearArgs, compute_units: int = 256) -> LinearPlan:
    p = LinearPlan()
    _check(lib().skinny_linear_int8_default_plan(ctypes.byref(args), compute_units, ctypes.byref(p)),
           "skinny_linear_int8_default_plan")
    return p


def skinny_route(args: RouteArgs, stream: int = 0) -> None:
    _check(lib().skinny_route(ctypes.byref(args), stream), "skinny_route")


def skinny_experts_workspace_bytes(M: int, k: int, E: int, I: int) -> int:
    """Workspace bytes of an experts call (0: no call with these sizes is accepted, or M is 0)."""
    return int(lib().skinny_experts_workspace_bytes(M, k, E, I))


def skinny_experts(args: ExpertsArgs, stream: int = 0) -> None:
    _check(lib().skinny_experts(ctypes.byref(args), stream), "skinny_experts")


# ---- tensor helpers ---------------------------------------------------------

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(device: torch.device) -> int:
    """The raw handle of torch's current stream on `device` (no Stream object built
    when torch exposes the raw getter)."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    if _raw_stream is not None:
        return int(_raw_stream(idx))
    return int(torch.cuda.current_stream(idx).cuda_stream)


class _on_device:
    """Make `device` current for the call, switching only when it is not already."""

    __slots__ = ("idx", "prev")

    def __init__(self, device: torch.device):
        self.idx = device.index
        self.prev = None

    def __enter__(self):
        if self.idx is not None:
            cur = torch.cuda.current_device()
            if cur != self.idx:
                self.prev = cur
                torch.cuda.set_device(self.idx)
        return self

    def __exit__(self, *exc):
        if self.prev is not None:
            torch.cuda.set_device(self.prev)
        return False


def _check_tensor(t: torch.Tensor, name: str, ndim: int = 2) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def gemm(x: torch.Tensor, W: torch.Tensor, out: torch.Tensor | None = None,
         plan: Plan | None = None, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """y = x @ W.T for bfloat16 x [M, K] (M <= 8) and W [N, K]; one kernel launch
    on the current stream. out_dtype torch.float32 keeps the float32 sums
    (skinny_gemm_bf16_f32out)."""
    _check_tensor(x, "x")
    _check_tensor(W, "W")
    M, K = x.shape
    N, K2 = W.shape
    if K != K2:
        raise ValueError(f"inner sizes differ: x {tuple(x.shape)}, W {tuple(W.shape)}")
    if W.device != x.device:
        raise ValueError("x and W must be on the same device")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    else:
        if out.dtype != out_dtype or out.device != x.device or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous {out_dtype} tensor on {x.device}")
        if tuple(out.shape) != (M, N):
            raise ValueError(f"out must be [{M}, {N}]")
    s = _stream_handle(x.device)
    with _on_device(x.device):
        if out_dtype == torch.float32:
            if plan is None:
                skinny_gemm_bf16_f32out(x.data_ptr(), W.data_ptr(), out.data_ptr(), M, N, K, s)
            else:
                skinny_gemm_bf16_f32out_ex(x.data_ptr(), W.data_ptr(), out.data_ptr(), M, N, K,
                                           plan, s)
        elif plan is None:
            skinny_gemm_bf16(x.data_ptr(), W.data_ptr(), out.data_ptr(), M, N, K, s)
        else:
            skinny_gemm_bf16_ex(x.data_ptr(), W.data_ptr(), out.data_ptr(), M, N, K, plan, s)
    return out


def gemm_pair(x: torch.Tensor, W0: torch.Tensor, W1: torch.Tensor,
              out0: torch.Tensor | None = None, out1: torch.Tensor | None = None,
              plan: Plan | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(x @ W0.T, x @ W1.T) for two same-shape bfloat16 weights, one kernel launch."""
    _check_tensor(x, "x")
    _check_tensor(W0, "W0")
    _check_tensor(W1, "W1")
    M, K = x.shape
    if tuple(W0.shape) != tuple(W1.shape) or W0.shape[1] != K:
        raise ValueError(f"shapes: x {tuple(x.shape)}, W0 {tuple(W0.shape)}, W1 {tuple(W1.shape)}")
    N = W0.shape[0]
    if W0.device != x.device or W1.device != x.device:
        raise ValueError("x, W0 and W1 must be on the same device")
    outs = []
    for o, name in ((out0, "out0"), (out1, "out1")):
        if o is None:
            o = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
        else:
            _check_tensor(o, name)
            if o.device != x.device:
                raise ValueError(f"{name} must be on {x.device}")
            if tuple(o.shape) != (M, N):
                raise ValueError(f"{name} must be [{M}, {N}]")
        outs.append(o)
    s = _stream_handle(x.device)
    with _on_device(x.device):
        if plan is None:
            skinny_gemm_bf16_pair(x.data_ptr(), W0.data_ptr(), W1.data_ptr(), outs[0].data_ptr(),
                                  outs[1].data_ptr(), M, N, K, s)
        else:
            skinny_gemm_bf16_pair_ex(x.data_ptr(), W0.data_ptr(), W1.data_ptr(), outs[0].data_ptr(),
                                     outs[1].data_ptr(), M, N, K, plan, s)
    return outs[0], outs[1]


def _check_rowview(t: torch.Tensor, name: str) -> None:
    """A 2-D bfloat16 GPU view with unit column stride (rows may be strided)."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.device.type != "cuda":
        raise TypeError(f"{name} must be a bfloat16 GPU tensor")
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride, got stride {t.stride()}")


def gemm_pair_strided(x0: torch.Tensor, x1: torch.Tensor, W0: torch.Tensor, W1: torch.Tensor,
                      out0: torch.Tensor | None = None, out1: torch.Tensor | None = None,
                      plan: Plan | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(x0 @ W0.T, x1 @ W1.T) in one launch, x0 and x1 being row-strided views with
    the same row stride (e.g. the two halves of a merged [M, 2K] activation); out0
    and out1 may likewise be views of one merged [M, 2N] output."""
    _check_rowview(x0, "x0")
    _check_rowview(x1, "x1")
    _check_tensor(W0, "W0")
    _check_tensor(W1, "W1")
    M, K = x0.shape
    if tuple(x1.shape) != (M, K) or x1.stride(0) != x0.stride(0):
        raise ValueError("x0 and x1 must have the same shape and row stride")
    if tuple(W0.shape) != tuple(W1.shape) or W0.shape[1] != K:
        raise ValueError(f"shapes: x {tuple(x0.shape)}, W0 {tuple(W0.shape)}, W1 {tuple(W1.shape)}")
    N = W0.shape[0]
    if x1.device != x0.device or W0.device != x0.device or W1.device != x0.device:
        raise ValueError("x0, x1, W0 and W1 must be on the same device")
    if out0 is None and out1 is None:
        merged = torch.empty((M, 2 * N), dtype=torch.bfloat16, device=x0.device)
        out0, out1 = merged[:, :N], merged[:, N:]
    elif out0 is None or out1 is None:
        raise ValueError("give both out0 and out1, or neither")
    for o, name in ((out0, "out0"), (out1, "out1")):
        _check_rowview(o, name)
        if o.device != x0.device:
            raise ValueError(f"{name} must be on {x0.device}")
        if tuple(o.shape) != (M, N):
            raise ValueError(f"{name} must be [{M}, {N}]")
    if out0.stride(0) != out1.stride(0):
        raise ValueError("out0 and out1 must have the same row stride")
    ldx = x0.stride(0) if M > 1 else K
    ldy = out0.stride(0) if M > 1 else N
    s = _stream_handle(x0.device)
    with _on_device(x0.device):
        args = (x0.data_ptr(), x1.data_ptr(), ldx, W0.data_ptr(), W1.data_ptr(), out0.data_ptr(),
                out1.data_ptr(), ldy, M, N, K)
        if plan is None:
            skinny_gemm_bf16_pair_strided(*args, s)
        else:
            skinny_gemm_bf16_pair_strided_ex(*args, plan, s)
    return out0, out1


def split_k_workspace(M: int, N: int, K: int, plan: Plan | None = None,
                      device: torch.device | str = "cuda") -> torch.Tensor:
    """A zero-filled uint8 device buffer big enough for split-K calls of this shape
    and plan (allocate it once, outside any graph capture, and reuse it)."""
    nbytes = skinny_gemm_split_k_workspace_bytes(M, N, K, plan)
    if nbytes == 0:
        raise SkinnyError(SKINNY_ERR_INVALID_ARG, "skinny_gemm_split_k_workspace_bytes")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def _split_args(x: torch.Tensor, W: torch.Tensor, out: torch.Tensor | None):
    _check_tensor(x, "x")
    _check_tensor(W, "W")
    M, K = x.shape
    N, K2 = W.shape
    if K != K2:
        raise ValueError(f"inner sizes differ: x {tuple(x.shape)}, W {tuple(W.shape)}")
    if W.device != x.device:
        raise ValueError("x and W must be on the same device")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    else:
        _check_tensor(out, "out")
        if out.device != x.device or tuple(out.shape) != (M, N):
            raise ValueError(f"out must be a contiguous bfloat16 [{M}, {N}] tensor on {x.device}")
    return M, N, K, out


def gemm_split_k(x: torch.Tensor, W: torch.Tensor, workspace: torch.Tensor,
                 plan: Plan | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """y = x @ W.T with cross-block split-K (skinny_gemm_bf16_split_k), partials in
    `workspace` (from split_k_workspace, reused across calls on one stream)."""
    M, N, K, out = _split_args(x, W, out)
    if workspace.device != x.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {x.device}")
    s = _stream_handle(x.device)
    with _on_device(x.device):
        skinny_gemm_bf16_split_k(x.data_ptr(), W.data_ptr(), out.data_ptr(), M, N, K, plan,
                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(), s)
    return out


def gemm_split_k_noalloc(x: torch.Tensor, W: torch.Tensor, plan: Plan | None = None,
                         out: torch.Tensor | None = None) -> torch.Tensor:
    """y = x @ W.T with cross-block split-K on the library's static workspace
    (skinny_gemm_bf16_split_k_noalloc); with `out` given, nothing is allocated."""
    M, N, K, out = _split_args(x, W, out)
    s = _stream_handle(x.device)
    with _on_device(x.device):
        skinny_gemm_bf16_split_k_noalloc(x.data_ptr(), W.data_ptr(), out.data_ptr(), M, N, K, plan, s)
    return out


def _matrix(t: torch.Tensor, name: str, dtype: torch.dtype, device: torch.device,
            shape: tuple | None = None) -> int:
    """Check a 2-D row-strided GPU matrix and return its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device.type != "cuda" or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {device or 'a GPU'}, got {t.device}")
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must be {list(shape) if shape else '2-D'}, got {list(t.shape)}")
    if max(t.shape) > 0x7FFFFFFF:  # the argument structures would cut them off
        raise ValueError(f"{name}'s sizes must fit in 31 bits, got {list(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride, got stride {t.stride()}")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _vector(t: torch.Tensor | None, name: str, dtype: torch.dtype, device: torch.device,
            shape: tuple) -> int | None:
    """Check an optional contiguous GPU tensor and return its address."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.device != device or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor on {device}, got "
                         f"{list(t.shape)} on {t.device}")
    return t.data_ptr()


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: torch.Tensor | None = None, quant: str | None = None,
             out: torch.Tensor | None = None, scale: torch.Tensor | None = None,
             residual_out: torch.Tensor | None = None):
    """Root-mean-square norm of x [M, D] (rows may be strided), or of x + residual:
    y = h * weight / sqrt(mean(h^2) + eps), one kernel launch on the current stream.

    quant None: y is bfloat16. quant "row" or "group": y is float8_e4m3fn with float32
    scales per row ([M]) or per 128 columns ([M, ceil(D / 128)]). quant "int8": y is int8 with
    float32 scales per row. Returns y, or (y, scale) with quant; with a residual the new residual h (bfloat16) is returned last. out, scale
    and residual_out may be given; residual_out may be residual or x, and out may be x."""
    ldx = _matrix(x, "x", torch.bfloat16, None)
    M, D = x.shape
    if D == 0:
        raise ValueError("the width must be above 0")
    if quant not in (None, "row", "group", "int8"):
        raise ValueError(f"quant must be None, 'row', 'group' or 'int8', got {quant!r}")
    if residual is None and residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if quant is None and scale is not None:
        raise ValueError("scale needs quant")
    a = NormArgs(x=x.data_ptr(), ldx=ldx, M=M, D=D, eps=eps, group=128 if quant == "group" else 0)
    a.weight = _vector(weight, "weight", torch.bfloat16, x.device, (D,))
    if weight is None:
        raise TypeError("weight must be a torch.Tensor")
    dtype = torch.bfloat16 if quant is None else torch.int8 if quant == "int8" else torch.float8_e4m3fn
    if out is None:
        out = torch.empty((M, D), dtype=dtype, device=x.device)
    a.ldy = _matrix(out, "out", dtype, x.device, (M, D))
    a.y = out.data_ptr()
    if residual is not None:
        a.ldr = _matrix(residual, "residual", torch.bfloat16, x.device, (M, D))
        a.residual = residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty((M, D), dtype=torch.bfloat16, device=x.device)
        a.ldro = _matrix(residual_out, "residual_out", torch.bfloat16, x.device, (M, D))
        a.residual_out = residual_out.data_ptr()
    got = [out]
    if quant is not None:
        shape = (M, -(-D // 128)) if quant == "group" else (M,)
        if scale is None:
            scale = torch.empty(shape, dtype=torch.float32, device=x.device)
        a.scale = _vector(scale, "scale", torch.float32, x.device, shape)
        got.append(scale)
    if residual is not None:
        got.append(residual_out)
    s = _stream_handle(x.device)
    with _on_device(x.device):
        (skinny_rms_norm_bf16 if quant is None else
         skinny_rms_norm_int8 if quant == "int8" else skinny_rms_norm_fp8)(a, s)
    return got[0] if len(got) == 1 else tuple(got)


def quantize_int8(x: torch.Tensor, out: torch.Tensor | None = None,
                  scale: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(q, scale): the rows of bfloat16 x [M, D] (rows may be strided) as int8 [M, D] with one
    float32 scale each [M], the row's largest magnitude / 127; one kernel launch on the
    current stream. out and scale may be given."""
    ldx = _matrix(x, "x", torch.bfloat16, None)
    M, D = x.shape
    if D == 0:
        raise ValueError("the width must be above 0")
    if out is None:
        out = torch.empty((M, D), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty((M,), dtype=torch.float32, device=x.device)
    a = NormArgs(x=x.data_ptr(), ldx=ldx, M=M, D=D, y=out.data_ptr(),
                 ldy=_matrix(out, "out", torch.int8, x.device, (M, D)),
                 scale=_vector(scale, "scale", torch.float32, x.device, (M,)))
    s = _stream_handle(x.device)
    with _on_device(x.device):
        skinny_quantize_int8(a, s)
    return out, scale


def linear(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None,
           residual: torch.Tensor | None = None, act: str = "none",
           W_up: torch.Tensor | None = None, bias_up: torch.Tensor | None = None,
           x_scale: torch.Tensor | None = None, w_scale: torch.Tensor | None = None,
           w_up_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
           out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """y = act(x @ W.T + bias) + residual for any number of rows of x [M, K] (rows may be
    strided), or the gated form act(x @ W.T + bias) * (x @ W_up.T + bias_up); one kernel
    launch on the current stream.

    x and W are bfloat16, or int8 with float32 scales per row (x_scale [M], w_scale [N]; K at
    most 131071), or float8_e4m3fn with float32 scales: per row (x_scale [M],
    w_scale [N]) or per 128 columns of x and 128 x 128 block of W (x_scale
    [M, ceil(K/128)], w_scale [ceil(N/128), ceil(K/128)]). act: none, relu, gelu,
    gelu_tanh or silu. out may be given; a bfloat16 out may be the residual itself."""
    int8 = isinstance(x, torch.Tensor) and x.dtype == torch.int8
    fp8 = isinstance(x, torch.Tensor) and x.dtype == torch.float8_e4m3fn
    dtype = x.dtype if int8 or fp8 else torch.bfloat16
    ldx = _matrix(x, "x", dtype, None)
    M, K = x.shape
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, got {act!r}")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    _matrix(W, "W", dtype, x.device)
    N = W.shape[0]
    if tuple(W.shape) != (N, K):
        raise ValueError(f"inner sizes differ: x {tuple(x.shape)}, W {tuple(W.shape)}")
    if W_up is None and bias_up is not None:
        raise ValueError("bias_up needs W_up")
    if W_up is not None and residual is not None:
        raise ValueError("the gated form takes no residual")
    if W_up is not None and N * K == 0 and M > 0:
        raise ValueError("the gated form needs N and K above 0")
    if int8 and K > 131071:
        raise ValueError(f"int8 sums hold at most 131071 products, got {K}")
    if not (int8 or fp8) and not (x_scale is None and w_scale is None and w_up_scale is None):
        raise ValueError("scales belong to float8_e4m3fn and int8 inputs")
    a = LinearArgs(x=x.data_ptr(), ldx=ldx, M=M, N=N, K=K, act=ACTS[act],
                   out_f32=out_dtype == torch.float32)
    a.W0 = _vector(W, "W", dtype, x.device, (N, K))
    a.W1 = _vector(W_up, "W_up", dtype, x.device, (N, K))
    a.bias0 = _vector(bias, "bias", torch.bfloat16, x.device, (N,))
    a.bias1 = _vector(bias_up, "bias_up", torch.bfloat16, x.device, (N,))
    if int8 or fp8:
        if x_scale is None or w_scale is None or (W_up is not None) != (w_up_scale is not None):
            raise ValueError(f"{dtype} inputs need x_scale and a scale for each weight")
        blocks = fp8 and w_scale.dim() == 2
        kb, nb = -(-K // 128), -(-N // 128)
        a.scales = SKINNY_SCALES_BLOCK if blocks else SKINNY_SCALES_ROW
        ws = (nb, kb) if blocks else (N,)
        a.x_scale = _vector(x_scale, "x_scale", torch.float32, x.device, (M, kb) if blocks else (M,))
        a.w0_scale = _vector(w_scale, "w_scale", torch.float32, x.device, ws)
        a.w1_scale = _vector(w_up_scale, "w_up_scale", torch.float32, x.device, ws)
    if residual is not None:
        a.ldr = _matrix(residual, "residual", torch.bfloat16, x.device, (M, N))
        a.residual = residual.data_ptr()
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    a.ldy = _matrix(out, "out", out_dtype, x.device, (M, N))
    a.y = out.data_ptr()
    s = _stream_handle(x.device)
    with _on_device(x.device):
        (skinny_linear_fp8 if fp8 else skinny_linear_int8 if int8 else skinny_linear_bf16)(a, s)
    return out


def route(logits: torch.Tensor, k: int, score: str = "softmax", bias: torch.Tensor | None = None,
          groups: int = 1, kept: int = 1, renormalize: bool = True, scale: float = 1.0,
          out_ids: torch.Tensor | None = None,
          out_weights: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(ids, weights), int32 and float32 [M, k]: the k best of the experts of float32 logits
    [M, E] (rows may be strided), best first and equal ones by index, and scale times their
    scores ("softmax" over the row or "sigmoid"), which renormalize makes sum to 1 before. They
    are ranked by the logits, or by score + bias where float32 bias [E] is given. groups > 1
    takes them from `kept` of that many runs of experts only: those of the largest rank, or,
    with a bias, of the largest sum of two ranks. One kernel launch on the current stream;
    E at most 1024, k and groups at most 64. out_ids and out_weights may be given."""
    ldl = _matrix(logits, "logits", torch.float32, None)
    M, E = logits.shape
    if score not in SCORES:
        raise ValueError(f"score must be one of {', '.join(SCORES)}, got {score!r}")
    if not 1 <= E <= 1024:
        raise ValueError(f"the number of experts must be 1..1024, got {E}")
    if not (1 <= groups <= 64 and E % groups == 0 and 1 <= kept <= groups):
        raise ValueError(f"groups must be 1..64 and divide {E}, and kept 1..groups, got {groups} and {kept}")
    if not 1 <= k <= min(64, kept * (E // groups)):
        raise ValueError(f"k must be 1..{min(64, kept * (E // groups))}, got {k}")
    if out_ids is None:
        out_ids = torch.empty((M, k), dtype=torch.int32, device=logits.device)
    if out_weights is None:
        out_weights = torch.empty((M, k), dtype=torch.float32, device=logits.device)
    a = RouteArgs(logits=logits.data_ptr(), ldl=ldl, M=M, E=E, k=k, score=SCORES[score], groups=groups, kept=kept,
                  renormalize=bool(renormalize), scale=scale,
                  bias=_vector(bias, "bias", torch.float32, logits.device, (E,)),
                  ids=_vector(out_ids, "out_ids", torch.int32, logits.device, (M, k)),
                  weights=_vector(out_weights, "out_weights", torch.float32, logits.device, (M, k)))
    s = _stream_handle(logits.device)
    with _on_device(logits.device):
        skinny_route(a, s)
    return out_ids, out_weights


def _stack(t: torch.Tensor, name: str, dtype: torch.dtype, device: torch.device, shape: tuple) -> int:
    """Check a GPU tensor whose parts t[e] are contiguous and return the stride of e."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.device != device or tuple(t.shape) != tuple(shape) or (shape[0] > 0 and not t[0].is_contiguous()):
        raise ValueError(f"{name} must be {list(shape)} with contiguous parts on {device}, got {list(t.shape)} of strides "
                         f"{t.stride()} on {t.device}")
    return t.stride(0) if shape[0] > 1 else t[0].numel()


def experts_workspace(M: int, k: int, E: int, I: int, device: torch.device | str = "cuda") -> torch.Tensor:
    """A uint8 device buffer big enough for experts calls of up to M rows with these sizes (to
    reuse in calls that follow one another on one stream)."""
    nbytes = skinny_experts_workspace_bytes(M, k, E, I)
    if nbytes == 0:
        raise SkinnyError(SKINNY_ERR_INVALID_ARG, "skinny_experts_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w_gate: torch.Tensor,
            w_up: torch.Tensor, w_down: torch.Tensor, gate_scale: torch.Tensor | None = None,
            up_scale: torch.Tensor | None = None, down_scale: torch.Tensor | None = None,
            residual: torch.Tensor | None = None, act: str = "silu", out: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m] = sum_j weights[m, j] * (act(x[m] @ w_gate[e].T) * (x[m] @ w_up[e].T)) @ w_down[e].T
    + residual[m] with e = ids[m, j], for bfloat16 x [M, H] (rows may be strided), int32 ids and
    float32 weights [M, k]; an id outside 0..E-1 is left out.

    w_gate and w_up [E, I, H] and w_down [E, H, I] are bfloat16, or int8 with float32 scales per
    row (gate_scale and up_scale [E, I], down_scale [E, H]), or float8_e4m3fn with those or with
    scales per 128 x 128 block ([E, ceil(I/128), ceil(H/128)], [E, ceil(H/128), ceil(I/128)]). Parts
    [e] must be contiguous; the two halves of a merged [E, 2 I, H] weight are taken as views.
    Two kernel launches for every 128 rows on the current stream; for up to some hundred rows.
    act(..) * (..) is rounded to bfloat16 in batches that give an expert more than a few rows, and
    held in 16 bits else, so a row's last bits depend on the batch. out (which may be the residual)
    and workspace (from experts_workspace) may be given."""
    ldx = _matrix(x, "x", torch.bfloat16, None)
    M, H = x.shape
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, got {act!r}")
    if not isinstance(w_gate, torch.Tensor) or w_gate.dtype not in (torch.bfloat16, torch.int8, torch.float8_e4m3fn):
        raise TypeError("w_gate must be a bfloat16, int8 or float8_e4m3fn tensor")
    if w_gate.dim() != 3:
        raise ValueError(f"w_gate must be [E, I, H], got {list(w_gate.shape)}")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be an [M, k] tensor")
    dtype, (E, I, _), k = w_gate.dtype, w_gate.shape, ids.shape[1]
    if not (1 <= E <= 1024 and 1 <= k <= 32 and H >= 1 and I >= 1):
        raise ValueError(f"E must be 1..1024, k 1..32, H and I above 0, got {E}, {k}, {H} and {I}")
    if max(H, I) > 0x7FFFFFFF:
        raise ValueError(f"H and I must fit in 31 bits, got {H} and {I}")
    a = ExpertsArgs(x=x.data_ptr(), ldx=ldx, M=M, E=E, k=k, H=H, I=I, act=ACTS[act])
    a.ids = _vector(ids, "ids", torch.int32, x.device, (M, k))
    a.weights = _vector(weights, "weights", torch.float32, x.device, (M, k))
    if weights is None:
        raise TypeError("weights must be a torch.Tensor")
    a.up_stride = _stack(w_gate, "w_gate", dtype, x.device, (E, I, H))
    if _stack(w_up, "w_up", dtype, x.device, (E, I, H)) != a.up_stride:
        raise ValueError("w_gate and w_up must have the same strides")
    a.down_stride = _stack(w_down, "w_down", dtype, x.device, (E, H, I))
    a.w_gate, a.w_up, a.w_down = w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr()
    if dtype == torch.bfloat16:
        if not (gate_scale is None and up_scale is None and down_scale is None):
            raise ValueError("scales belong to float8_e4m3fn and int8 weights")
    else:
        if gate_scale is None or up_scale is None or down_scale is None:
            raise ValueError(f"{dtype} weights need a scale each")
        blocks = dtype == torch.float8_e4m3fn and gate_scale.dim() == 3
        hb, ib = -(-H // 128), -(-I // 128)
        a.type = (SKINNY_WEIGHTS_INT8_ROW if dtype == torch.int8 else
                  SKINNY_WEIGHTS_E4M3_BLOCK if blocks else SKINNY_WEIGHTS_E4M3_ROW)
        shape = (E, ib, hb) if blocks else (E, I)
        a.up_scale_stride = _stack(gate_scale, "gate_scale", torch.float32, x.device, shape)
        if _stack(up_scale, "up_scale", torch.float32, x.device, shape) != a.up_scale_stride:
            raise ValueError("gate_scale and up_scale must have the same strides")
        a.down_scale_stride = _stack(down_scale, "down_scale", torch.float32, x.device,
                                     (E, hb, ib) if blocks else (E, H))
        a.gate_scale, a.up_scale, a.down_scale = gate_scale.data_ptr(), up_scale.data_ptr(), down_scale.data_ptr()
    if residual is not None:
        a.ldr = _matrix(residual, "residual", torch.bfloat16, x.device, (M, H))
        a.residual = residual.data_ptr()
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    a.ldy = _matrix(out, "out", torch.bfloat16, x.device, (M, H))
    a.y = out.data_ptr()
    if M == 0:
        return out
    if workspace is None:
        workspace = experts_workspace(M, k, E, I, x.device)
    elif workspace.device != x.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {x.device}")
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    s = _stream_handle(x.device)
    with _on_device(x.device):
        skinny_experts(a, s)
    return out


__all__ = [
    "SkinnyError", "Plan", "lib", "variants", "gemm", "gemm_pair", "gemm_pair_strided",
    "split_k_variants", "split_k_workspace", "gemm_split_k", "gemm_split_k_noalloc",
    "skinny_gemm_split_k_workspace_bytes", "skinny_gemm_bf16_split_k",
    "skinny_gemm_bf16_split_k_noalloc", "skinny_gemm_split_k_num_variants",
    "skinny_gemm_split_k_get_variant", "skinny_gemm_split_k_default_plan", "SKINNY_KIND_SPLIT_K",
    "skinny_gemm_bf16_pair_strided", "skinny_gemm_bf16_pair_strided_ex",
    "skinny_gemm_init", "skinny_gemm_bf16", "skinny_gemm_bf16_pair", "skinny_gemm_bf16_ex",
    "skinny_gemm_bf16_pair_ex", "skinny_gemm_bf16_f32out", "skinny_gemm_bf16_f32out_ex",
    "skinny_gemm_get_plan", "skinny_gemm_num_variants",
    "skinny_gemm_get_variant", "skinny_gemm_status_string", "skinny_gemm_version",
    "SKINNY_OK", "SKINNY_ERR_INVALID_ARG", "SKINNY_ERR_UNSUPPORTED", "SKINNY_ERR_NOT_INITIALIZED",
    "SKINNY_ERR_LAUNCH", "SKINNY_KIND_FIXED_K", "SKINNY_KIND_LOOP_K", "SKINNY_KIND_SCALAR",
    "SKINNY_KIND_MFMA", "NormArgs", "LinearArgs", "LinearPlan", "ACTS", "rms_norm", "linear",
    "skinny_rms_norm_bf16", "skinny_rms_norm_fp8", "skinny_linear_bf16", "skinny_linear_fp8",
    "skinny_linear_default_plan", "RouteArgs", "ExpertsArgs", "SCORES", "route", "experts",
    "experts_workspace", "skinny_route", "skinny_experts", "skinny_experts_workspace_bytes",
    "SKINNY_SCORE_SOFTMAX", "SKINNY_SCORE_SIGMOID", "SKINNY_WEIGHTS_BF16", "SKINNY_WEIGHTS_E4M3_ROW",
    "SKINNY_WEIGHTS_E4M3_BLOCK", "SKINNY_WEIGHTS_INT8_ROW", "quantize_int8", "skinny_rms_norm_int8", "skinny_quantize_int8",
    "skinny_linear_int8", "skinny_linear_int8_default_plan", "SKINNY_LINEAR_ELEMENTS", "SKINNY_LINEAR_STREAM", "SKINNY_LINEAR_TILE",
    "SKINNY_ACT_NONE", "SKINNY_ACT_RELU", "SKINNY_ACT_GELU", "SKINNY_ACT_GELU_TANH",
    "SKINNY_ACT_SILU", "SKINNY_SCALES_ROW", "SKINNY_SCALES_BLOCK",
]

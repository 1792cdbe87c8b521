"""Each kernel that a projection may be given, against its definition in 64 bits: at a size that
takes it, ending inside a block of rows, of outputs and of K, with everything around the operands
NaN and everything around the result watched."""
from __future__ import annotations

import pytest
import torch

from .linear_choices import CHOICES, ROWS, SCALES
from .test_gpu_ops import check_linear, skg  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

KERNELS = [(key, i) for key in CHOICES for i in range(len(CHOICES[key]))]


def name(kernel):
    (scales, gated, rows, f32), i = kernel
    return "-".join([SCALES[scales], "gated" if gated else "one", ROWS[rows].replace(" ", ""),
                     "f32" if f32 else "any", str(i)])


@pytest.mark.parametrize("kernel", KERNELS, ids=name)
def test_kernel(skg, kernel):  # noqa: F811
    (scales, gated, rows, f32), i = kernel
    M, N, K = CHOICES[kernel[0]][i]
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("the sizes are for 256 compute units")
    mode = SCALES[scales]
    # a row stride of x that is no multiple of 128 bytes, but one of the 16 that kernels need
    ld = K + 16
    for out_f32 in ([bool(f32)] if (scales, gated, rows, 1) in CHOICES else [False, True]):
        if gated:
            check_linear(skg, M, N, K, mode, gated=True, act="silu", bias=True, f32=out_f32, ld=ld, ldy=N + 3,
                         seed=N + i)
        else:
            check_linear(skg, M, N, K, mode, act="gelu", bias=True, residual=True, f32=out_f32, ld=ld, ldy=N + 3,
                         seed=N + i)
        check_linear(skg, M, N, K, mode, gated=bool(gated), f32=out_f32, seed=K + i)

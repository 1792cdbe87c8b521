"""The argument checks of include/skinny_ops.h under the address and undefined-behaviour
sanitizers (host code only, plain C++)."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_ops_validation_under_asan_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    exe = str(tmp_path / "ops_fuzz")
    build = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
             "-D__HIP_PLATFORM_AMD__=1", "-I", os.path.join(ROOT, "include"),
             "-I", "/opt/rocm/include", os.path.join(ROOT, "tests", "sanitize", "ops_fuzz.cpp"), "-o", exe]
    res = subprocess.run(build, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, (res.stdout + res.stderr)[-4000:]
    assert "ops validation: ok" in res.stdout

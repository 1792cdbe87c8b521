"""The choice of the experts' kernels (csrc/experts_plan.hpp), asked on the CPU: every kernel that
calls choose among is taken by one of the sizes that the GPU tests run."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from .experts_choices import CHOICES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    exe = str(tmp_path_factory.mktemp("plan") / "experts_plan")
    build = [gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__=1", "-I", os.path.join(ROOT, "include"),
             "-I", "/opt/rocm/include", os.path.join(ROOT, "tests", "native", "experts_plan.cpp"), "-o", exe]
    res = subprocess.run(build, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]

    def ask(*args, sizes=()):
        lines = "".join(" ".join(map(str, s)) + "\n" for s in sizes)
        res = subprocess.run([exe, *args], input=lines, capture_output=True, text=True, timeout=60)
        assert res.returncode == 0
        return [line.split() for line in res.stdout.splitlines()]
    return ask


def test_every_offered_kernel_is_taken_by_a_size_that_is_run(ask):
    offered = {tuple(line) for line in ask("all")}
    sizes = [(kind, *s) for kinds in CHOICES for kind in kinds for s in CHOICES[kinds]]
    taken = {tuple(line[1:]) for line in ask(sizes=sizes)}
    assert taken == offered, (sorted(offered - taken), sorted(taken - offered))


def test_rows_and_places(ask):
    """Heights of tiles by the pairs of an expert; x in LDS as long as it fits, then streamed with
    at least 8 rows."""
    def plan(*size):
        up, down = ask(sizes=[size])
        assert up[1] == "up" and down[1] == "down" and up[4] == down[3] == up[0]
        return tuple(int(v) for v in (up[4], up[6], up[7]))  # rows, stages, room
    assert [plan(3, M, 64, 6, 2048)[0] for M in (1, 30, 61, 128)] == [4, 8, 16, 16]
    assert plan(0, 3, 64, 4, 14416)[::2] == plan(3, 70, 300, 2, 14416)[::2] == (8, 0)
    for kind in range(4):
        plans = [plan(kind, 16, 7, 4, H) for H in (512, 2800, 3200, 4096)]
        assert [p[1] for p in plans[:3]] == [6, 4, 3] and [p[2] > 0 for p in plans] == [True, True, True, False]

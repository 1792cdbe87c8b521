"""The tiled projection kernels share buffers in LDS between waves: behind each barrier some
buffer may be written again, so no wave may reach one with its own reads of that buffer still
on their way. No result shows a missing wait, so the built gfx950 code itself is read: at each
barrier no LDS read may be outstanding but the youngest two, and those only where they bring a
fragment of W (the first operand of the matrix products), whose buffer is freed later."""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def registers(operand):
    """{("v", 4), ("v", 5)} of "v[4:5]"; empty for anything but vector registers."""
    m = re.match(r"^([va])(?:(\d+)|\[(\d+):(\d+)\])$", operand.strip())
    if not m:
        return set()
    first, last = (m.group(2), m.group(2)) if m.group(2) else m.group(3, 4)
    return {(m.group(1), i) for i in range(int(first), int(last) + 1)}


def at_barriers(listing):
    """{kernel: [what is on its way at each barrier]}: "none", "W" (two reads or fewer, each of
    which a matrix product takes as its first operand next) or "other"."""
    kernels, reads, passed = {}, [], []
    for line in listing.splitlines():
        head = re.match(r"^[0-9a-f]+ <(.*)>:", line)
        if head:
            barriers = kernels.setdefault(head.group(1).split("(")[0], [])
            reads, passed = [], []
            continue
        op, _, rest = line.split("//")[0].strip().partition(" ")
        operands = [registers(o.split(" offset")[0]) for o in rest.split(",")]
        if op.startswith("ds_read"):
            reads.append(operands[0])
        elif op == "s_waitcnt" and (left := re.search(r"lgkmcnt\((\d+)\)", rest)):
            reads = reads[max(0, len(reads) - int(left.group(1))):]  # LDS returns in order
        elif op == "s_barrier":
            barriers.append("none" if not reads else "W" if len(reads) <= 2 else "other")
            if barriers[-1] == "W":
                passed += [(r, barriers, len(barriers) - 1) for r in reads]
        elif passed:
            used = [p for p in passed if any(p[0] & o for o in operands)]
            for dest, of, at in used:
                if not (op.startswith("v_mfma") and dest <= operands[1] and not dest & operands[2]):
                    of[at] = "other"
            passed = [p for p in passed if p not in used]
    for _, of, at in passed:
        of[at] = "other"
    return kernels


def test_reading_of_a_listing():
    """The reader itself, on lines of the form it reads."""
    got = at_barriers("""
0000000000001900 <void k<1>(A)>:
    ds_read_b128 v[0:3], v9
    ds_read_b128 v[4:7], v9 offset:16
    s_waitcnt vmcnt(3)
    s_barrier                                                  // 000000001904: BF8A0000
    s_waitcnt lgkmcnt(0)
    v_mfma_f32_16x16x128_f8f6f4 a[0:3], v[0:7], v[8:15], a[0:3]
    s_barrier
    ds_read_b128 v[0:3], v9
    s_waitcnt vmcnt(0) lgkmcnt(1)
    s_barrier
    v_mfma_f32_16x16x32_bf16 a[0:3], v[8:11], v[0:3], a[0:3]
0000000000001a00 <void k<2>(A)>:
    ds_read_b128 v[0:3], v9
    ds_read_b128 v[4:7], v9 offset:16
    ds_read_b32 v8, v9
    s_barrier
    s_waitcnt lgkmcnt(1)
    s_barrier
""")
    assert got == {"void k<1>": ["W", "none", "other"], "void k<2>": ["other", "other"]}


def test_no_wave_passes_a_barrier_before_its_reads_of_lds(tmp_path):
    from bf16_skinny_gemm_amd.build import LIB_PATH

    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    if not os.path.exists(LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    lib = shutil.copy(LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    tiles = {}
    for code in glob.glob(str(tmp_path / "*gfx950")):
        names = subprocess.run([OBJDUMP, "--syms", "-C", code], check=True, capture_output=True, text=True).stdout
        if "linear_tile_kernel" not in names:
            continue
        res = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "-C", code], check=True, capture_output=True,
                             text=True)
        tiles.update({k: v for k, v in at_barriers(res.stdout).items() if "linear_tile_kernel" in k})
    assert len(tiles) > 10 and all(len(v) >= 5 for v in tiles.values())
    assert {k: v for k, v in tiles.items() if "other" in v} == {}
    # with scales of blocks nothing pins the order of the reads: none may be outstanding
    assert {k: v for k, v in tiles.items() if "linear_tile_kernel<2" in k and set(v) != {"none"}} == {}

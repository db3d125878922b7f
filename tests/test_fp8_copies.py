"""The FP8 tile kernels as compiled: each operand line of a stage is copied into LDS once."""
import os
import re
import subprocess

import pytest

from block_scaled_precision_requant_amd import build

# BM, BN, WM, WN, RING, KG, silu, rows of each kernel (the instances of device/fp8_copies.hip)
KERNELS = [(16, 16, 16, 16, 4, 4, 0, 0), (16, 32, 16, 32, 4, 4, 0, 0), (16, 64, 16, 64, 3, 4, 0, 0),
           (16, 128, 16, 128, 2, 4, 0, 0), (64, 128, 32, 64, 3, 1, 0, 1), (128, 128, 64, 64, 2, 1, 1, 2),
           (32, 16, 32, 16, 4, 4, 0, 0), (64, 64, 64, 32, 3, 2, 0, 0), (256, 256, 128, 64, 2, 1, 0, 0)]


@pytest.fixture(scope="module")
def copies(tmp_path_factory):
    """Name of each kernel -> number of the 16-byte copies from memory to LDS inside its loops, as instructions."""
    out = str(tmp_path_factory.mktemp("copies") / "fp8_copies.s")
    subprocess.run([build.HIPCC, *build.FLAGS, "-S", "--offload-device-only",
                    os.path.join(os.path.dirname(os.path.abspath(__file__)), "device", "fp8_copies.hip"), "-o", out], check=True)
    found, name, inside = {}, None, False
    with open(out) as f:
        for line in f:
            start = re.match(r"(_Z\w*fp8_gemm_kernel\w*):", line)
            if start:
                name = start.group(1)
                found[name], inside = 0, False
            elif re.match(r"\.LBB|; %bb\.", line):  # a block, with the loop it is part of
                inside = "Loop Header" in line or "in Loop" in line
            elif inside and re.match(r"\s+buffer_load_dwordx4 .*\blds\b", line):
                found[name] += 1
    return found


@pytest.mark.parametrize("bm, bn, wm, wn, ring, kg, silu, rows", KERNELS)
def test_each_line_is_copied_once(copies, bm, bn, wm, wn, ring, kg, silu, rows):
    name = f"fp8_gemm_kernelILi{bm}ELi{bn}ELi{wm}ELi{wn}ELi{ring}ELi{kg}ELb{silu}ELNS0_4RowsE{rows}E"
    got = [n for k, n in copies.items() if name in k]
    assert len(got) == 1, list(copies)
    # what a wave copies of a stage, for each height of the kernel's tile (every height has its own loop)
    parts = [1]
    if rows and wm >= 64:
        parts.append(4)
    if rows and wm >= 32 and bm >= 64:
        parts.append(2)
    waves = bm // wm * (bn // wn)
    assert got[0] == sum(-(-(bm // p // 8) // waves) + bn // 8 // waves for p in parts)

"""Which kernel the limit tests of the grouped products reach (the host rule that the launcher runs)."""
import os
import subprocess

import pytest

import test_gpu_moe_limits as limits


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path_factory.mktemp("choice") / "grouped_choice")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", f"-I{root}/block_scaled_precision_requant_amd/csrc",
                    os.path.join(root, "tests", "host", "grouped_choice.cpp"), "-o", exe], check=True)
    return lambda *sizes: subprocess.run([exe, *map(str, sizes)], check=True, capture_output=True, text=True).stdout.strip()


def test_limit_cases_reach_both_kernels(choice):
    c = limits.PAST_4_GIB
    assert choice(sum(c["counts"].values()), c["experts"], c["n"], c["k"]) == "tiles"
    got = [choice(rows, experts, limits.GATHERED_N, k) for k, rows, experts in limits.GATHERED]
    assert got == ["gemv 16", "tiles"] * 2

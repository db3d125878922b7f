"""The host rule of the FP8 products: which kernel the GPU tests' sizes reach, and that a launch covers its output."""
import os
import random
import subprocess

import pytest

import test_gpu_fp8 as gpu

NUM_SHAPES = 17


@pytest.fixture(scope="module")
def choices(tmp_path_factory):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path_factory.mktemp("choice") / "fp8_choice")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", f"-I{root}/block_scaled_precision_requant_amd/csrc",
                    os.path.join(root, "tests", "host", "fp8_choice.cpp"), "-o", exe], check=True)

    def ask(cases):  # (rows, experts, n, k, silu) each -> (shape, bm, bn, tiles_m, tiles_n, threads)
        text = "\n".join(" ".join(str(int(v)) for v in c) for c in cases)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


def test_every_shape_is_tested(choices):
    dense = [c[0] for c in choices([(m, 1, n, k, 0) for m, n, k in gpu.SHAPES])]
    assert sorted(dense) == list(range(NUM_SHAPES)), dense
    heights = [c[1] for c in choices([(m, 1, 256 * (n // 256 + 1), k, 0) for m, n, k in gpu.SHAPES[8:]])]
    assert heights == [64, 64, 64, 64, 128, 128, 256, 256, 128], heights  # test_last_rows_of_an_expert
    assert {c[0] for c in choices([(m, 1, n, k, 0) for m, n, k in gpu.DENSE])} >= {-1}
    for silu in (0, 1):
        got = choices([(r, e, 256 * -(-n // 256) if silu else n, k, silu) for r, e, n, k, _ in gpu.GROUPED])
        want = set(range(NUM_SHAPES)) | {-1}
        if silu:
            want -= {0, 4, 8}  # (16 columns: a gate and an up tile are 32)
        assert {c[0] for c in got} >= want, sorted(want - {c[0] for c in got})


def test_a_launch_covers_the_output(choices):
    r = random.Random(5)
    cases = []
    for _ in range(3000):
        grouped, silu = r.random() < 0.5, r.random() < 0.3
        rows = int(2 ** r.uniform(0, 24))
        cases.append((rows, int(2 ** r.uniform(0, 16)) if grouped else 1, 256 * int(2 ** r.uniform(0, 8)) if silu else
                      int(2 ** r.uniform(0, 20)), 128 * int(2 ** r.uniform(0, 15)), silu and grouped))
    for (rows, experts, n, k, silu), (shape, bm, bn, tiles_m, tiles_n, threads) in zip(cases, choices(cases)):
        cols = n // 2 if silu and shape < 0 else n
        assert tiles_n * bn >= cols > (tiles_n - 1) * bn
        used = min(rows, experts)
        # whatever the offsets, each expert with rows adds less than one tile of padding
        assert tiles_m == (rows + used * (bm - 1)) // bm
        assert not silu or shape < 0 or bn >= 32
        assert threads % (tiles_m * tiles_n * 64) == 0 and threads // (tiles_m * tiles_n) <= 1024

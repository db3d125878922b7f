"""Which kernel the sizes of test_gpu_fp8_reach.py run, by the host rule."""
import pytest

import test_gpu_fp8_reach as gpu
from test_fp8_choices import NUM_SHAPES, choices  # noqa: F401  (a fixture)


@pytest.mark.parametrize("silu", [False, True])
def test_groups_of_every_shape_pass_64_blocks(choices, silu):  # noqa: F811
    cases = [(m, 1, 256 * (n // 256 + 1) if silu else n, k, silu) for m, n, k in gpu.LONG]
    seen = set()
    for (_, _, _, k, _), got in zip(cases, choices(cases)):
        assert got[0] >= 0
        if -(-(k // 128) // gpu.GROUPS[got[0]]) > 64:
            seen.add(got[0])
    # (the SiLU product has no tiles of 16 columns)
    assert seen == set(range(NUM_SHAPES)) - ({0, 4, 8} if silu else set())


def test_dense_and_one_expert_choose_alike(choices):  # noqa: F811
    got = choices([(m, 1, n, k, 0) for m, n, k in gpu.DENSE + gpu.SHAPES])
    assert {c[0] for c in got} == set(range(-1, NUM_SHAPES))


def test_past_4_gib(choices):  # noqa: F811
    n, k = gpu.WIDE_N, gpu.WIDE_K
    assert gpu.EXPERTS * n * k > 1 << 32
    for silu in (0, 1):
        assert [c[1:3] for c in choices([(3 + last, gpu.EXPERTS, n, k, silu) for last in gpu.LAST])] == [(64, 128), (256, 128), (256, 256)]
        assert choices([(gpu.GATHER_PICKS, 1, 512, k, silu)])[0][0] == -1  # streamed
    assert (1 << 32) - k <= gpu.GATHER_ROWS * k < 1 << 32

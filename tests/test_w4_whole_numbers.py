"""The whole-number cases of the 4-bit GEMV would show a lost part of K: checked on the CPU, with the mistake planted
in the reference."""
import numpy as np
import pytest

import test_gpu_w4_exact as w4


@pytest.mark.parametrize("m, n, k, group, zero", [c for c in w4.WHOLE if c[1] <= 1000])
def test_a_lost_block_changes_the_bits(m, n, k, group, zero):
    rng = np.random.default_rng(m * 3 + n + k + group)
    x, wp, scale, z, codes = w4.whole_case(rng, (), m, n, k, group, zero)
    want = w4.bf16_rne(w4.whole_product(x, codes, scale, z))
    assert np.array_equal(np.stack((wp & 15, wp >> 4), axis=-1).reshape(codes.shape), codes)
    blocks = k // 32
    for skip in ([0], [blocks // 2], [blocks - 1], range(blocks - blocks % 4, blocks)):
        if len(skip) == 0:
            continue
        lost = w4.bf16_rne(w4.whole_product(x, codes, scale, z, skip=skip))
        assert not w4.same_values(lost, want)
        if n >= 30:  # in every row of the output, and in every column tile of 16
            for tile in range(0, n - 15, 16):
                assert (lost[:, tile:tile + 16] != want[:, tile:tile + 16]).any(1).all()


@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_a_zero_point_off_by_one_changes_the_bits(group):
    rng = np.random.default_rng(group)
    x, _, scale, z, codes = w4.whole_case(rng, (), 3, 40, 14336, group, "4 bit")
    want = w4.bf16_rne(w4.whole_product(x, codes, scale, z))
    z[:, -1] += 1
    assert not w4.same_values(w4.bf16_rne(w4.whole_product(x, codes, scale, z)), want)

"""The 4-bit GEMV where every sum is exact."""
import numpy as np
import pytest
import torch

from block_scaled_precision_requant_amd import bsr
from gpu_util import DEV, canary_out, host, say, to_dev
from oracle.compare import bf16_bits_to_f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 3, 16])
@pytest.mark.parametrize("zero", [None, 5])
def test_row_scale_sums_do_not_cancel_over_all_of_k(m, zero):
    """One scale per weight row; elements e and e + 32 of every 64 have the same activation (193, 195 .. 255) and codes
    z + d and z - d, so they cancel, while a wave's sums of x * (16 + c) over its 4096 elements or more pass 2^24 and
    are odd there.  Only the last element of K has no counterpart: the output is scale * x * -d of it, and every sum
    over 128 elements is a whole number under 2^24 (at most 128 * 255 * 31)."""
    say("pairs", m, zero)
    n, k = 4096, 65536
    z = 8 if zero is None else zero
    g = torch.Generator(DEV).manual_seed(m)
    x = 2 * torch.randint(96, 128, (m, k // 64, 1, 32), device=DEV, generator=g) + 1
    x = x.expand(m, k // 64, 2, 32).reshape(m, k).clone()
    x[:, -33], x[:, -1] = 0, 3
    d = torch.randint(-5, 6, (n, k // 64, 1, 32), device=DEV, generator=g)
    codes = torch.cat((z + d, z - d), dim=2).reshape(n, k // 2, 2)                # within 0 .. 13
    wp = (codes[..., 0] | codes[..., 1] << 4).to(torch.uint8)
    # (a wave takes a 16th of K at least)
    assert (codes[0].reshape(-1, k // 16) * x[0].reshape(16, -1) + 16 * x[0].reshape(16, -1)).sum(1).max() > 1 << 24
    scale = torch.full((n, 1), 0.5, device=DEV)
    zt = None if zero is None else torch.full((n, 1), z, dtype=torch.uint8, device=DEV)
    out = canary_out(m, n)
    bsr.w4a16_group_gemv(x.to(torch.bfloat16), wp, scale, out, zero=zt)
    want = (-1.5 * d[:, -1, 0, -1].double()).cpu().numpy()
    got = bf16_bits_to_f64(host(out))
    assert np.array_equal(got, np.broadcast_to(want, got.shape)), np.abs(got - want).max()

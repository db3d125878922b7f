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


def _powers(m, n, k, group, exponent, scale_exponent, zero):
    """x = +-2^exponent, codes 0 .. 15, scales 2^scale_exponent and a zero point per group: y = sum of +-(c - z), a
    whole number under 2^24, times 2^(exponent + scale_exponent)."""
    g = torch.Generator(DEV).manual_seed(k + n + m)
    cols = 1 if group == 0 else k // group
    sign = 2 * torch.randint(0, 2, (m, k), device=DEV, generator=g) - 1
    codes = torch.randint(0, 16, (n, k // 2, 2), device=DEV, generator=g)
    z = torch.randint(0, 256, (n, cols), device=DEV, generator=g) if zero else torch.full((n, cols), 8, device=DEV)
    d = codes.reshape(n, k) - z.repeat_interleave(k // cols, dim=1)
    y = (sign.double() @ d.double().T) * 2.0 ** (exponent + scale_exponent)
    assert float(d.abs().sum(1).max()) < 1 << 24
    x = torch.ldexp(sign.float(), torch.tensor(exponent, device=DEV)).to(torch.bfloat16)
    scale = torch.full((n, cols), 2.0 ** scale_exponent, device=DEV)
    wp = (codes[..., 0] | codes[..., 1] << 4).to(torch.uint8)
    return x, wp, scale, z.to(torch.uint8) if zero else None, y


@pytest.mark.parametrize("m, n, k", [(1, 100, 160), (4, 64, 1056), (9, 33, 4096), (16, 40, 14336), (16, 8200, 256)])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("exponent, scale_exponent", [(126, -126), (-126, 126), (0, -120)])
def test_activations_of_any_finite_size(m, n, k, group, zero, exponent, scale_exponent):
    """The offset sums x * (16 + c) and (16 + z) * x of activations near BF16's largest value would pass binary32's,
    while the result is a small number; those near its smallest normal value, and results near it, are not lost."""
    if group and k % group:
        pytest.skip("the group does not divide K")
    say("exponent", m, n, k, group, zero, exponent, scale_exponent)
    x, wp, scale, zt, y = _powers(m, n, k, group, exponent, scale_exponent, zero)
    out = canary_out(m, n)
    bsr.w4a16_group_gemv(x, wp, scale, out, zero=zt)
    want = y.to(torch.bfloat16).view(torch.int16)  # (through binary32, which holds it exactly)
    got = torch.from_numpy(host(out).view(np.int16)).to(DEV)
    bad = (got.view(torch.bfloat16) != want.view(torch.bfloat16)).sum().item()
    assert bad == 0, f"{bad} of {m * n} differ"


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("m", [3, 16])
def test_rows_without_finite_activations_stay_among_themselves(m, group):
    """A row of infinities or NaN leaves the other rows of its tile as they are without it."""
    g = torch.Generator(DEV).manual_seed(m)
    n, k = 200, 704
    x = torch.randn((m, k), device=DEV, generator=g).bfloat16()
    wp = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV, generator=g)
    s = torch.rand((n, k // group if group else 1), device=DEV, generator=g)
    off = torch.tensor([0, 1, m], dtype=torch.int32, device=DEV)
    outs = []
    for bad in (0.0, float("inf"), float("nan"), -float("inf")):
        x[1] = bad
        x[m - 1, ::7] = bad
        out, by_expert = canary_out(m, n), canary_out(m, n // 2)
        bsr.w4a16_group_gemv(x, wp, s, out)
        bsr.w4a16_group_gemv_experts(x, torch.stack((wp, wp)), torch.stack((s, s)), off, by_expert, silu_mul=True)
        outs.append((host(out), host(by_expert)))
    keep = [r for r in range(m) if r not in (1, m - 1)]
    for a, b in outs[1:]:
        assert np.array_equal(a[keep], outs[0][0][keep]) and np.array_equal(b[keep], outs[0][1][keep])
        assert not np.isfinite(bf16_bits_to_f64(a[1])).any()

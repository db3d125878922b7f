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


@pytest.mark.parametrize("m, n, k, group", [
    (m, n, k, group) for m, n, k in [(1, 100, 160), (4, 64, 1056), (9, 33, 4096), (16, 40, 14336), (16, 8200, 256)]
    for group in (0, 32, 64, 128) if group == 0 or k % group == 0])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("exponent, scale_exponent", [(126, -126), (-126, 126), (0, -120)])
def test_activations_of_any_finite_size(m, n, k, group, zero, exponent, scale_exponent):
    """The offset sums x * (16 + c) and (16 + z) * x of activations near BF16's largest value would pass binary32's,
    while the result is a small number; those near its smallest normal value, and results near it, are not lost."""
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


# ---- whole numbers: a lost block, or another group's scale, changes the bits ----

def whole_case(rng, lead, m, n, k, group, zero):
    """Activations -4 .. 4, codes 0 .. 15, scales +-2^-2 .. 1 and zero points: (x, w_packed, scale, zero, codes)."""
    cols = 1 if group == 0 else k // group
    x = rng.integers(1, 5, (m, k)) * rng.choice([-1, 1], (m, k))
    codes = rng.integers(0, 16, (*lead, n, k))
    scale = 2.0 ** rng.integers(-2, 1, (*lead, n, cols)) * rng.choice([-1, 1], (*lead, n, cols))
    z = rng.integers(0, 256 if zero == "any" else 16, (*lead, n, cols)) if zero else None
    return x, (codes[..., ::2] | codes[..., 1::2] << 4).astype(np.uint8), scale, z, codes


def whole_product(x, codes, scale, z, skip=()):
    """sum over the 32-blocks of K (but those of `skip`) of x * scale * (c - z), exact in binary32 in any order: the
    terms are multiples of 2^-2 whose magnitudes add up to less than 2^22, as do the partial sums of the codes."""
    k = codes.shape[-1]
    rep = k // scale.shape[-1]
    d = codes - (8 if z is None else np.repeat(z, rep, axis=-1))
    keep = np.ones(k, dtype=bool)
    for b in skip:
        keep[32 * b:32 * b + 32] = False
    s = np.repeat(scale, rep, axis=-1)
    y = 0.0
    t = 0.0
    step = min(rep, 128)  # the kernel's unit: a group, or 128 elements of a row's scale
    for lo in range(0, k, step):
        part = (x[:, lo:lo + step] * keep[lo:lo + step]) @ (d[:, lo:lo + step] * s[:, lo:lo + step]).T
        y, t = y + part, t + np.abs(part)
    assert t.max() < 1 << 22 and np.abs(x).max() * 128 * 271 < 1 << 24
    return y


def bf16_rne(y):
    f = np.ascontiguousarray(y, dtype=np.float32)
    assert np.array_equal(f.astype(np.float64), y), "not exact in binary32"
    u = f.view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + (u >> 16 & 1)) >> 16).astype(np.uint16)


def same_values(bits, want):
    """Equal BF16 numbers (a sum of exactly 0 may have either sign)."""
    return np.array_equal(bf16_bits_to_f64(bits), bf16_bits_to_f64(want))


WHOLE = [  # m, n, k, group, zero points
    # tiles of up to 4 rows, of 16, and two column tiles a workgroup; chunks cut short, waves with one chunk and many
    (1, 33, 32, 32, None), (3, 50, 96, 32, "any"), (4, 40, 1056, 32, "4 bit"), (2, 30, 14336, 32, "any"),
    (1, 1000, 192, 64, "any"), (4, 64, 4160, 64, None), (3, 4000, 1024, 64, "4 bit"), (2, 50, 14336, 64, "any"),
    (1, 20, 128, 128, "4 bit"), (4, 300, 1408, 128, "any"), (3, 70, 14336, 128, None),
    (3, 4000, 1056, 0, "4 bit"), (2, 50, 14336, 0, "any"), (1, 130, 8192, 0, None), (4, 17, 32, 0, "any"),
    (16, 40, 14336, 32, "any"), (5, 33, 1056, 32, None), (17, 100, 96, 32, "4 bit"), (16, 48, 14336, 64, None),
    (9, 500, 448, 64, "any"), (16, 64, 14336, 128, "any"), (40, 30, 640, 128, "4 bit"), (16, 50, 14336, 0, "any"),
    (7, 300, 4128, 0, None), (33, 20, 96, 0, "4 bit"), (5, 8200, 160, 32, "any"), (16, 8193, 192, 64, None),
    (12, 8225, 384, 128, "4 bit"), (16, 8200, 288, 0, "any")]


@pytest.mark.parametrize("m, n, k, group, zero", WHOLE)
def test_whole_numbers(m, n, k, group, zero):
    say("whole", m, n, k, group, zero)
    rng = np.random.default_rng(m * 3 + n + k + group)
    x, wp, scale, z, codes = whole_case(rng, (), m, n, k, group, zero)
    want = bf16_rne(whole_product(x, codes, scale, z))
    xb = torch.from_numpy(x).to(torch.bfloat16).to(DEV)
    zt = None if z is None else to_dev(z.astype(np.uint8))
    for kind in (torch.float32, torch.float16, torch.bfloat16):
        out = canary_out(m, n)
        bsr.w4a16_group_gemv(xb, to_dev(wp), torch.from_numpy(scale).to(kind).to(DEV), out, zero=zt)
        assert same_values(host(out), want), kind


@pytest.mark.parametrize("counts, n, k, group, zero", [
    ([1, 0, 3], 100, 14336, 0, "any"), ([2, 1, 0, 1], 66, 14336, 64, None), ([0, 5, 1, 40], 34, 1056, 32, "any"),
    ([16, 0, 16], 48, 14336, 128, "4 bit"), ([9, 30, 1], 2000, 416, 0, "4 bit"), ([1] * 70, 64, 384, 128, "any")])
@pytest.mark.parametrize("gather", [False, True])
def test_whole_numbers_by_expert(counts, n, k, group, zero, gather):
    say("whole by expert", counts, n, k, group, zero, gather)
    rng = np.random.default_rng(n + k + group)
    experts, rows = len(counts), sum(counts)
    x, wp, scale, z, codes = whole_case(rng, (experts,), rows, n, k, group, zero)
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    index = rng.integers(0, rows, rows).astype(np.int32) if gather else None
    xr = x[index] if gather else x
    args = (torch.from_numpy(x).to(torch.bfloat16).to(DEV), to_dev(wp), to_dev(scale.astype(np.float32)), to_dev(off))
    how = dict(zero=None if z is None else to_dev(z.astype(np.uint8)), row_index=None if index is None else to_dev(index))
    out = canary_out(rows, n)
    bsr.w4a16_group_gemv_experts(*args, out, **how)
    # the SiLU product of the same sums, with scales that keep the gates within the exponential's reach
    small = 2.0 ** -9
    pair = canary_out(rows, n // 2)
    bsr.w4a16_group_gemv_experts(args[0], args[1], args[2] * small, args[3], pair, silu_mul=True, **how)
    got, got_pair = host(out), bf16_bits_to_f64(host(pair))
    for e in range(experts):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        y = whole_product(xr[lo:hi], codes[e], scale[e], None if z is None else z[e])
        assert same_values(got[lo:hi], bf16_rne(y)), e
        gate, up = y[:, :n // 2] * small, y[:, n // 2:] * small
        ref = gate / (1 + np.exp(-gate)) * up
        # gate and up are exact; the exponential is off by 2 steps of 2^-24 at most and its argument not at all, 1 + e,
        # the quotient and the product by half a step each, the output by half a step of 2^-7, below 2^-126 (an
        # exponential past binary32's range) by all of it
        assert (np.abs(got_pair[lo:hi] - ref) <= (2.0 ** -8 + 8 * 2.0 ** -24) * np.abs(ref) + 2.0 ** -100).all()

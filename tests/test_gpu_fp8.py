"""FP8 products on the GPU against the 64-bit oracle: dense and grouped by expert, the
SiLU product, values that are not finite, offsets outside the rows, whole numbers bit
for bit."""
import numpy as np
import pytest
import torch

from block_scaled_precision_requant_amd import bsr
from gpu_util import CANARY, DEV, canary_out, host, largest_products, say, to_dev
from oracle import fp8, moe
from oracle.compare import bf16_bits_to_f64, bf16_ulp, check_bf16

pytestmark = pytest.mark.gpu


def codes(rng, *shape):
    """E4M3 codes over all finite values."""
    c = rng.integers(0, 127, shape).astype(np.uint8)
    return c | (rng.integers(0, 2, shape).astype(np.uint8) << 7)


def scales(rng, *shape):
    return (rng.uniform(0.5, 2.0, shape) * 2.0 ** rng.integers(-12, -4, shape)).astype(np.float32)


def blocks(n):
    return -(-n // 128)


def product(a, w):
    """(y, T) of operands given as values, T so that fp8.terms of its steps bound the error: with the matrix core's cut."""
    y, t = fp8.product(a, w)
    return y, t + fp8.CUT * 2.0 ** 24 / (fp8.terms(a.shape[1]) + 2) * largest_products(a, w)


def run_dense(a, w, a_s, w_s):
    m, n = len(a), len(w)
    # (the rows around the output show what is written outside it)
    around = canary_out(m + 2, n)
    out = around[1:m + 1]
    bsr.fp8_gemm_blockscaled(to_dev(a), to_dev(w), to_dev(a_s), to_dev(w_s), out)
    got = host(around)
    assert (got[0] == CANARY).all() and (got[-1] == CANARY).all()
    return got[1:-1].view(np.uint16)


DENSE = [  # one row to many, one block to past 64 of them, columns off every tile
    (1, 1, 128), (1, 128, 128), (1, 4096, 256), (2, 130, 14336), (3, 33, 256), (4, 65, 8320), (5, 40, 128), (16, 64, 384),
    (17, 257, 640), (32, 48, 1152), (33, 96, 1152), (63, 640, 128), (64, 200, 1024), (65, 129, 256), (100, 300, 512),
    (128, 128, 8320), (129, 257, 384), (255, 1000, 512), (300, 130, 16640), (1000, 77, 256), (1025, 513, 384)]
SHAPES = [  # one size for each shape of tile, a few rows and columns short of whole ones (test_fp8_choices.py)
    (13, 4090, 640), (15, 8190, 384), (9, 16380, 640), (16, 28670, 128), (30, 4090, 640), (27, 8188, 384), (32, 16381, 640),
    (31, 28671, 256), (61, 4090, 640), (127, 4093, 384), (255, 4091, 640), (63, 28669, 256), (510, 4090, 384),
    (1021, 4093, 640), (2045, 4089, 384), (4091, 4090, 640), (2501, 8190, 256)]


@pytest.mark.parametrize("m, n, k", DENSE + SHAPES)
def test_dense(m, n, k):
    say("fp8", m, n, k)
    rng = np.random.default_rng(m * 7919 + n * 31 + k)
    a, w = codes(rng, m, k), codes(rng, n, k)
    a_s, w_s = scales(rng, m, k // 128), scales(rng, blocks(n), k // 128)
    got = run_dense(a, w, a_s, w_s)
    y, t = product(fp8.values_a(a, a_s), fp8.values_w(w, w_s))
    res = check_bf16(got, y, t, k, fp8.terms(k))
    say(f"  {res}")
    assert res.ok, str(res)
    assert np.array_equal(got, run_dense(a, w, a_s, w_s)), "equal calls give equal bits"


@pytest.mark.parametrize("m, n, k", [(1, 160, 512), (16, 33, 1280), (64, 128, 256), (130, 130, 1280), (40, 300, 8448)] + SHAPES)
def test_dense_whole_numbers(m, n, k):
    """Small whole codes and scales of powers of two: every partial sum is exact, so the result is the BF16 nearest to
    it, bit for bit -- a block, row or column that is left out or taken twice shows at once."""
    say("fp8 whole", m, n, k)
    rng = np.random.default_rng(m + n + k)
    small = fp8.e4m3_nearest(np.arange(-4.0, 5.0))
    a, w = small[rng.integers(0, 9, (m, k))], small[rng.integers(0, 9, (n, k))]
    a_s = (2.0 ** rng.integers(-2, 3, (m, k // 128))).astype(np.float32)
    w_s = (2.0 ** rng.integers(-2, 3, (blocks(n), k // 128))).astype(np.float32)
    y, _ = fp8.product(fp8.values_a(a, a_s), fp8.values_w(w, w_s))
    want = torch.from_numpy(y.astype(np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)
    got = run_dense(a, w, a_s, w_s)
    assert np.array_equal(got & 0x7FFF | (got & 0x8000) * (got & 0x7FFF != 0),
                          want & 0x7FFF | (want & 0x8000) * (want & 0x7FFF != 0))


@pytest.mark.parametrize("m, n, k", [(3, 200, 384), (40, 300, 512), (300, 400, 384)] + [(m, n, 384) for m, n, _ in SHAPES])
def test_not_finite_stays_in_its_place(m, n, k):
    say("fp8 nan", m, n, k)
    rng = np.random.default_rng(5)
    a, w = codes(rng, m, k), codes(rng, n, k)
    a_s, w_s = scales(rng, m, k // 128), scales(rng, blocks(n), k // 128)
    clean = run_dense(a, w, a_s, w_s)
    bad_row, bad_col, bad_block = m - 2, n // 2, blocks(n) - 1
    a[bad_row, k - 1] = 0x7F
    a_s[0, 1] = np.inf
    w[bad_col, 5] = 0xFF
    w_s[bad_block, 0] = np.nan
    got = run_dense(a, w, a_s, w_s)
    touched = np.zeros((m, n), dtype=bool)
    touched[[0, bad_row]] = True
    touched[:, bad_col] = True
    touched[:, 128 * bad_block:] = True
    assert np.array_equal(got[~touched], clean[~touched])
    assert not np.isfinite(bf16_bits_to_f64(got[:, bad_col])).any()
    assert not np.isfinite(bf16_bits_to_f64(got[[0, bad_row]])).any()
    assert not np.isfinite(bf16_bits_to_f64(got[:, 128 * bad_block:])).any()


def test_out_of_any_alignment_and_views():
    """An output two bytes off, operands inside larger buffers, float8 tensors."""
    rng = np.random.default_rng(9)
    for m, n, k in ((5, 64, 256), (150, 260, 256)):
        a, w = codes(rng, m + 1, k), codes(rng, n + 3, k)
        a_s, w_s = scales(rng, m + 1, k // 128), scales(rng, blocks(n), k // 128)
        flat = canary_out(1, m * n + 2)[0]
        out = flat[1:-1].view(m, n)
        bsr.fp8_gemm_blockscaled(to_dev(a)[1:].view(torch.float8_e4m3fn), to_dev(w)[2:-1], to_dev(a_s)[1:], to_dev(w_s), out)
        y, t = product(fp8.values_a(a[1:], a_s[1:]), fp8.values_w(w[2:-1], w_s))
        res = check_bf16(host(out).view(np.uint16), y, t, k, fp8.terms(k))
        assert res.ok, str(res)
        assert int(flat[0]) == CANARY and int(flat[-1]) == CANARY


# ---- grouped ------------------------------------------------------------------

def counts(kind, experts, rows, rng):
    """Rows of each expert: `rows` in all, or fewer."""
    if kind == "even":
        return np.full(experts, rows // experts)
    if kind == "one":
        c = np.zeros(experts, dtype=int)
        c[experts // 2] = rows
        return c
    cuts = np.sort(rng.integers(0, rows + 1, experts - 1)) if experts > 1 else np.array([], dtype=int)
    c = np.diff(np.concatenate(([0], cuts, [rows])))
    if kind == "holes":
        c[rng.random(experts) < 0.4] = 0
    return c


def run_grouped(a, w, a_s, w_s, offsets, index, rows, silu):
    n = w.shape[1]
    out = canary_out(rows, n // 2 if silu else n)
    bsr.fp8_grouped_gemm_blockscaled(to_dev(a), to_dev(w), to_dev(a_s), to_dev(w_s), to_dev(offsets.astype(np.int32)), out,
                                     row_index=None if index is None else to_dev(index.astype(np.int32)), silu_mul=silu)
    return host(out).view(np.uint16)


def check_grouped(got, a, w, a_s, w_s, offsets, index, rows, silu, k):
    y, t, covered = fp8.grouped(fp8.values_a(a, a_s), w, w_s, offsets, index, rows, product)
    assert (got[~covered] == CANARY).all(), "a row outside the offsets was written"
    if not covered.any():
        return
    if not silu:
        res = check_bf16(got[covered], y[covered], t[covered], k, fp8.terms(k))
        say(f"  {res}")
        assert res.ok, str(res)
        return
    want, bound = moe.silu_mul(y[covered], t[covered], fp8.terms(k))
    out = bf16_bits_to_f64(got[covered])
    err = np.abs(out - want)
    # the nearest BF16 is half a step away, a step where the bound crosses a power of two
    assert (err <= bound + bf16_ulp(np.abs(want) + bound) + 2.0 ** -133).all(), np.max(err - bound)


GROUPED = [  # rows, experts, n, k, counts
    (1, 1, 256, 128, "even"), (1, 4, 40, 128, "one"), (8, 64, 256, 256, "random"), (15, 3, 33, 384, "random"),
    (16, 1, 256, 128, "even"), (17, 1, 130, 256, "even"), (40, 5, 64, 512, "holes"), (64, 2, 768, 1024, "random"),
    (100, 3, 129, 384, "random"), (130, 4, 256, 2176, "one"), (200, 200, 48, 256, "even"), (300, 6, 512, 512, "holes"),
    (515, 2, 384, 768, "random"), (1000, 8, 256, 256, "random"), (1100, 3, 300, 384, "one"), (2600, 4, 768, 384, "random"),
    (700, 2, 4096, 256, "random"), (5000, 70, 130, 128, "holes"), (5000, 3, 5120, 256, "random")]
GROUPED += [(m, 1, 256 * (n // 256 + 1), k, "even") for m, n, k in SHAPES] + [(m, 3, n, k, "random") for m, n, k in SHAPES[4:]]


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("rows, experts, n, k, kind", GROUPED)
def test_grouped(rows, experts, n, k, kind, gather, silu):
    if silu and n % 256:
        n = 256 * blocks(n)
    say("fp8 grouped", rows, experts, n, k, kind, gather, silu)
    rng = np.random.default_rng(rows * 101 + experts * 7 + n + k)
    a_rows = max(1, rows // 3) if gather else rows
    a, w = codes(rng, a_rows, k), codes(rng, experts, n, k)
    # (gates of a few units, so that the SiLU's bend is inside)
    a_s, w_s = scales(rng, a_rows, k // 128), scales(rng, experts, blocks(n), k // 128)
    a_s *= np.float32(2.0 ** -7)
    offsets = np.concatenate(([0], np.cumsum(counts(kind, experts, rows, rng))))
    index = None
    if gather:
        index = rng.integers(0, a_rows, rows)
        index[rng.random(rows) < 0.1] = -1
        index[rng.random(rows) < 0.05] = a_rows
    got = run_grouped(a, w, a_s, w_s, offsets, index, rows, silu)
    check_grouped(got, a, w, a_s, w_s, offsets, index, rows, silu, k)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("part", [2, 4, 16])
@pytest.mark.parametrize("size, height", zip(SHAPES[8:], (64, 64, 64, 64, 128, 128, 256, 256, 128)))
def test_last_rows_of_an_expert(size, height, part, silu):
    """Fewer rows used than there is room for: the last tile of one expert holds a half, a quarter, a sixteenth of its
    rows."""
    m, n, k = size
    say("fp8 last rows", m, n, k, part, silu)
    n = 256 * (n // 256 + 1)
    rng = np.random.default_rng(m + n + part)
    used = (m - 1) // height * height + height // part - 1
    used = used if used <= m else used - height
    a, w = codes(rng, m, k), codes(rng, 1, n, k)
    a_s, w_s = scales(rng, m, k // 128) * np.float32(2.0 ** -7), scales(rng, 1, n // 128, k // 128)
    index = rng.permutation(m)
    for idx in (None, index):
        got = run_grouped(a, w, a_s, w_s, np.array([0, used]), idx, m, silu)
        check_grouped(got, a, w, a_s, w_s, np.array([0, used]), idx, m, silu, k)


@pytest.mark.parametrize("offsets", [
    [0, 0, 0, 0, 0], [5, 5, 9, 9, 12], [-3, 4, 4, 100, 7], [40, 3, 3, 2, 1], [0, 300, 300, 300, 300], [2, 290, 1, 1, 1],
    [-(2 ** 31), 2 ** 31 - 1, 0, 0, 0]])
@pytest.mark.parametrize("rows", [12, 300])
def test_offsets_outside_the_rows(offsets, rows):
    say("fp8 offsets", offsets, rows)
    rng = np.random.default_rng(rows)
    n, k = 160, 256
    a, w = codes(rng, rows, k), codes(rng, 4, n, k)
    a_s, w_s = scales(rng, rows, 2), scales(rng, 4, 2, 2)
    got = run_grouped(a, w, a_s, w_s, np.array(offsets), None, rows, False)
    check_grouped(got, a, w, a_s, w_s, np.array(offsets), None, rows, False, k)


@pytest.mark.parametrize("shape", [(4, 128, 128), (16, 384, 256)])
def test_data_gradient_on_the_transposed_weight(shape):
    """d_x = d_y @ W on the transposed codes and scales is the product with W's own values."""
    experts, n, k = shape
    rng = np.random.default_rng(3)
    w_bf = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).bfloat16().to(DEV)
    new = lambda *s, dt=torch.uint8: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
    q, qt = new(experts, n, k), new(experts, k, n)
    s, st = new(experts, n // 128, k // 128, dt=torch.float32), new(experts, k // 128, n // 128, dt=torch.float32)
    bsr.quantize_w_fp8(w_bf, q, s, w_qt=qt, w_scale_t=st)
    rows = 50
    d, d_s = codes(rng, rows, n), scales(rng, rows, n // 128)
    offsets = np.concatenate(([0], np.cumsum(counts("random", experts, rows, rng))))
    out = canary_out(rows, k)
    bsr.fp8_grouped_gemm_blockscaled(to_dev(d), qt, to_dev(d_s), st, to_dev(offsets.astype(np.int32)), out)
    got = host(out).view(np.uint16)
    d64, qh, sh = fp8.values_a(d, d_s), q.cpu().numpy(), s.cpu().numpy()
    for e in range(experts):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            v = fp8.values_w(qh[e], sh[e])
            res = check_bf16(got[lo:hi], *product(d64[lo:hi], np.ascontiguousarray(v.T)), n, fp8.terms(n))
            assert res.ok, str(res)


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("scale", [0.25, 2.0 ** -6, 2.0 ** -20, 2.0 ** 30])
def test_silu_over_its_range(rows, scale):
    """Gates of every code of both signs times `scale` (up to 112, and far past it), exact in binary32, ups of the row's
    own scale; streamed rows and tiles."""
    n, k = 512, 128
    w = np.zeros((1, n, k), np.uint8)
    w[0, :128, 0] = np.minimum(np.arange(128), 126)      # gates, two blocks of them
    w[0, 128:256, 0] = w[0, :128, 0] | 0x80
    w[0, 256:, 0] = 0x38                                 # ups: 1
    w_s = np.array([scale, scale, 1, 1], np.float32).reshape(1, 4, 1)
    a = np.zeros((rows, k), np.uint8)
    a[:, 0] = 0x38
    a_s = (2.0 ** -(np.arange(rows) % 5)).astype(np.float32)[:, None]
    got = run_grouped(a, w, a_s, w_s, np.array([0, rows]), None, rows, True)
    got = torch.from_numpy(got.view(np.int16)).view(torch.bfloat16).double().numpy()
    g = a_s.astype(np.float64) * np.concatenate((fp8.E4M3[w[0, :128, 0]], fp8.E4M3[w[0, 128:256, 0]])) * scale
    y = g / (1 + np.exp(-np.clip(g, -700, 700))) * a_s
    # the kernel's own steps, one rounding to BF16 (half of eps 2^-7) and half its smallest step; below -88.7 exp(-gate) is past binary32
    # and the result 0, which leaves out less than 89 * 2^-128
    tol = np.abs(y) * ((1.25 * np.abs(g) + 8) * 2.0 ** -24 + 2.0 ** -8 * (1 + 2.0 ** -9)) + 2.0 ** -134
    tol[g < -88.7] = 89 * 2.0 ** -128
    assert np.isfinite(got).all()
    bad = np.argwhere(~(np.abs(got - y) <= tol))
    assert not len(bad), [(g[i, j], got[i, j], y[i, j]) for i, j in bad[:4]]
    assert np.array_equal(np.signbit(got)[g != 0], np.signbit(g)[g != 0])  # (a sum of zeros of both signs is +0)


@pytest.mark.parametrize("rows", [3, 40])
def test_silu_of_subnormal_gates(rows):
    """Gates of every code times 2^-140, whole steps of binary32's smallest, and ups large enough that the product is an
    ordinary BF16: the quotient is the nearest step."""
    n, k = 512, 128
    w = np.zeros((1, n, k), np.uint8)
    w[0, :128, 0] = np.minimum(np.arange(128), 126)
    w[0, 128:256, 0] = w[0, :128, 0] | 0x80
    w[0, 256:, 0] = 0x38                                 # 1
    w_s = np.array([2.0 ** -70, 2.0 ** -70, 2.0 ** 127, 2.0 ** 127], np.float32).reshape(1, 4, 1)
    a = np.zeros((rows, k), np.uint8)
    a[:, 0] = 0x38
    a_s = np.full((rows, 1), 2.0 ** -70, np.float32)
    got = run_grouped(a, w, a_s, w_s, np.array([0, rows]), None, rows, True)
    got = torch.from_numpy(got.view(np.int16)).view(torch.bfloat16).double().numpy()
    g, up = np.concatenate((fp8.E4M3[w[0, :128, 0]], fp8.E4M3[w[0, 128:256, 0]])) * 2.0 ** -140, 2.0 ** 57
    y = g / (1 + np.exp(-g)) * up
    # the quotient's rounding is half a step of 2^-149 there (past it by less than the 2^-20 of what it rounds); then the
    # kernel's own steps and one rounding to BF16, as in test_silu_over_its_range
    tol = up * 2.0 ** -150 * (1 + 2.0 ** -20) + np.abs(y) * (8 * 2.0 ** -24 + 2.0 ** -8 * (1 + 2.0 ** -9))
    bad = np.argwhere(~(np.abs(got - y) <= tol))
    assert not len(bad), [(g[j] * 2.0 ** 149, got[i, j] / up * 2.0 ** 149) for i, j in bad[:4]]


def test_dense_equals_one_expert():
    rng = np.random.default_rng(11)
    for m, n, k in ((7, 256, 384), (600, 512, 256)):
        a, w = codes(rng, m, k), codes(rng, 1, n, k)
        a_s, w_s = scales(rng, m, k // 128), scales(rng, 1, n // 128, k // 128)
        one = run_grouped(a, w, a_s, w_s, np.array([0, m]), None, m, False)
        check_grouped(one, a, w, a_s, w_s, np.array([0, m]), None, m, False, k)

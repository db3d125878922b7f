"""Expert-layer operators on the GPU against the 64-bit oracle: the router, the
products grouped by expert, the 4-bit group GEMV (dense and by expert), the
weighted sum, and the layer they make together."""
import numpy as np
import pytest
import torch

import oracle
from block_scaled_precision_requant_amd import bsr, inputs
from gpu_util import CANARY, DEV, canary_out, host, say, to_dev
from oracle import moe
from oracle.compare import bf16_bits_to_f64, bf16_ulp, check_bf16

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LEFT = -77  # what int32 outputs are filled with before a call


# ---- router -------------------------------------------------------------------

def _route(logits, top_k, score=bsr.SCORE_SOFTMAX, renorm=True, scale=1.0, ws=None):
    t, e = logits.shape
    full = lambda *s: torch.full(s, LEFT, dtype=torch.int32, device=DEV)  # noqa: E731
    ids, pos, offsets, row_token = full(t, top_k), full(t, top_k), full(e + 1), full(t * top_k)
    weights = torch.full((t, top_k), float("nan"), dtype=torch.float32, device=DEV)
    need = bsr.moe_route_ws_bytes(t, e, top_k)
    if ws is None and need:
        ws = torch.full((need // 4,), -1, dtype=torch.int32, device=DEV)
    bsr.moe_route(logits, ids, weights, offsets, row_token, pos, ws, score=score, renorm=renorm, scale=scale)
    return ids, weights, offsets, row_token, pos


def _check_route(logits, top_k, score, renorm, scale):
    got = [x.cpu().numpy() for x in _route(logits, top_k, score, renorm, scale)]
    x = logits.double().cpu().numpy()
    ids, w, off, tok, pos = moe.route(x, top_k, score == bsr.SCORE_SIGMOID, renorm, scale)
    assert np.array_equal(got[0], ids) and np.array_equal(got[2], off) and np.array_equal(got[4], pos)
    assert np.array_equal(got[3][:len(tok)], tok)
    assert (got[3][len(tok):] == LEFT).all()
    # Roundings relative to a weight: the distance to the maximum (its own rounding moves the exponential by
    # |distance| * 2^-24, in the numerator and in the sum), the exponential's and the sum's (2 ulp each, at most 10 + 16
    # additions), a division, 1 + e, and the factor.
    fin = np.where(np.isfinite(x), x, 0.0)
    d = 2 * np.abs(fin).max(initial=0.0)
    err = np.abs(got[1] - w)
    assert (err <= (2 * d + 44) * 2.0 ** -24 * np.abs(w) + 2.0 ** -120).all(), err.max()


@pytest.mark.parametrize("tokens, experts, top_k", [
    (1, 1, 1), (1, 64, 8), (3, 7, 7), (31, 65, 3), (32, 128, 6), (33, 16, 16), (64, 8, 2), (257, 256, 8), (700, 300, 5),
    (130, 1000, 16), (5000, 1024, 1), (8200, 33, 4), (9001, 64, 8)])
@pytest.mark.parametrize("kind, score, renorm, scale", [
    ("f32", bsr.SCORE_SOFTMAX, True, 1.0), ("bf16", bsr.SCORE_SOFTMAX, False, 0.5),
    ("f16", bsr.SCORE_SIGMOID, True, 2.5), ("bf16", bsr.SCORE_SIGMOID, False, 1.0)])
def test_route(tokens, experts, top_k, kind, score, renorm, scale):
    say("route", tokens, experts, top_k, kind, score, renorm)
    g = torch.Generator().manual_seed(tokens * 1031 + experts)
    x = 2 * torch.randn(tokens, experts, generator=g)
    x[torch.rand(tokens, generator=g) < 0.1] = -np.inf          # padded tokens
    x[torch.rand(tokens, experts, generator=g) < 0.05] = -np.inf
    x = torch.where(torch.rand(tokens, experts, generator=g) < 0.3, x.round(), x)  # ties
    _check_route(x.to(TYPES[kind]).to(DEV), top_k, score, renorm, scale)


@pytest.mark.parametrize("score", [bsr.SCORE_SOFTMAX, bsr.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_special_values(score, renorm):
    """Infinities, NaN, both zeros, the type's lowest value, rows of one value, far apart and far negative logits."""
    inf, nan, low = np.inf, np.nan, float(np.finfo(np.float32).min)
    rows = [[0.0, -0.0, 0.0, -0.0, 0.0, -0.0], [nan] * 6, [-inf] * 6, [nan, 1.0, -inf, 1.0, nan, 0.0],
            [inf, 0.0, inf, 1.0, -inf, inf], [low, low, -inf, low, low, low], [-200.0, -201.0, -199.5, -300.0, low, -inf],
            [88.0, 87.0, -88.0, 0.0, 1e-30, -1e-30], [100.0, 3e38, -3e38, 0.0, 0.0, 0.0], [-inf, -inf, -inf, -inf, -inf, -90.0]]
    x = torch.tensor(rows, dtype=torch.float32, device=DEV)
    got = [y.cpu().numpy() for y in _route(x, 4, score, renorm)]
    ids, w, off, tok, pos = moe.route(x.cpu().numpy(), 4, score == bsr.SCORE_SIGMOID, renorm)
    assert np.array_equal(got[0], ids) and np.array_equal(got[2], off) and np.array_equal(got[4], pos)
    assert np.array_equal(got[3][:len(tok)], tok) and (got[3][len(tok):] == LEFT).all()
    # logits here are small whole or half numbers or out of the exponential's reach, so distances round exactly;
    # below 2^-120 binary32's exponential underflows
    assert np.isfinite(got[1]).all()
    assert (np.abs(got[1] - w) <= 44 * 2.0 ** -24 * w + 2.0 ** -120).all(), (got[1], w)


def test_route_no_tokens_and_strided_rows():
    offsets = _route(torch.zeros((0, 9), device=DEV), 2)[2]
    assert offsets.tolist() == [0] * 10
    wide = torch.randn(777, 50, device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    for lo in (0, 1, 6):  # rows 50 elements apart, off any wider alignment
        _check_route(wide[:, lo:lo + 37], 5, bsr.SCORE_SOFTMAX, True, 1.0)
        _check_route(wide.bfloat16()[:, lo:lo + 37], 5, bsr.SCORE_SOFTMAX, True, 1.0)


# ---- grouped products ---------------------------------------------------------

def _counts(kind, experts, rows, rng):
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


def _int8_operands(rng, shape_a, shape_w):
    k = shape_a[-1]
    a = rng.integers(-127, 128, shape_a).astype(np.int8)
    w = rng.integers(-127, 128, shape_w).astype(np.int8)
    a_s = (rng.uniform(0.5, 2.0, (*shape_a[:-1], k // 32)) * 2.0 ** -8).astype(np.float32)
    w_s = (rng.uniform(0.5, 2.0, (*shape_w[:-1], k // 32)) * 2.0 ** -10).astype(np.float32)
    return a, w, a_s, w_s


def _check_rows(got, y, t, covered, terms=None, k=32):
    assert (got[~covered] == CANARY).all(), "a row outside the offsets was written"
    if covered.any():
        res = check_bf16(got[covered], y[covered], t[covered], k, terms)
        say(f"  {res}")
        assert res.ok, str(res)


GROUPED = [  # rows, experts, n, k, counts
    (1, 1, 1, 32, "even"), (1, 4, 40, 64, "one"), (8, 64, 96, 256, "random"), (15, 3, 33, 96, "random"),
    (16, 1, 64, 128, "even"), (17, 1, 130, 160, "even"), (40, 5, 64, 512, "holes"), (64, 2, 200, 1024, "random"),
    (100, 3, 129, 288, "random"), (130, 4, 256, 2080, "one"), (200, 200, 48, 256, "even"), (300, 6, 260, 512, "holes"),
    (515, 2, 384, 768, "random"), (1000, 8, 128, 256, "random"), (1100, 3, 300, 320, "one"),
    (2600, 4, 640, 384, "random"), (700, 2, 4096, 256, "random"), (4100, 3, 1100, 128, "random"),
    (48, 1, 4096, 256, "even"), (3000, 1, 1000, 544, "even"), (5000, 70, 130, 64, "holes")]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("rows, experts, n, k, kind", GROUPED)
def test_grouped(rows, experts, n, k, kind, gather):
    say("grouped", rows, experts, n, k, kind, gather)
    rng = np.random.default_rng(rows * 7 + n * 3 + k + gather)
    cap = rows + (5 if rows % 2 else 0)                # rows behind the last expert's
    first = 2 if cap > rows else 0                     # and before the first one's
    offsets = (first + np.concatenate(([0], np.cumsum(_counts(kind, experts, rows, rng))))).astype(np.int32)
    a_rows = max(1, rows // 3) if gather else cap
    a, w, a_s, w_s = _int8_operands(rng, (a_rows, k), (experts, n, k))
    index = None
    if gather:
        index = rng.integers(0, a_rows, cap).astype(np.int32)
        index[rng.random(cap) < 0.05] = rng.choice([-1, a_rows, -2 ** 31, 2 ** 31 - 1])
    out = canary_out(cap, n)
    bsr.int8_grouped_gemm_blockscaled(to_dev(a), to_dev(w), to_dev(a_s), to_dev(w_s), to_dev(offsets), out,
                                      row_index=None if index is None else to_dev(index))
    y, t, covered = moe.grouped(a, w, a_s, w_s, offsets, index, cap)
    _check_rows(host(out), y, t, covered, k=k)


@pytest.mark.parametrize("rows", [5, 300])
@pytest.mark.parametrize("offsets", [
    [0, 0, 0, 0], [-5, 2, 3, 4], [4, 2, 3, 5], [0, 3, 3, 10 ** 6], [-2 ** 31, 0, 2 ** 31 - 1, 0], [2 ** 31 - 1] * 4])
def test_grouped_offsets_outside_the_rows(offsets, rows):
    """Offsets are device values: whatever they hold, rows outside the clamped ranges stay as they were."""
    say("offsets", offsets, rows)
    rng = np.random.default_rng(11)
    n, k, experts = 72, 128, 3
    a, w, a_s, w_s = _int8_operands(rng, (rows, k), (experts, n, k))
    off = np.array(offsets, dtype=np.int32)
    out = canary_out(rows, n)
    bsr.int8_grouped_gemm_blockscaled(to_dev(a), to_dev(w), to_dev(a_s), to_dev(w_s), to_dev(off), out)
    y, t, covered = moe.grouped(a, w, a_s, w_s, off, None, rows)
    _check_rows(host(out), y, t, covered, k=k)
    wp, sc = rng.integers(0, 256, (experts, n, k // 2)).astype(np.uint8), rng.uniform(0.5, 1, (experts, n, 4)).astype(np.float32)
    x = inputs.bf16_normal(rng, rows, k)
    out = canary_out(rows, n)
    bsr.w4a16_group_gemv_experts(to_dev(x.view(np.int16)), to_dev(wp), to_dev(sc), to_dev(off), out)
    y, t, covered = moe.w4_experts(moe.bf16_f64(x), wp, sc, None, off, None, rows)
    _check_rows(host(out), y, t, covered, terms=moe.w4_terms(k, 32))


# ---- 4-bit weights ------------------------------------------------------------

def _w4(rng, lead, n, k, group, kind, zero):
    g = k if group == 0 else group
    wp = rng.integers(0, 256, (*lead, n, k // 2)).astype(np.uint8)
    s = torch.from_numpy(rng.uniform(0.5, 1.5, (*lead, n, k // g)) * rng.choice([-0.01, 0.01], (*lead, n, k // g)))
    s = s.to(TYPES[kind])
    z = rng.integers(0, 256 if zero == "any" else 16, (*lead, n, k // g)).astype(np.uint8) if zero else None
    return wp, s, z


W4 = [  # m, n, k, group, scale type, zero points
    (1, 1, 32, 32, "f32", None), (1, 17, 64, 0, "bf16", "4 bit"), (2, 33, 96, 32, "f16", "any"),
    (3, 64, 128, 64, "bf16", None), (1, 130, 128, 128, "f32", "4 bit"), (5, 100, 160, 32, "bf16", "any"),
    (16, 48, 192, 64, "f16", "4 bit"), (17, 70, 256, 128, "bf16", "any"), (1, 300, 512, 0, "f32", None),
    (4, 512, 4096, 128, "bf16", "4 bit"), (8, 96, 1056, 32, "f16", None), (16, 256, 2048, 32, "f32", "4 bit"),
    (9, 4096, 256, 64, "bf16", "4 bit"), (40, 80, 640, 128, "f16", None), (1, 14336, 384, 128, "bf16", "4 bit"),
    (16, 1000, 14336, 32, "f16", None), (2, 50, 14336, 0, "bf16", "any"), (7, 333, 4480, 64, "f32", "any"),
    (1, 4096, 6144, 128, "f16", "4 bit"), (33, 65, 96, 0, "f16", None),
    # two column tiles a workgroup, the last one of 1 or 8 columns; one column, chunks cut short
    (5, 8200, 160, 32, "bf16", "any"), (16, 8193, 96, 32, "f16", None), (12, 8225, 448, 64, "f32", "4 bit"),
    # the most LDS a workgroup takes: 16 waves of 4 rows
    (4, 4096, 14336, 128, "bf16", None), (3, 4000, 8192, 0, "f16", "4 bit"),
    (1, 1, 1440, 32, "f32", "4 bit"), (16, 1, 288, 32, "bf16", "any"), (4, 17, 704, 64, "f16", "any")]


@pytest.mark.parametrize("m, n, k, group, kind, zero", W4)
def test_w4_group(m, n, k, group, kind, zero):
    say("w4", m, n, k, group, kind, zero)
    rng = np.random.default_rng(m * 5 + n + k)
    wp, s, z = _w4(rng, (), n, k, group, kind, zero)
    x = inputs.bf16_normal(rng, m, k)
    out = canary_out(m, n)
    bsr.w4a16_group_gemv(to_dev(x.view(np.int16)), to_dev(wp), s.to(DEV), out, zero=None if z is None else to_dev(z))
    y, t = moe.w4_group(moe.bf16_f64(x), wp, s.double().numpy(), z)
    _check_rows(host(out), y, t, np.ones(m, dtype=bool), terms=moe.w4_terms(k, group))


W4E = [  # rows, experts, n, k, group, type, zero, counts
    (1, 3, 34, 64, 32, "bf16", "4 bit", "one"), (8, 64, 256, 512, 128, "f16", None, "random"),
    (20, 4, 130, 288, 32, "f32", "any", "holes"), (50, 2, 64, 1024, 64, "bf16", "4 bit", "random"),
    (35, 1, 96, 160, 0, "bf16", None, "even"), (200, 70, 48, 256, 64, "f16", "4 bit", "random"),
    (6, 6, 2048, 2048, 128, "bf16", "4 bit", "even")]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("rows, experts, n, k, group, kind, zero, counts", W4E)
def test_w4_experts(rows, experts, n, k, group, kind, zero, counts, silu, gather):
    say("w4 experts", rows, experts, n, k, group, kind, zero, counts, silu, gather)
    rng = np.random.default_rng(rows + n + k)
    cap = rows + 3
    offsets = (1 + np.concatenate(([0], np.cumsum(_counts(counts, experts, rows, rng))))).astype(np.int32)
    wp, s, z = _w4(rng, (experts,), n, k, group, kind, zero)
    x_rows = max(1, rows // 2) if gather else cap
    x = inputs.bf16_normal(rng, x_rows, k)
    if gather:
        x[0] = 0x7FC0  # a NaN row that no index names
    index = None
    if gather:
        index = rng.integers(min(1, x_rows - 1), x_rows, cap).astype(np.int32)
        index[rng.random(cap) < 0.1] = -1
        if x_rows == 1:
            x[0] = 0x3F80
    out = canary_out(cap, n // 2 if silu else n)
    bsr.w4a16_group_gemv_experts(to_dev(x.view(np.int16)), to_dev(wp), s.to(DEV), to_dev(offsets), out,
                                 zero=None if z is None else to_dev(z),
                                 row_index=None if index is None else to_dev(index), silu_mul=silu)
    xf = np.nan_to_num(moe.bf16_f64(x))
    y, t, covered = moe.w4_experts(xf, wp, s.double().numpy(), z, offsets, index, cap)
    terms = moe.w4_terms(k, group)
    if not silu:
        _check_rows(host(out), y, t, covered, terms=terms)
        return
    got = host(out)
    assert (got[~covered] == CANARY).all()
    ref, bound = moe.silu_mul(y, t, terms)
    v = bf16_bits_to_f64(got[covered])
    ref, bound = ref[covered], bound[covered]
    assert np.isfinite(v).all()
    assert (np.abs(v - ref) <= bound + 0.5 * bf16_ulp(np.abs(ref) + bound)).all()


def test_w4_silu_of_far_gates():
    """exp(-gate) overflows for a far negative gate (the product is 0) and vanishes for a far positive one."""
    k, half = 64, 3
    x = np.full((2, k), 0x3F80, dtype=np.uint16)          # 1.0; row 1: -1.0
    x[1] = 0xBF80
    wp = np.full((1, 2 * half, k // 2), 0x99, dtype=np.uint8)   # code 9: +1 with zero point 8
    s = np.array([[2.0], [100.0], [1e30], [1.0], [1.0], [1.0]], dtype=np.float32)[None]
    out = canary_out(2, half)
    bsr.w4a16_group_gemv_experts(to_dev(x.view(np.int16)), to_dev(wp), to_dev(s), to_dev(np.array([0, 2], dtype=np.int32)),
                                 out, silu_mul=True)
    v = bf16_bits_to_f64(host(out))
    gate, up = np.array([[128.0, 6400.0, 64e30]]) * [[1], [-1]], np.array([[64.0], [-64.0]])
    ref = np.where(gate > 0, gate * up, 0.0)
    assert (np.abs(v - ref) <= 2.0 ** -8 * np.abs(ref) + 64 * 128 * np.exp(-88.0)).all(), v


# ---- combine ------------------------------------------------------------------

@pytest.mark.parametrize("tokens, top_k, rows, n, residual, shift", [
    (1, 1, 1, 1, False, 0), (3, 8, 24, 4096, True, 0), (5, 2, 7, 33, True, 0), (40, 16, 640, 200, False, 0),
    (9, 3, 27, 2056, True, 0), (4, 4, 16, 64, True, 1), (4, 4, 16, 64, False, 3), (700, 6, 4200, 264, False, 0),
    (3, 2, 0, 40, True, 0)])
def test_combine(tokens, top_k, rows, n, residual, shift):
    say("combine", tokens, top_k, rows, n, residual, shift)
    rng = np.random.default_rng(tokens + n)

    def placed(x):  # the tensor `shift` elements off its buffer's alignment
        buf = torch.zeros(x.size + 8, dtype=torch.int16, device=DEV)
        buf[shift:shift + x.size] = to_dev(x.view(np.int16)).reshape(-1)
        return buf[shift:shift + x.size].reshape(x.shape)

    y, r = inputs.bf16_normal(rng, rows, n), inputs.bf16_normal(rng, tokens, n)
    pos = rng.integers(0, max(rows, 1), (tokens, top_k)).astype(np.int32)
    bad = rng.random(pos.shape) < 0.2
    pos[bad] = rng.choice(np.array([-1, rows, -2 ** 31, 2 ** 31 - 1], dtype=np.int32), int(bad.sum()))
    pos[0] = pos[0] if tokens == 1 else -1             # a token without experts
    if rows > 1:
        pos[(pos >= 0) & (pos < rows)] = np.maximum(pos[(pos >= 0) & (pos < rows)], 1)
        y[0] = 0x7FC0                                  # NaN in a row that no position names
    w = rng.uniform(-1, 1, pos.shape).astype(np.float32)
    out = canary_out(tokens, n)
    bsr.moe_combine(placed(y), to_dev(pos), to_dev(w), out, residual=placed(r) if residual else None)
    ref, t = moe.combine(np.nan_to_num(moe.bf16_f64(y)), pos, w, moe.bf16_f64(r) if residual else None)
    res = check_bf16(host(out), ref, t, 32, terms=top_k)  # one rounding per slot
    assert res.ok, str(res)
    if residual:  # in place
        rr = placed(r)
        bsr.moe_combine(placed(y), to_dev(pos), to_dev(w), rr, residual=rr)
        assert np.array_equal(host(rr), host(out))
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("rows, experts, n, k, kind", [
    # the GEMV of few rows per expert: tiles of 4 and of 16 rows, K split over 1 to 16 waves, chunks cut short
    (4, 2, 16, 32, "even"), (3, 9, 17, 224, "random"), (7, 7, 4096, 128, "random"), (8, 2, 300, 14336, "random"),
    (33, 2, 100, 4128, "random"), (90, 6, 130, 1120, "holes"), (64, 4, 128, 2048, "one"), (16, 16, 512, 4096, "holes"),
    (2, 2, 28672, 256, "even"), (140, 9, 72, 96, "random"), (1, 1, 1, 1440, "even"), (5, 1, 17, 416, "even"),
    (16, 1, 1, 160, "even")])
def test_grouped_few_rows(rows, experts, n, k, kind, gather):
    test_grouped(rows, experts, n, k, kind, gather)

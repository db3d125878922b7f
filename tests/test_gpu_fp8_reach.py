"""Parts of the FP8 products' kernels that only long rows, large operands or a second entry point reach: the weight's
scales read again every 64 blocks, tiles and streamed rows past 4 GiB, the dense and the grouped call on one weight.
test_fp8_reach.py holds which kernel each size runs."""
import numpy as np
import pytest
import torch

from block_scaled_precision_requant_amd import bsr
from gpu_util import CANARY, DEV, canary_out, host, largest_products, say, to_dev
from oracle import fp8, moe
from oracle.compare import bf16_bits_to_f64, bf16_ulp, check_bf16
from test_gpu_fp8 import DENSE, SHAPES, blocks, codes, scales

pytestmark = pytest.mark.gpu

GROUPS = (4, 4, 4, 4, 4, 4, 4, 3, 4, 4, 2, 1, 2, 1, 1, 1, 1)  # K groups of each shape, in the order of SHAPES
# a group takes more than 64 blocks, those with one group two times 64
LONG = [(m, n, 128 * ((64 if g > 1 else 128) * g + 3)) for (m, n, _), g in zip(SHAPES, GROUPS)]


@pytest.fixture(autouse=True)
def _release_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def whole(g, rows, k, low, high):
    """Codes of -4..4, scales of powers of two and the values, on the device."""
    small = torch.from_numpy(fp8.e4m3_nearest(np.arange(-4.0, 5.0))).to(DEV)
    pick = torch.randint(0, 9, (rows, k), generator=g, device=DEV)
    s = torch.exp2(torch.randint(low, high, (rows, k // 128), generator=g, device=DEV).float())
    return small[pick], s, pick.double() - 4


def exact_product(a, a_s, w, w_s):
    """(a * a_s) @ (w * w_s) and the sum of the terms' magnitudes, in 64 bits; w_s per 128 rows of w."""
    a = a * a_s.double().repeat_interleave(128, 1)
    w = w * w_s.double().repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)
    wt = w.t().contiguous()
    return a @ wt, a.abs() @ wt.abs()


@pytest.mark.parametrize("m, n, k", LONG)
def test_whole_numbers_past_64_blocks(m, n, k):
    """Every partial sum is exact in binary32 in any order, so the result is the nearest BF16: another block's scale shows
    at once.  Dense, and by expert with an expert that takes a part of a tile."""
    say("fp8 long", m, n, k)
    g = torch.Generator(DEV).manual_seed(m + n + k)
    a, a_s, av = whole(g, m, k, -2, 3)
    w, w_s, wv = whole(g, n, k, -2, 3)
    w_s = w_s[:blocks(n)].contiguous()
    y, t = exact_product(av, a_s, wv, w_s)
    assert float(t.max()) < 2.0 ** 20  # of whole 2^-4
    want = y.float().bfloat16()
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    bsr.fp8_gemm_blockscaled(a, w, a_s, w_s, out)
    assert torch.equal(out, want)
    out.fill_(float("nan"))
    bsr.fp8_grouped_gemm_blockscaled(a, w[None], a_s, w_s[None], torch.tensor([0, m], dtype=torch.int32, device=DEV), out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("m, n, k", LONG)
def test_silu_past_64_blocks(m, n, k):
    """The same with the SiLU product on rows picked by index: gate and up are exact, what is left is the kernel's own
    SiLU and one rounding."""
    n = 256 * (n // 256 + 1)
    say("fp8 long silu", m, n, k)
    g = torch.Generator(DEV).manual_seed(m + n + k)
    a, a_s, av = whole(g, m, k, -12, -7)
    w, w_s, wv = whole(g, n, k, -2, 3)
    w_s = w_s[:n // 128].contiguous()
    y, t = exact_product(av, a_s, wv, w_s)
    assert float(t.max()) < 2.0 ** 10  # of whole 2^-14
    pick = torch.randperm(m, generator=g, device=DEV).int()
    out = torch.full((m, n // 2), float("nan"), dtype=torch.bfloat16, device=DEV)
    bsr.fp8_grouped_gemm_blockscaled(a, w[None], a_s, w_s[None], torch.tensor([0, m], dtype=torch.int32, device=DEV), out,
                                     row_index=pick, silu_mul=True)
    y = y[pick.long()]
    gate, up = y[:, :n // 2], y[:, n // 2:]
    want = gate / (1 + torch.exp(-gate)) * up
    # (1.25 |gate| + 8) 2^-24 of it, half a BF16 step (2^-8) of what that leaves, half its smallest step
    tol = want.abs() * ((1.25 * gate.abs() + 8) * 2.0 ** -24 + 2.0 ** -8 * (1 + 2.0 ** -9)) + 2.0 ** -134
    far = gate < -88.7  # there exp(-gate) is past binary32 and the result 0
    tol[far] = 89 * 2.0 ** -128 * up.abs()[far]
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("m, n, k", DENSE + SHAPES)
def test_dense_is_one_expert(m, n, k):
    """The dense call and the grouped one on a single weight run the same kernel, with the same order of sums."""
    say("fp8 dense = one expert", m, n, k)
    rng = np.random.default_rng(m + 3 * n + k)
    a, w = to_dev(codes(rng, m, k)), to_dev(codes(rng, n, k))
    a_s, w_s = to_dev(scales(rng, m, k // 128)), to_dev(scales(rng, blocks(n), k // 128))
    dense, one, picked = (canary_out(m, n) for _ in range(3))
    off = torch.tensor([0, m], dtype=torch.int32, device=DEV)
    bsr.fp8_gemm_blockscaled(a, w, a_s, w_s, dense)
    bsr.fp8_grouped_gemm_blockscaled(a, w[None], a_s, w_s[None], off, one)
    bsr.fp8_grouped_gemm_blockscaled(a, w[None], a_s, w_s[None], off, picked,
                                     row_index=torch.arange(m, dtype=torch.int32, device=DEV))
    assert torch.equal(dense, one) and torch.equal(dense, picked)


# ---- past 32-bit offsets --------------------------------------------------------

def random_codes(g, *shape):
    return torch.randint(0, 127, shape, dtype=torch.uint8, device=DEV, generator=g)


def product(a, w):
    """(y, T) of operands given as values, T with the matrix core's cut (as in test_gpu_fp8.py)."""
    y, t = fp8.product(a, w)
    return y, t + fp8.CUT * 2.0 ** 24 / (fp8.terms(a.shape[1]) + 2) * largest_products(a, w)


EXPERTS, WIDE_N, WIDE_K = 40, 8192, 16384  # 5 GiB of codes
LAST = (300, 2000, 5000)                   # rows of the last expert: 64 x 128, 256 x 128 and 256 x 256 tiles


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("last", LAST)
def test_tiles_of_weights_past_4_gib(last, silu):
    n, k = WIDE_N, WIDE_K
    say("fp8 tiles past 4 GiB", last, silu)
    g = torch.Generator(DEV).manual_seed(1)
    w = random_codes(g, EXPERTS, n, k)
    w_s = torch.rand(EXPERTS, n // 128, k // 128, device=DEV, generator=g) * 2.0 ** -12
    rows = 3 + last
    a, a_s = random_codes(g, rows, k), torch.rand(rows, k // 128, device=DEV, generator=g) * 2.0 ** -8
    counts = torch.zeros(EXPERTS, dtype=torch.int32)
    counts[0], counts[-2], counts[-1] = 1, 2, last
    off = torch.cat((torch.zeros(1, dtype=torch.int32), counts.cumsum(0).int())).to(DEV)
    width = n // 2 if silu else n
    out = canary_out(rows, width)
    bsr.fp8_grouped_gemm_blockscaled(a, w, a_s, w_s, off, out, silu_mul=silu)
    cols = np.arange(width - 140, width)
    weight_rows = np.concatenate((cols, cols + width)) if silu else cols
    for e, picks in ((0, [0]), (EXPERTS - 2, [1, 2]), (EXPERTS - 1, [3, 4, rows - 1])):
        y, t = product(fp8.values_a(a[picks].cpu().numpy(), a_s[picks].cpu().numpy()),
                       fp8.values_w(w[e].cpu().numpy(), w_s[e].cpu().numpy())[weight_rows])
        got = host(out[picks][:, width - 140:].contiguous()).view(np.uint16)
        if silu:
            want, bound = moe.silu_mul(y, t, fp8.terms(k))
            assert (np.abs(bf16_bits_to_f64(got) - want) <= bound + bf16_ulp(np.abs(want) + bound)).all()
        else:
            res = check_bf16(got, y, t, k, fp8.terms(k))
            say(f"  expert {e}: {res}")
            assert res.ok, str(res)
    assert not (out == CANARY).all(1).any()


GATHER_ROWS, GATHER_PICKS = 262143, 4  # rows times 16384 just under 2^32 bytes; as many as are streamed


@pytest.mark.parametrize("silu", [False, True])
def test_streamed_gather_just_under_4_gib(silu):
    n, k, rows = 512, WIDE_K, GATHER_ROWS
    say("fp8 streamed gather", silu)
    g = torch.Generator(DEV).manual_seed(2)
    a, w = random_codes(g, rows, k), random_codes(g, 1, n, k)
    a_s, w_s = torch.rand(rows, k // 128, device=DEV, generator=g) * 2.0 ** -8, torch.rand(1, n // 128, k // 128, device=DEV, generator=g) * 2.0 ** -12
    for picks in ([rows - 1, -1, rows, 131072], [0, rows - 1, 131071, 2 ** 31 - 1]):
        assert len(picks) == GATHER_PICKS
        out = canary_out(GATHER_PICKS, n // 2 if silu else n)
        bsr.fp8_grouped_gemm_blockscaled(a, w, a_s, w_s, torch.tensor([0, GATHER_PICKS], dtype=torch.int32, device=DEV), out,
                                         row_index=torch.tensor(picks, dtype=torch.int32, device=DEV), silu_mul=silu)
        there = [i for i, p in enumerate(picks) if 0 <= p < rows]
        at = [picks[i] for i in there]
        y, t = product(fp8.values_a(a[at].cpu().numpy(), a_s[at].cpu().numpy()), fp8.values_w(w[0].cpu().numpy(), w_s[0].cpu().numpy()))
        got = host(out).view(np.uint16)
        if silu:
            want, bound = moe.silu_mul(y, t, fp8.terms(k))
            assert (np.abs(bf16_bits_to_f64(got[there]) - want) <= bound + bf16_ulp(np.abs(want) + bound)).all()
        else:
            res = check_bf16(got[there], y, t, k, fp8.terms(k))
            assert res.ok, str(res)
        assert not got[[i for i in range(GATHER_PICKS) if i not in there]].any()


def test_quantized_codes_past_4_gib():
    """Codes and transposed codes past 4 GiB: the last expert is as it is alone."""
    e, n, k = 17, 16384, 16384
    last = torch.randn(n, k, generator=torch.Generator(DEV).manual_seed(4), device=DEV).bfloat16()
    w = torch.zeros(e, n, k, dtype=torch.bfloat16, device=DEV)
    w[-1] = last
    new = lambda *s: torch.full(s, 0xA5, dtype=torch.uint8, device=DEV)  # noqa: E731
    q, qt, s, st = new(e, n, k), new(e, k, n), torch.empty(e, n // 128, k // 128, device=DEV), torch.empty(e, k // 128, n // 128, device=DEV)
    bsr.quantize_w_fp8(w, q, s, w_qt=qt, w_scale_t=st)
    q1, s1 = new(n, k), torch.empty(n // 128, k // 128, device=DEV)
    bsr.quantize_w_fp8(last, q1, s1)
    assert torch.equal(q[-1], q1) and torch.equal(s[-1], s1)
    assert torch.equal(qt[-1], q1.t()) and torch.equal(st[-1], s1.t())
    for v in (q, s, qt, st):
        assert not v[:-1].any()

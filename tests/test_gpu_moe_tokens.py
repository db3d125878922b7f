"""Rows copied into the experts' order, its gradient, and the gradient of the weighted
sum, on the GPU against the 64-bit oracle and against differences."""
import numpy as np
import pytest
import torch

from block_scaled_precision_requant_amd import bsr
from gpu_util import CANARY, DEV, canary_out, host, say, to_dev
from oracle import fp8, moe
from oracle.compare import bf16_ulp

pytestmark = pytest.mark.gpu

SIZES = [  # tokens, top_k, n
    (1, 1, 1), (1, 16, 8), (3, 2, 7), (5, 8, 64), (33, 3, 2047), (17, 6, 2048), (64, 4, 2049), (100, 8, 4095), (16, 8, 4096),
    (257, 1, 129), (9, 16, 8200), (2, 3, 14336), (4001, 8, 16)]


def positions(rng, tokens, top_k, rows):
    """Distinct rows, some slots without one: negative, or past the rows."""
    pos = rng.permutation(max(rows, tokens * top_k))[:tokens * top_k].reshape(tokens, top_k).astype(np.int32)
    pos[rng.random(pos.shape) < 0.1] = -1
    pos[rng.random(pos.shape) < 0.05] = -(2 ** 31)
    if tokens > 2:
        pos[1] = -1          # a padded token
    return pos               # (with fewer rows than slots the others lie past them)


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).bfloat16()


def raw(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("tokens, top_k, n", SIZES)
def test_dispatch(tokens, top_k, n, off):
    """off: rows that start two bytes off."""
    say("dispatch", tokens, top_k, n, off)
    rng = np.random.default_rng(tokens + top_k + n)
    rows = max(1, tokens * top_k - tokens // 3)
    pos = positions(rng, tokens, top_k, rows)
    x = torch.empty(tokens * n + off, dtype=torch.bfloat16, device=DEV)[off:].view(tokens, n)
    x.copy_(bf16(rng, tokens, n))
    flat = canary_out(1, rows * n + 2 + off)[0]
    out = flat[1 + off:-1].view(rows, n)
    bsr.moe_dispatch(x, to_dev(pos), out)
    want = fp8.dispatch(host(raw(x)), pos, np.full((rows, n), CANARY, np.uint16))
    assert np.array_equal(host(out), want)
    assert (host(flat)[:1 + off] == CANARY).all() and int(flat[-1]) == CANARY


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("tokens, top_k, n", SIZES)
def test_dispatch_grad(tokens, top_k, n, off):
    say("dispatch_grad", tokens, top_k, n, off)
    rng = np.random.default_rng(tokens * top_k + n)
    rows = max(1, tokens * top_k - tokens // 3)
    pos = positions(rng, tokens, top_k, rows)
    d = torch.empty(rows * n + off, dtype=torch.bfloat16, device=DEV)[off:].view(rows, n)
    d.copy_(bf16(rng, rows, n))
    flat = canary_out(1, tokens * n + 2 + off)[0]
    bsr.moe_dispatch_grad(d, to_dev(pos), flat[1 + off:-1].view(tokens, n))
    got = flat[1 + off:-1].view(torch.bfloat16).view(tokens, n).double().cpu().numpy()
    want, mag = fp8.dispatch_grad(d.double().cpu().numpy(), pos)
    # top_k - 1 roundings in binary32, then half a BF16 step of the sum that was rounded
    bound = (top_k - 1) * 2.0 ** -24 * mag
    assert (np.abs(got - want) <= bound + bf16_ulp(np.abs(want) + bound) / 2 * (1 + 2.0 ** -7)).all()
    assert (host(flat)[:1 + off] == CANARY).all() and int(flat[-1]) == CANARY


def run_combine_grad(d_out, y, pos, w, in_place=False):
    d_y = y if in_place else torch.full(y.shape, CANARY, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    d_w = torch.full(w.shape, float("nan"), device=DEV)
    bsr.moe_combine_grad(d_out, y, pos, w, d_y, d_w)
    return d_y, d_w


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("tokens, top_k, n", SIZES)
def test_combine_grad(tokens, top_k, n, off):
    say("combine_grad", tokens, top_k, n, off)
    rng = np.random.default_rng(tokens * 3 + top_k * n)
    rows = max(1, tokens * top_k - tokens // 3)
    pos = positions(rng, tokens, top_k, rows)
    y = torch.empty(rows * n + off, dtype=torch.bfloat16, device=DEV)[off:].view(rows, n)
    y.copy_(bf16(rng, rows, n))
    d_out = bf16(rng, tokens, n).to(DEV)
    w = torch.from_numpy(rng.uniform(-1, 2, (tokens, top_k)).astype(np.float32))
    d_y, d_w = run_combine_grad(d_out, y, to_dev(pos), w.to(DEV))
    want_y, want_w, mag = fp8.combine_grad(d_out.double().cpu().numpy(), y.double().cpu().numpy(), pos, w.numpy())
    named = ~np.isnan(want_y[:, 0])
    assert (host(raw(d_y))[~named] == CANARY).all()
    got = d_y.double().cpu().numpy()[named]
    # one product, rounded to binary32 and then to BF16
    assert (np.abs(got - want_y[named]) <= bf16_ulp(want_y[named]) / 2 * (1 + 2.0 ** -7)).all()
    # a BF16 product is exact in binary32 (8 bits times 8): n terms, n - 1 additions at most in any order
    assert (np.abs(d_w.double().cpu().numpy() - want_w) <= n * 2.0 ** -24 * mag).all()
    again, w_again = run_combine_grad(d_out, y.clone(), to_dev(pos), w.to(DEV), in_place=True)
    assert torch.equal(w_again, d_w) and torch.equal(raw(again)[torch.from_numpy(named)], raw(d_y)[torch.from_numpy(named)])


def test_combine_grad_against_differences():
    """d_weights and d_y are the slopes of sum(d_out * combine): on values whose sums are exact in BF16."""
    rng = np.random.default_rng(8)
    tokens, top_k, n = 6, 3, 24
    pos = rng.permutation(tokens * top_k).reshape(tokens, top_k).astype(np.int32)
    pos[4, 1] = -1
    y = torch.from_numpy(rng.integers(-3, 4, (tokens * top_k, n)).astype(np.float32)).bfloat16().to(DEV)
    d_out = torch.from_numpy(rng.integers(-3, 4, (tokens, n)).astype(np.float32)).bfloat16().to(DEV)
    w = torch.from_numpy(rng.integers(-2, 3, (tokens, top_k)).astype(np.float32)).to(DEV)
    p = to_dev(pos)

    def loss(y, w):
        out = torch.empty(tokens, n, dtype=torch.bfloat16, device=DEV)
        bsr.moe_combine(y, p, w, out)
        return float((out.double() * d_out.double()).sum())

    d_y, d_w = run_combine_grad(d_out, y, p, w)
    for t in range(tokens):
        for s in range(top_k):
            more, less = w.clone(), w.clone()
            more[t, s] += 1
            less[t, s] -= 1
            assert float(d_w[t, s]) == (loss(y, more) - loss(y, less)) / 2
    for r, j in rng.integers(0, (tokens * top_k, n), (40, 2)):
        if r not in pos:
            continue
        more, less = y.clone(), y.clone()
        more[r, j] += 1
        less[r, j] -= 1
        assert float(d_y[r, j]) == (loss(more, w) - loss(less, w)) / 2


def test_not_finite_and_subnormal():
    """NaN, infinities and subnormals pass through copies and sums as binary32 has them."""
    n = 16
    vals = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e-40, -0.0, 3.3e38, 1.0, -1e-40] * 2).bfloat16()
    x = torch.stack((vals, vals.flip(0))).to(DEV)
    pos = to_dev(np.array([[0, 2], [1, 3]], np.int32))
    out = torch.zeros(4, n, dtype=torch.bfloat16, device=DEV)
    bsr.moe_dispatch(x, pos, out)
    assert torch.equal(raw(out[[0, 2]]), raw(x[[0, 0]])) and torch.equal(raw(out[[1, 3]]), raw(x[[1, 1]]))
    d_x = torch.zeros(2, n, dtype=torch.bfloat16, device=DEV)
    bsr.moe_dispatch_grad(out, pos, d_x)
    want = (x.float() + x.float()).bfloat16()
    assert torch.equal(torch.isnan(d_x), torch.isnan(want)) and torch.equal(d_x[~torch.isnan(want)], want[~torch.isnan(want)])
    w = torch.tensor([[0.5, float("nan")], [float("inf"), 2.0 ** -120]], device=DEV)
    w[0, 1] = torch.tensor(0x7FFFFFFF, dtype=torch.int32).view(torch.float32)  # a NaN of all ones stays one
    d_y, d_w = run_combine_grad(x, out, pos, w)
    want = (w.t().reshape(-1, 1) * x.float()[[0, 1, 0, 1]]).bfloat16()
    assert torch.equal(torch.isnan(d_y), torch.isnan(want)) and torch.equal(d_y[~torch.isnan(want)], want[~torch.isnan(want)])
    assert torch.isnan(d_w).all()


def test_no_rows_and_no_columns():
    pos = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    empty = torch.empty(0, 8, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(3, 8, dtype=torch.bfloat16, device=DEV)
    bsr.moe_dispatch(x, pos, empty)
    d_x = torch.ones(3, 8, dtype=torch.bfloat16, device=DEV)
    bsr.moe_dispatch_grad(empty, pos, d_x)
    assert not d_x.any()
    w, d_w = torch.ones(3, 2, device=DEV), torch.ones(3, 2, device=DEV)
    bsr.moe_combine_grad(x, empty, pos, w, empty, d_w)
    assert not d_w.any()
    d_w.fill_(1)
    thin = torch.empty(6, 0, dtype=torch.bfloat16, device=DEV)
    bsr.moe_combine_grad(thin[:3], thin, pos, w, thin, d_w)
    assert not d_w.any()
    bsr.moe_dispatch(thin[:3], pos, thin)
    bsr.moe_dispatch_grad(thin, pos, thin[:3])


def test_past_4_gib():
    """Rows past 2^32 elements."""
    n, rows, tokens = 16384, 270000, 40
    pos = torch.arange(rows - 2 * tokens, rows, dtype=torch.int32, device=DEV).view(2, tokens).t().contiguous()
    g = torch.Generator(DEV).manual_seed(6)
    x = torch.randn(tokens, n, generator=g, device=DEV).bfloat16()
    big = torch.empty(rows, n, dtype=torch.bfloat16, device=DEV)
    small, near = torch.empty(2 * tokens, n, dtype=torch.bfloat16, device=DEV), pos - (rows - 2 * tokens)
    bsr.moe_dispatch(x, pos, big)
    assert torch.equal(big[-2 * tokens:].view(2, tokens, n), x.expand(2, tokens, n))
    small.copy_(torch.randn(2 * tokens, n, generator=g, device=DEV))
    big[-2 * tokens:] = small
    a, b = torch.empty_like(x), torch.empty_like(x)
    bsr.moe_dispatch_grad(big, pos, a)
    bsr.moe_dispatch_grad(small, near, b)
    assert torch.equal(a, b)
    w = torch.randn(tokens, 2, generator=g, device=DEV)
    d_big, w_big = torch.empty_like(w), torch.empty_like(w)
    d_small = torch.empty_like(small)
    bsr.moe_combine_grad(x, small, near, w, d_small, d_big)
    bsr.moe_combine_grad(x, big, pos, w, big, w_big)
    assert torch.equal(d_big, w_big) and torch.equal(big[-2 * tokens:], d_small)

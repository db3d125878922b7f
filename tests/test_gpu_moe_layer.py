"""The expert-layer operators together, as a layer runs them: every step of the
two layer paths against the oracle fed with the step before it, the layers in a
captured graph and on two streams, and operands and outputs past 4 GiB."""
import numpy as np
import pytest
import torch

import oracle
from block_scaled_precision_requant_amd import bsr, inputs
from gpu_util import DEV, canary_out, host, say, to_dev
from oracle import moe
from oracle.compare import bf16_bits_to_f64, bf16_ulp, check_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _release_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _bits(t):
    return host(t.view(torch.int16))


class _Layer:
    """Weights of one expert layer in both forms, and its inputs."""

    def __init__(self, seed, tokens, experts, top_k, hidden, inter, group=64):
        rng = np.random.default_rng(seed)
        self.dims = (tokens, experts, top_k, hidden, inter)
        self.rng = rng
        q = lambda n, k: [(rng.integers(-127, 128, (experts, n, k)).astype(np.int8)),  # noqa: E731
                          (rng.uniform(0.5, 2, (experts, n, k // 32)) * 2.0 ** -12).astype(np.float32)]
        self.w13, self.s13 = q(2 * inter, hidden)
        self.w2, self.s2 = q(hidden, inter)
        w4 = lambda n, k: [rng.integers(0, 256, (experts, n, k // 2)).astype(np.uint8),  # noqa: E731
                           (rng.uniform(0.5, 1.5, (experts, n, k // group)) * 0.02).astype(np.float32),
                           rng.integers(4, 12, (experts, n, k // group)).astype(np.uint8)]
        self.p13, self.ps13, self.z13 = w4(2 * inter, hidden)
        self.p2, self.ps2, self.z2 = w4(hidden, inter)
        self.i8 = [to_dev(x) for x in (self.w13, self.s13, self.w2, self.s2)]
        self.w4 = [to_dev(x) for x in (self.p13, self.ps13, self.z13, self.p2, self.ps2, self.z2)]
        self.scratch = bsr.MoeScratch(tokens, experts, top_k, hidden, inter)
        self.x = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=DEV)
        self.residual = torch.empty_like(self.x)
        self.logits = torch.empty((tokens, experts), dtype=torch.float32, device=DEV)
        self.new_inputs()

    def new_inputs(self):
        t, e, _, h, _ = self.dims
        self.x.view(torch.int16).copy_(to_dev(inputs.bf16_normal(self.rng, t, h).view(np.int16)))
        self.residual.view(torch.int16).copy_(to_dev(inputs.bf16_normal(self.rng, t, h).view(np.int16)))
        x = self.rng.standard_normal((t, e)).astype(np.float32)
        x[self.rng.random(t) < 0.2] = -np.inf  # padded tokens
        self.logits.copy_(to_dev(x))

    def prefill(self, out):
        bsr.moe_prefill(self.x, self.logits, *self.i8, out, self.scratch, residual=self.residual)

    def decode(self, out):
        bsr.moe_decode_w4(self.x, self.logits, *self.w4, out, self.scratch, residual=self.residual,
                          score=bsr.SCORE_SIGMOID, scale=2.0)

    def outs(self):
        t, _, _, h, _ = self.dims
        return [torch.full((t, h), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]


def _combined(layer, out, y_bits, sigmoid, scale):
    t, e, k, h, _ = layer.dims
    s = layer.scratch
    ids, w, off, tok, pos = moe.route(layer.logits.cpu().numpy(), k, sigmoid=sigmoid, scale=scale)
    assert np.array_equal(s.ids.cpu().numpy(), ids) and np.array_equal(s.pos.cpu().numpy(), pos)
    assert np.array_equal(s.offsets.cpu().numpy(), off) and np.array_equal(s.row_token.cpu().numpy()[:len(tok)], tok)
    got_w = s.weights.cpu().numpy()
    # |logits| < 6 here: (2 * 12 + 44) roundings as in the router's own test
    assert (np.abs(got_w - w) <= 68 * 2.0 ** -24 * w).all()
    ref, mag = moe.combine(bf16_bits_to_f64(y_bits), pos, got_w, bf16_bits_to_f64(_bits(layer.residual)))
    res = check_bf16(_bits(out), ref, mag, 32, terms=k)
    assert res.ok, str(res)
    return off, tok


@pytest.mark.parametrize("tokens, experts, top_k, hidden, inter", [(1, 16, 4, 256, 128), (37, 8, 2, 512, 384),
                                                                   (300, 12, 3, 384, 320)])
def test_prefill_layer_step_by_step(tokens, experts, top_k, hidden, inter):
    say("prefill layer", tokens, experts, top_k, hidden, inter)
    layer = _Layer(tokens, tokens, experts, top_k, hidden, inter)
    out = layer.outs()[0]
    layer.prefill(out)
    s = layer.scratch
    y_bits = _bits(s.y)
    off, tok = _combined(layer, out, y_bits, False, 1.0)
    rows = len(tok)
    qa, sa = oracle.requant_a(_bits(layer.x))
    y, t, cov = moe.grouped(qa, layer.w13, sa, layer.s13, off, tok, rows)
    assert cov.all() or rows == 0
    gu = _bits(s.gate_up)[:rows]
    res = check_bf16(gu, y, t, hidden)
    assert res.ok, str(res)
    qh, sh = oracle.silu_mul_requant(np.ascontiguousarray(gu[:, :inter]), np.ascontiguousarray(gu[:, inter:]))
    assert np.array_equal(s.h_i8.cpu().numpy()[:rows], qh) and np.array_equal(s.h_scale.cpu().numpy()[:rows], sh)
    y, t, _ = moe.grouped(qh, layer.w2, sh, layer.s2, off, None, rows)
    res = check_bf16(y_bits[:rows], y, t, inter)
    assert res.ok, str(res)


@pytest.mark.parametrize("tokens, experts, top_k, hidden, inter", [(1, 16, 4, 256, 128), (19, 8, 2, 512, 384)])
def test_decode_layer_step_by_step(tokens, experts, top_k, hidden, inter):
    say("decode layer", tokens, experts, top_k, hidden, inter)
    layer = _Layer(tokens + 7, tokens, experts, top_k, hidden, inter)
    out = layer.outs()[0]
    layer.decode(out)
    s = layer.scratch
    y_bits = _bits(s.y)
    off, tok = _combined(layer, out, y_bits, True, 2.0)
    rows = len(tok)
    y, t, _ = moe.w4_experts(bf16_bits_to_f64(_bits(layer.x)), layer.p13, layer.ps13, layer.z13, off, tok, rows)
    ref, bound = moe.silu_mul(y, t, moe.w4_terms(hidden, 64))
    h_bits = _bits(s.h)[:rows]
    assert (np.abs(bf16_bits_to_f64(h_bits) - ref) <= bound + 0.5 * bf16_ulp(np.abs(ref) + bound)).all()
    y, t, _ = moe.w4_experts(bf16_bits_to_f64(h_bits), layer.p2, layer.ps2, layer.z2, off, None, rows)
    res = check_bf16(y_bits[:rows], y, t, inter, terms=moe.w4_terms(inter, 64))
    assert res.ok, str(res)


def test_scratch_serves_fewer_tokens_and_refuses_more():
    layer = _Layer(3, 40, 8, 2, 256, 128)
    out = layer.outs()[0]
    layer.prefill(out)
    fewer, own = torch.empty_like(out[:7]), torch.empty_like(out[:7])
    for o, scratch in ((fewer, layer.scratch), (own, bsr.MoeScratch(7, 8, 2, 256, 128))):
        bsr.moe_prefill(layer.x[:7], layer.logits[:7], *layer.i8, o, scratch, residual=layer.residual[:7])
    assert torch.equal(fewer.view(torch.int16), own.view(torch.int16))
    for path in (lambda *a, **k: bsr.moe_prefill(*a[:2], *layer.i8, *a[2:], **k),
                 lambda *a, **k: bsr.moe_decode_w4(*a[:2], *layer.w4, *a[2:], **k)):  # no tokens at all
        path(layer.x[:0], layer.logits[:0], out[:0], layer.scratch, residual=layer.residual[:0])
        assert layer.scratch.offsets.tolist() == [0] * 9
    with pytest.raises(ValueError, match="41 tokens"):
        layer.scratch.route(torch.zeros((41, 8), device=DEV))


def test_layers_replay_in_graph():
    a, b = _Layer(5, 130, 16, 4, 512, 256), _Layer(6, 5, 64, 8, 512, 256)
    big = _Layer(8, 9000, 24, 2, 64, 64)  # the router's two launches, with its workspace
    outs = a.outs() + b.outs() + big.outs()

    def step():
        a.prefill(outs[0])
        a.decode(outs[1])
        b.prefill(outs[2])
        b.decode(outs[3])
        big.prefill(outs[4])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(4):
        for layer in (a, b, big):
            layer.new_inputs()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        step()
        torch.cuda.synchronize()
        for i in range(5):
            assert torch.equal(got[i].view(torch.int16), outs[i].view(torch.int16)), f"replay {rep}, output {i}"
        say(f"graph replay {rep} equal")


def test_layers_on_two_streams():
    layers = [_Layer(11, 200, 8, 2, 512, 256), _Layer(12, 260, 16, 4, 384, 128)]
    outs = [layer.outs() for layer in layers]
    torch.cuda.synchronize()
    alone = []
    for layer, o in zip(layers, outs):
        layer.prefill(o[0])
        layer.decode(o[1])
        torch.cuda.synchronize()
        alone.append([x.clone() for x in o])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        for o in outs:
            for x in o:
                x.zero_()
        torch.cuda.synchronize()
        for layer, o, s in zip(layers, outs, streams):
            with torch.cuda.stream(s):
                layer.prefill(o[0])
                layer.decode(o[1])
        torch.cuda.synchronize()
        for o, ref in zip(outs, alone):
            for x, y in zip(o, ref):
                assert torch.equal(x.view(torch.int16), y.view(torch.int16)), rep
    # and on a stream passed by argument
    bsr.moe_prefill(layers[0].x, layers[0].logits, *layers[0].i8, outs[0][0], layers[0].scratch,
                    residual=layers[0].residual, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(outs[0][0].view(torch.int16), alone[0][0].view(torch.int16))


# ---- past 32-bit offsets ----------------------------------------------------------

def test_grouped_weights_past_4_gib():
    """Weights and their scales start past 4 GiB for the last experts; every row of two of them against the oracle."""
    experts, n, k, rows = 40, 8192, 16384, 6
    g = torch.Generator(DEV).manual_seed(1)
    w = torch.randint(-127, 128, (experts, n, k), dtype=torch.int8, device=DEV, generator=g)
    w_s = torch.rand((experts, n, k // 32), device=DEV, generator=g) * 2.0 ** -12
    assert w.numel() > 1 << 32
    a = torch.randint(-127, 128, (rows, k), dtype=torch.int8, device=DEV, generator=g)
    a_s = torch.rand((rows, k // 32), device=DEV, generator=g) * 2.0 ** -8
    counts = torch.zeros(experts, dtype=torch.int32)
    counts[0], counts[-2], counts[-1] = 1, 2, 3
    off = torch.cat((torch.zeros(1, dtype=torch.int32), counts.cumsum(0).int())).to(DEV)
    out = canary_out(rows, n)
    bsr.int8_grouped_gemm_blockscaled(a, w, a_s, w_s, off, out)
    got = host(out)
    for e, lo, hi in ((0, 0, 1), (experts - 2, 1, 3), (experts - 1, 3, 6)):
        y, t, _ = moe.grouped(a[lo:hi].cpu().numpy(), w[e:e + 1].cpu().numpy(), a_s[lo:hi].cpu().numpy(),
                              w_s[e:e + 1].cpu().numpy(), np.array([0, hi - lo]), None, hi - lo)
        res = check_bf16(got[lo:hi], y, t, k)
        say(f"expert {e}: {res}")
        assert res.ok, str(res)


def test_w4_weights_past_4_gib():
    experts, n, k, rows = 80, 8192, 16384, 4
    g = torch.Generator(DEV).manual_seed(2)
    wp = torch.randint(0, 256, (experts, n, k // 2), dtype=torch.uint8, device=DEV, generator=g)
    assert wp.numel() > 1 << 32
    s = torch.rand((experts, n, k // 128), device=DEV, generator=g) * 0.02
    z = torch.randint(0, 16, (experts, n, k // 128), dtype=torch.uint8, device=DEV, generator=g)
    x = torch.randn((rows, k), device=DEV, generator=g).bfloat16()
    off = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    off[-2:] = torch.tensor([1, 4], dtype=torch.int32, device=DEV)  # expert E-2: one row, the last: three
    out = canary_out(rows, n)
    bsr.w4a16_group_gemv_experts(x, wp, s, off, out, zero=z)
    got, xf = host(out), x.double().cpu().numpy()
    for e, lo, hi in ((experts - 2, 0, 1), (experts - 1, 1, 4)):
        y, t = moe.w4_group(xf[lo:hi], wp[e].cpu().numpy(), s[e].cpu().numpy(), z[e].cpu().numpy())
        res = check_bf16(got[lo:hi], y, t, k, terms=moe.w4_terms(k, 128))
        assert res.ok, str(res)


def test_outputs_past_4_gib():
    """More than 2^32 output elements of the grouped product, and a weighted sum that reads them."""
    rows, n, k, experts = 70000, 65536, 32, 3
    g = torch.Generator(DEV).manual_seed(3)
    a = torch.randint(-127, 128, (rows, k), dtype=torch.int8, device=DEV, generator=g)
    w = torch.randint(-127, 128, (experts, n, k), dtype=torch.int8, device=DEV, generator=g)
    a_s = torch.rand((rows, 1), device=DEV, generator=g) * 2.0 ** -8
    w_s = torch.rand((experts, n, 1), device=DEV, generator=g) * 2.0 ** -10
    off = torch.tensor([0, 100, 65530, rows], dtype=torch.int32, device=DEV)
    out = torch.full((rows, n), 0x7FA5, dtype=torch.int16, device=DEV)
    assert out.numel() > 1 << 32
    bsr.int8_grouped_gemm_blockscaled(a, w, a_s, w_s, off, out)
    picks = np.array([0, 99, 100, 32767, 65529, 65530, 65535, 65536, rows - 1])
    at = torch.from_numpy(picks).to(DEV)
    expert = np.array([0, 0, 1, 1, 1, 2, 2, 2, 2])
    got = host(out[at])
    for e in range(experts):
        sel = expert == e
        y, t, _ = moe.grouped(a[at].cpu().numpy()[sel], w[e:e + 1].cpu().numpy(), a_s[at].cpu().numpy()[sel],
                              w_s[e:e + 1].cpu().numpy(), np.array([0, sel.sum()]), None, int(sel.sum()))
        res = check_bf16(got[sel], y, t, k)
        assert res.ok, str(res)
    pos = torch.tensor([[rows - 1, 65536], [0, -1], [65535, 100]], dtype=torch.int32, device=DEV)
    weights = torch.tensor([[0.5, 0.25], [1.5, 3.0], [-1.0, 2.0]], device=DEV)
    res_out = canary_out(3, n)
    bsr.moe_combine(out, pos, weights, res_out)
    bits = {int(p): bf16_bits_to_f64(host(out[int(p)])) for p in (rows - 1, 65536, 0, 65535, 100)}
    y = np.stack([0.5 * bits[rows - 1] + 0.25 * bits[65536], 1.5 * bits[0], -bits[65535] + 2 * bits[100]])
    t = np.stack([0.5 * abs(bits[rows - 1]) + 0.25 * abs(bits[65536]), 1.5 * abs(bits[0]),
                  abs(bits[65535]) + 2 * abs(bits[100])])
    res = check_bf16(host(res_out), y, t, 32, terms=2)
    assert res.ok, str(res)


def test_route_of_many_tokens():
    """Millions of tokens: runs of thousands of tokens per workgroup, against stable sorts."""
    t, e, k = 3_000_001, 8, 2
    g = torch.Generator(DEV).manual_seed(4)
    x = torch.randn((t, e), device=DEV, generator=g)
    full = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)  # noqa: E731
    ids, pos, offsets, row_token = full(t, k), full(t, k), full(e + 1), full(t * k)
    weights = torch.empty((t, k), device=DEV)
    ws = torch.empty(bsr.moe_route_ws_bytes(t, e, k), dtype=torch.uint8, device=DEV)
    bsr.moe_route(x, ids, weights, offsets, row_token, pos, ws)
    want = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), want)
    flat = want.reshape(-1)
    src = torch.sort(flat, stable=True).indices
    assert torch.equal(row_token.long(), src // k)
    assert torch.equal(pos.reshape(-1)[src].long(), torch.arange(t * k, device=DEV))
    assert torch.equal(offsets[1:].long(), torch.bincount(flat, minlength=e).cumsum(0)) and int(offsets[0]) == 0

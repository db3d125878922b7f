"""The FP8 operators together, as a layer runs them: the forward path step by step against the oracle fed with the step
before it, a training step with every gradient against 64 bits, captured graphs, two streams, operands past 4 GiB."""
import numpy as np
import pytest
import torch

import oracle
from block_scaled_precision_requant_amd import bsr
from gpu_util import CANARY, DEV, canary_out, host, largest_products, say, to_dev
from oracle import fp8, moe
from oracle.compare import bf16_bits_to_f64, bf16_ulp, check_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _release_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def product(a, w):
    """(y, T) of operands given as values, T with the matrix core's cut (as in test_gpu_fp8.py)."""
    y, t = fp8.product(a, w)
    return y, t + fp8.CUT * 2.0 ** 24 / (fp8.terms(a.shape[1]) + 2) * largest_products(a, w)


def bits(t):
    return host(t.view(torch.int16))


class Layer:
    """One expert layer: weights quantized here, with their transposes, and inputs."""

    def __init__(self, seed, tokens, experts, top_k, hidden, inter):
        self.dims = (tokens, experts, top_k, hidden, inter)
        self.g = torch.Generator(DEV).manual_seed(seed)
        self.w13 = self._weight(experts, 2 * inter, hidden)
        self.w2 = self._weight(experts, hidden, inter)
        self.scratch = bsr.MoeScratch(tokens, experts, top_k, hidden, inter)
        self.x = torch.empty(tokens, hidden, dtype=torch.bfloat16, device=DEV)
        self.residual, self.d_out = torch.empty_like(self.x), torch.empty_like(self.x)
        self.logits = torch.empty(tokens, experts, device=DEV)
        self.new_inputs()

    def _weight(self, e, n, k):
        """(codes, scales, codes transposed, scales transposed)."""
        w = (torch.randn(e, n, k, generator=self.g, device=DEV) / k ** 0.5).bfloat16()
        new = lambda *s, dt=torch.float8_e4m3fn: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
        q, s = new(e, n, k), new(e, n // 128, k // 128, dt=torch.float32)
        qt, st = new(e, k, n), new(e, k // 128, n // 128, dt=torch.float32)
        bsr.quantize_w_fp8(w, q, s, w_qt=qt, w_scale_t=st)
        return q, s, qt, st

    def new_inputs(self):
        t, e = self.logits.shape
        r = lambda *s: torch.randn(*s, generator=self.g, device=DEV)  # noqa: E731
        for v in (self.x, self.residual, self.d_out):
            v.copy_(r(*v.shape))
        self.logits.copy_(r(t, e))
        self.logits[torch.rand(t, generator=self.g, device=DEV) < 0.2] = -np.inf  # padded tokens

    def forward(self, out):
        bsr.moe_prefill_fp8(self.x, self.logits, *self.w13[:2], *self.w2[:2], out, self.scratch, residual=self.residual)


@pytest.mark.parametrize("tokens, experts, top_k, hidden, inter", [
    (1, 16, 4, 256, 128), (3, 4, 2, 128, 256), (37, 8, 2, 512, 384), (300, 12, 3, 384, 640), (900, 3, 2, 256, 1024)])
def test_layer_step_by_step(tokens, experts, top_k, hidden, inter):
    say("fp8 layer", tokens, experts, top_k, hidden, inter)
    layer = Layer(tokens, tokens, experts, top_k, hidden, inter)
    s = layer.scratch
    for b in (s.h, s.y):  # what lies behind the last row is not read
        b.fill_(float("nan"))
    out = torch.full((tokens, hidden), float("nan"), dtype=torch.bfloat16, device=DEV)
    layer.forward(out)
    ids, w, off, tok, pos = moe.route(layer.logits.cpu().numpy(), top_k)
    assert np.array_equal(s.offsets.cpu().numpy(), off) and np.array_equal(s.pos.cpu().numpy(), pos)
    rows = len(tok)
    xq, xs = oracle.quant_act(bits(layer.x), 128, e4m3=True)
    assert np.array_equal(s.a_i8.cpu().numpy().view(np.uint8), xq)
    q13, s13 = (v.cpu() for v in layer.w13[:2])
    q2, s2 = (v.cpu() for v in layer.w2[:2])
    y, t, _ = fp8.grouped(fp8.values_a(xq, xs), q13.view(torch.uint8).numpy(), s13.numpy(), off, tok, rows, product)
    ref, bound = moe.silu_mul(y, t, fp8.terms(hidden))
    h = bits(s.h)[:rows]
    assert (np.abs(bf16_bits_to_f64(h) - ref) <= bound + bf16_ulp(np.abs(ref) + bound)).all()
    hq, hs = oracle.quant_act(h, 128, e4m3=True) if rows else (np.zeros((0, inter), np.uint8), np.zeros((0, inter // 128), np.float32))
    y, t, _ = fp8.grouped(fp8.values_a(hq, hs), q2.view(torch.uint8).numpy(), s2.numpy(), off, None, rows, product)
    yb = bits(s.y)
    if rows:
        res = check_bf16(yb[:rows], y, t, inter, fp8.terms(inter))
        say(f"  {res}")
        assert res.ok, str(res)
    ref, mag = moe.combine(bf16_bits_to_f64(yb), pos, s.weights.cpu().numpy(), bf16_bits_to_f64(bits(layer.residual)))
    res = check_bf16(bits(out), ref, mag, 32, terms=top_k)
    assert res.ok, str(res)


def quantized(x):
    """E4M3 codes and scales of BF16 rows, by the library."""
    q = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    s = torch.empty(x.shape[0], x.shape[1] // 128, device=DEV)
    bsr.quantize_act(x.contiguous(), q, s, group=128, fmt=bsr.FMT_E4M3)
    return q, s


class Step:
    """A training step of the layer (weights as they are): forward with what the gradients need kept, then the gradients
    of the input, of the routing weights and of each projection's rows."""

    def __init__(self, layer):
        t, e, k, h, i = layer.dims
        new = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
        self.layer, r = layer, t * k
        self.rows_x, self.gate_up, self.y, self.out = new(r, h), new(r, 2 * i), new(r, h), new(t, h)
        self.d_y, self.d_w, self.d_h, self.d_rows, self.d_x = new(r, h), new(t, k, dt=torch.float32), new(r, i), new(r, h), new(t, h)
        self.d_gate_up = None

    def run(self):
        m, s = self.layer, self.layer.scratch
        i = m.dims[4]
        s.route(m.logits)
        # forward: rows copied into the experts' order, since the step keeps them
        bsr.moe_dispatch(m.x, s.pos, self.rows_x)
        xq, xs = quantized(self.rows_x)
        bsr.fp8_grouped_gemm_blockscaled(xq, m.w13[0], xs, m.w13[1], s.offsets, self.gate_up)
        gate, up = self.gate_up[:, :i].float(), self.gate_up[:, i:].float()
        sig = torch.sigmoid(gate)
        self.h = (gate * sig * up).bfloat16()
        hq, hs = quantized(self.h)
        bsr.fp8_grouped_gemm_blockscaled(hq, m.w2[0], hs, m.w2[1], s.offsets, self.y)
        bsr.moe_combine(self.y, s.pos, s.weights, self.out, residual=m.residual)
        # backward
        bsr.moe_combine_grad(m.d_out, self.y, s.pos, s.weights, self.d_y, self.d_w)
        dq, ds = quantized(self.d_y)
        bsr.fp8_grouped_gemm_blockscaled(dq, m.w2[2], ds, m.w2[3], s.offsets, self.d_h)
        d_h = self.d_h.float()
        self.d_gate_up = torch.cat((d_h * up * sig * (1 + gate * (1 - sig)), d_h * gate * sig), 1).bfloat16()
        gq, gs = quantized(self.d_gate_up)
        bsr.fp8_grouped_gemm_blockscaled(gq, m.w13[2], gs, m.w13[3], s.offsets, self.d_rows)
        bsr.moe_dispatch_grad(self.d_rows, s.pos, self.d_x)

    def results(self):
        return [self.out, self.d_x, self.d_w, self.d_y, self.d_h]


def _dequantized(q, s):
    return q.double() * s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)


@pytest.mark.parametrize("tokens, experts, top_k, hidden, inter", [(6, 4, 2, 256, 128), (150, 6, 3, 384, 256)])
def test_training_step_gradients(tokens, experts, top_k, hidden, inter):
    """Gradients of sum(out * d_out) against autograd of the formulas in 64 bits, on the dequantized weights: what
    differs is the rounding of each step's rows to FP8 and BF16, bounded from what each step was given."""
    say("training step", tokens, experts, top_k, hidden, inter)
    layer = Layer(tokens + 1, tokens, experts, top_k, hidden, inter)
    step = Step(layer)
    step.run()
    s = layer.scratch
    pos, off = s.pos.long(), s.offsets.tolist()
    w13, w2 = _dequantized(*layer.w13[:2]), _dequantized(*layer.w2[:2])
    x, wt = layer.x.double().requires_grad_(), s.weights.double().requires_grad_()
    live = pos >= 0
    token = torch.arange(tokens, device=DEV)[:, None].expand_as(pos)
    rows = torch.zeros(tokens * top_k, hidden, dtype=torch.float64, device=DEV).index_put((pos[live],), x[token[live]])
    parts = []
    for e in range(experts):
        gu = rows[off[e]:off[e + 1]] @ w13[e].t().contiguous()
        g, u = gu[:, :inter], gu[:, inter:]
        parts.append((g * torch.sigmoid(g) * u) @ w2[e].t().contiguous())
    y = torch.cat(parts + [torch.zeros(tokens * top_k - off[-1], hidden, dtype=torch.float64, device=DEV)])
    out = layer.residual.double().index_add(0, token[live], wt[live][:, None] * y[pos[live]])
    out.backward(layer.d_out.double())
    # Each rounding to E4M3 is off by at most 2^-4 of an element (independent of the others), that to BF16 by 2^-9.  A
    # product of K such elements has a relative error in the 2-norm of about 2^-4 / sqrt(3), as its operand has; out
    # passes two of them and the SiLU product, whose slope is at most 1.1 of each factor: (2^-4 / sqrt(3)) * (1 + 2.1);
    # the gradients pass those of the forward values they are multiplied with and two more.  Twice that as a bound.
    unit = 2.0 ** -4 / 3 ** 0.5
    far = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    got = dict(out=far(step.out.double() - layer.residual.double(), out.detach() - layer.residual.double()),
               d_w=far(step.d_w, wt.grad), d_x=far(step.d_x, x.grad))
    say("  relative errors", got)
    assert got["out"] <= 2 * 3.1 * unit and got["d_w"] <= 2 * 3.1 * unit and got["d_x"] <= 2 * 5.2 * unit
    # and each step by itself on what it was given, where only its own rounding is left
    pos_n, wt_n = s.pos.cpu().numpy(), s.weights.cpu().numpy()
    want_y, want_w, mag = fp8.combine_grad(layer.d_out.double().cpu().numpy(), step.y.double().cpu().numpy(), pos_n, wt_n)
    assert (np.abs(step.d_w.double().cpu().numpy() - want_w) <= hidden * 2.0 ** -24 * mag).all()
    named = ~np.isnan(want_y[:, 0])
    err = np.abs(step.d_y.double().cpu().numpy()[named] - want_y[named])
    assert (err <= bf16_ulp(want_y[named]) / 2 * (1 + 2.0 ** -7)).all()
    dq, ds = oracle.quant_act(bits(step.d_y), 128, e4m3=True)
    qt, st = layer.w2[2].view(torch.uint8).cpu().numpy(), layer.w2[3].cpu().numpy()
    y64, t64, _ = fp8.grouped(fp8.values_a(dq, ds), qt, st, off, None, off[-1], product)
    res = check_bf16(bits(step.d_h)[:off[-1]], y64, t64, hidden, fp8.terms(hidden))
    assert res.ok, str(res)
    want, mag = fp8.dispatch_grad(step.d_rows.double().cpu().numpy(), pos_n)
    bound = (top_k - 1) * 2.0 ** -24 * mag
    assert (np.abs(step.d_x.double().cpu().numpy() - want) <= bound + bf16_ulp(np.abs(want) + bound) / 2 * (1 + 2.0 ** -7)).all()
    # the rows behind the last one stay as they were
    assert not step.d_rows[off[-1]:].any() and not step.y[off[-1]:].any()


def test_replay_in_graph():
    """The layer, a dense projection, the weight quantizer and a whole training step captured together; every replay
    against the same calls made eagerly, with other inputs each time."""
    a, b, c = Layer(5, 130, 16, 4, 512, 256), Layer(6, 2, 64, 8, 256, 128), Layer(7, 60, 6, 2, 256, 128)
    outs = [torch.zeros(m.dims[0], m.dims[3], dtype=torch.bfloat16, device=DEV) for m in (a, b)]
    step = Step(c)
    x, xq, xs = torch.empty(70, 512, dtype=torch.bfloat16, device=DEV), torch.empty(70, 512, dtype=torch.uint8, device=DEV), torch.empty(70, 4, device=DEV)
    w, wq, ws = torch.empty(260, 512, dtype=torch.bfloat16, device=DEV), torch.empty(260, 512, dtype=torch.uint8, device=DEV), torch.empty(3, 4, device=DEV)
    dense = torch.zeros(70, 260, dtype=torch.bfloat16, device=DEV)

    def everything():
        a.forward(outs[0])
        b.forward(outs[1])
        bsr.quantize_w_fp8(w, wq, ws)
        bsr.prefill_fp8(x, wq, ws, xq, xs, dense)
        step.run()

    def new_inputs():
        for m in (a, b, c):
            m.new_inputs()
        x.normal_(generator=a.g)
        w.normal_(generator=a.g)

    new_inputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        everything()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        everything()
    for rep in range(4):
        new_inputs()
        for v in outs + [dense] + step.results():  # (rows behind the last are left as they were: the same on both sides)
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in outs + [dense, wq, ws] + step.results()]
        for v in outs + [dense] + step.results():
            v.zero_()
        everything()
        torch.cuda.synchronize()
        for i, (g, v) in enumerate(zip(got, outs + [dense, wq, ws] + step.results())):
            assert torch.equal(g.view(torch.uint8), v.view(torch.uint8)), f"replay {rep}, output {i}"
        say(f"graph replay {rep} equal")


def test_two_streams():
    layers = [Layer(11, 200, 8, 2, 512, 256), Layer(12, 260, 16, 4, 384, 128)]
    steps = [Step(m) for m in layers]
    alone = []
    for m, st in zip(layers, steps):
        st.run()
        torch.cuda.synchronize()
        alone.append([v.clone() for v in st.results()])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        for st in steps:
            for v in st.results():
                v.zero_()
        torch.cuda.synchronize()
        for st, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                st.run()
        torch.cuda.synchronize()
        for st, ref in zip(steps, alone):
            for v, r in zip(st.results(), ref):
                assert torch.equal(v.view(torch.uint8), r.view(torch.uint8)), rep
    # and on a stream passed by argument
    out = torch.zeros_like(layers[0].x)
    layers[0].forward(out)
    torch.cuda.synchronize()
    other = torch.zeros_like(out)
    bsr.moe_prefill_fp8(layers[0].x, layers[0].logits, *layers[0].w13[:2], *layers[0].w2[:2], other, layers[0].scratch,
                        residual=layers[0].residual, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(out.view(torch.int16), other.view(torch.int16))


# ---- past 32-bit offsets --------------------------------------------------------

def _codes(g, *shape):
    return torch.randint(0, 127, shape, dtype=torch.uint8, device=DEV, generator=g)


@pytest.mark.parametrize("last", [3, 100])
def test_weights_past_4_gib(last):
    """Weights and scales of the last experts start past 4 GiB; streamed rows and tiles."""
    experts, n, k = 40, 8192, 16384
    g = torch.Generator(DEV).manual_seed(1)
    w = _codes(g, experts, n, k)
    w_s = torch.rand(experts, n // 128, k // 128, device=DEV, generator=g) * 2.0 ** -12
    rows = 3 + last
    a, a_s = _codes(g, rows, k), torch.rand(rows, k // 128, device=DEV, generator=g) * 2.0 ** -8
    counts = torch.zeros(experts, dtype=torch.int32)
    counts[0], counts[-2], counts[-1] = 1, 2, last
    off = torch.cat((torch.zeros(1, dtype=torch.int32), counts.cumsum(0).int())).to(DEV)
    out = canary_out(rows, n)
    bsr.fp8_grouped_gemm_blockscaled(a, w, a_s, w_s, off, out)
    cols = slice(n - 300, n)
    for e, lo, hi in ((0, 0, 1), (experts - 2, 1, 3), (experts - 1, 3, 3 + min(last, 5))):
        y, t = product(fp8.values_a(a[lo:hi].cpu().numpy(), a_s[lo:hi].cpu().numpy()),
                       fp8.values_w(w[e].cpu().numpy(), w_s[e].cpu().numpy())[cols])
        res = check_bf16(host(out[lo:hi, cols].contiguous()), y, t, k, fp8.terms(k))
        say(f"expert {e}: {res}")
        assert res.ok, str(res)


def test_activations_and_outputs_past_4_gib():
    """A dense product whose rows and outputs pass 2^32 elements, and a gathered one just under 4 GiB of operand."""
    m, n, k = 270000, 16640, 16384
    g = torch.Generator(DEV).manual_seed(2)
    a, w = _codes(g, m, k), _codes(g, n, k)
    a_s, w_s = torch.rand(m, k // 128, device=DEV, generator=g) * 2.0 ** -8, torch.rand(n // 128, k // 128, device=DEV, generator=g) * 2.0 ** -10
    out = torch.full((m, n), CANARY, dtype=torch.int16, device=DEV)
    bsr.fp8_gemm_blockscaled(a, w, a_s, w_s, out)
    picks = [0, 255, 262143, 262144, m - 1]
    cols = slice(n - 140, n)
    av = fp8.values_a(a[picks].cpu().numpy(), a_s[picks].cpu().numpy())
    wv = fp8.values_w(w.cpu().numpy(), w_s.cpu().numpy())[cols]
    y, t = product(av, wv)
    res = check_bf16(host(out[picks][:, cols].contiguous()), y, t, k, fp8.terms(k))
    assert res.ok, str(res)
    assert not (out == CANARY).all(1).any()
    del out
    rows = 262143  # times k just under 2^32 bytes
    index = torch.tensor([rows - 1, -1, rows, 0, 131072], dtype=torch.int32, device=DEV)
    for copies in (1, 30):  # streamed, and tiles
        idx = index.repeat(copies)
        got = canary_out(5 * copies, n)
        off = torch.tensor([0, 5 * copies], dtype=torch.int32, device=DEV)
        bsr.fp8_grouped_gemm_blockscaled(a[:rows], w[None], a_s[:rows], w_s[None], off, got, row_index=idx)
        at = [rows - 1, 0, 131072]
        y, t = product(fp8.values_a(a[at].cpu().numpy(), a_s[at].cpu().numpy()), wv)
        res = check_bf16(host(got[[5 * copies - 5, 5 * copies - 2, 5 * copies - 1]][:, cols].contiguous()), y, t, k, fp8.terms(k))
        assert res.ok, str(res)
        assert not got[[1, 2]].any()

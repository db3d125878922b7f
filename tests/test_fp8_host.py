"""FP8 products and token rows on the CPU: the refusals of the C ABI and of the binding, the device that layers run on,
and the oracle against independent forms."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from block_scaled_precision_requant_amd import bsr
from oracle import fp8

FAKE = ctypes.c_void_p(1 << 20)       # never dereferenced: every call below fails validation first
INV, NUL, ALI, OK, NODEV = bsr.BSR_EINVAL, bsr.BSR_ENULL, bsr.BSR_EALIGN, bsr.BSR_OK, bsr.BSR_EDEVICE
I8, I32, F32, U8, BF, E4 = torch.int8, torch.int32, torch.float32, torch.uint8, torch.bfloat16, torch.float8_e4m3fn


def _fake(off):
    return ctypes.c_void_p((1 << 20) + off)


def _call(name, defaults, **change):
    args = dict(defaults)
    assert set(change) <= set(args)
    args.update(change)
    return getattr(bsr.lib(), name)(*args.values())


QUANT = dict(w=FAKE, q=FAKE, s=FAKE, qt=None, st=None, experts=1, n=4, k=128, stream=None)
GEMM = dict(a=FAKE, w=FAKE, a_s=FAKE, w_s=FAKE, out=FAKE, m=4, n=8, k=128, stream=None)
GROUPED = dict(a=FAKE, w=FAKE, a_s=FAKE, w_s=FAKE, offsets=FAKE, row_index=None, silu_mul=0, out=FAKE, a_rows=4, rows=4,
               experts=2, n=8, k=128, stream=None)
DISPATCH = dict(x=FAKE, pos=FAKE, out=FAKE, tokens=4, top_k=2, rows=8, n=8, stream=None)
COMBINE_GRAD = dict(d_out=FAKE, y=FAKE, pos=FAKE, weights=FAKE, d_y=FAKE, d_weights=FAKE, tokens=4, top_k=2, rows=8, n=8,
                    stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(k=0), INV), (dict(k=64), INV), (dict(k=130), INV), (dict(qt=FAKE, st=FAKE, n=130), INV), (dict(n=0), OK),
    (dict(experts=0), OK), (dict(w=None), NUL), (dict(q=None), NUL), (dict(s=None), NUL), (dict(qt=FAKE, n=128), NUL),
    (dict(st=FAKE, n=128), NUL), (dict(w=_fake(8)), ALI), (dict(q=_fake(8)), ALI), (dict(s=_fake(2)), ALI),
    (dict(qt=_fake(8), st=FAKE, n=128), ALI), (dict(qt=FAKE, st=_fake(2), n=128), ALI),
    (dict(experts=1 << 24), INV), (dict(n=(1 << 32) - 1, k=(1 << 32) - 128), INV)])
def test_quantize_refusals(change, status):
    assert _call("quantize_w_fp8", QUANT, **change) == status


# sizes whose number of threads passes 64 bits: 2^56 blocks, as many and a few, just under 2^64
@pytest.mark.parametrize("change", [
    dict(experts=1 << 31, n=1 << 20, k=1 << 19), dict(experts=1 << 31, n=(1 << 20) + 1, k=1 << 19),
    dict(experts=(1 << 32) - 1, n=(1 << 32) - 128, k=128), dict(experts=(1 << 32) - 1, n=1, k=128 * ((1 << 25) - 1)),
    dict(experts=1 << 31, n=1 << 20, k=1 << 19, qt=FAKE, st=FAKE)])
def test_quantize_refuses_thread_counts_past_64_bits(change):
    assert _call("quantize_w_fp8", QUANT, **change) == INV


BOTH = [(dict(k=0), INV), (dict(k=64), INV), (dict(k=1 << 23), INV), (dict(n=1 << 31), INV), (dict(n=0), OK),
        (dict(a=None), NUL), (dict(w=None), NUL), (dict(a_s=None), NUL), (dict(w_s=None), NUL), (dict(out=None), NUL),
        (dict(a=_fake(8)), ALI), (dict(w=_fake(8)), ALI), (dict(a_s=_fake(2)), ALI), (dict(w_s=_fake(2)), ALI),
        (dict(out=_fake(1)), ALI)]


@pytest.mark.parametrize("change, status", BOTH + [(dict(m=0), OK), (dict(m=1 << 31), INV),
                                                   (dict(m=(1 << 31) - 1, n=1 << 20), INV)])
def test_gemm_refusals(change, status):
    assert _call("fp8_gemm_blockscaled", GEMM, **change) == status


@pytest.mark.parametrize("change, status", BOTH + [
    (dict(rows=0), OK), (dict(experts=0), OK), (dict(experts=65537), INV), (dict(rows=1 << 31, a_rows=1 << 31), INV),
    (dict(rows=5), INV), (dict(row_index=FAKE, a_rows=0), INV), (dict(row_index=FAKE, a_rows=1 << 25), INV),
    (dict(silu_mul=2), INV), (dict(silu_mul=1, n=128), INV), (dict(silu_mul=1, n=254), INV), (dict(offsets=None), NUL),
    (dict(offsets=_fake(2)), ALI), (dict(row_index=_fake(2)), ALI),
    (dict(rows=(1 << 31) - 1, a_rows=(1 << 31) - 1, n=1 << 20), INV)])
def test_grouped_refusals(change, status):
    assert _call("fp8_grouped_gemm_blockscaled", GROUPED, **change) == status


@pytest.mark.parametrize("name", ["moe_dispatch", "moe_dispatch_grad"])
@pytest.mark.parametrize("change, status", [
    (dict(top_k=0), INV), (dict(top_k=17), INV), (dict(n=1 << 31), INV), (dict(tokens=1 << 24), INV),
    (dict(tokens=1 << 23, top_k=1, n=4096), INV), (dict(tokens=0), OK), (dict(n=0), OK), (dict(x=None), NUL), (dict(pos=None), NUL),
    (dict(out=None), NUL), (dict(x=_fake(1)), ALI), (dict(pos=_fake(2)), ALI), (dict(out=_fake(1)), ALI)])
def test_dispatch_refusals(name, change, status):
    assert _call(name, DISPATCH, **change) == status


@pytest.mark.parametrize("change, status", [
    (dict(top_k=0), INV), (dict(top_k=17), INV), (dict(n=1 << 31), INV), (dict(tokens=1 << 24), INV), (dict(tokens=0), OK)] +
    [({a: None}, NUL) for a in ("d_out", "y", "pos", "weights", "d_y", "d_weights")] +
    [({a: _fake(1)}, ALI) for a in ("d_out", "y", "d_y")] + [({a: _fake(2)}, ALI) for a in ("pos", "weights", "d_weights")])
def test_combine_grad_refusals(change, status):
    assert _call("moe_combine_grad", COMBINE_GRAD, **change) == status


# Launches end at 2^32 threads: the last sizes that pass go on to the device check.
@pytest.mark.skipif(torch.cuda.is_available(), reason="the sizes that pass would be launched")
@pytest.mark.parametrize("name, defaults, change, status", [
    ("quantize_w_fp8", QUANT, dict(experts=(1 << 24) - 1), NODEV),
    ("quantize_w_fp8", QUANT, dict(n=1 << 31), INV),
    ("quantize_w_fp8", QUANT, dict(n=(1 << 31) - 128), NODEV),
    ("fp8_gemm_blockscaled", GEMM, dict(k=(1 << 23) - 128), NODEV),
    ("fp8_gemm_blockscaled", GEMM, dict(m=1 << 20, n=1 << 20), INV),
    ("fp8_gemm_blockscaled", GEMM, dict(m=1 << 20, n=1 << 18), NODEV),
    ("fp8_grouped_gemm_blockscaled", GROUPED, dict(row_index=FAKE, a_rows=(1 << 25) - 1), NODEV),
    ("moe_dispatch", DISPATCH, dict(tokens=(1 << 24) - 1, top_k=1), NODEV),
    ("moe_dispatch", DISPATCH, dict(tokens=(1 << 23) - 1, top_k=1, n=4096), NODEV),
    ("moe_dispatch_grad", DISPATCH, dict(rows=0, x=None), NODEV),
    ("moe_dispatch", DISPATCH, dict(rows=0, out=None), NODEV),
    ("moe_combine_grad", COMBINE_GRAD, dict(rows=0, y=None, d_y=None), NODEV),
    ("moe_combine_grad", COMBINE_GRAD, dict(n=0, d_out=None, y=None, d_y=None), NODEV)])
def test_launch_limits(name, defaults, change, status):
    assert _call(name, defaults, **change) == status


# ---- the binding --------------------------------------------------------------

def zeros(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt)


@pytest.fixture
def launched(monkeypatch):
    """Names of the launches that a call comes to, none of which runs."""
    names = []
    monkeypatch.setattr(bsr, "_launch", lambda name, *a: names.append(name))
    monkeypatch.setattr(bsr, "quantize_act", lambda *a, **k: names.append("quantize_act"))
    return names


class Layer:
    """Arguments of the FP8 layer, all right but for where they are."""

    def __init__(self, tokens=4, experts=3, top_k=2, h=128, i=256):
        self.scratch = bsr.MoeScratch(8, experts, top_k, h, i, device="cpu")
        self.args = dict(x_bf16=zeros(tokens, h), logits=zeros(tokens, experts, dt=F32), w_gate_up=zeros(experts, 2 * i, h, dt=E4),
                         gate_up_scale=zeros(experts, 2 * i // 128, h // 128, dt=F32), w_down=zeros(experts, h, i, dt=U8),
                         down_scale=zeros(experts, h // 128, i // 128, dt=F32), out=zeros(tokens, h))

    def __call__(self, **change):
        bsr.moe_prefill_fp8(**{**self.args, **change}, scratch=self.scratch)


def _calls():
    """name -> (call, its arguments, all right)."""
    x, rows, pos, wt = zeros(4, 256), zeros(8, 256), zeros(4, 2, dt=I32), zeros(4, 2, dt=F32)
    return {
        "quantize": (bsr.quantize_w_fp8, dict(w_bf16=zeros(2, 128, 256), w_q=zeros(2, 128, 256, dt=E4), w_scale=zeros(2, 1, 2, dt=F32),
                                              w_qt=zeros(2, 256, 128, dt=U8), w_scale_t=zeros(2, 2, 1, dt=F32))),
        "gemm": (bsr.fp8_gemm_blockscaled, dict(a_q=zeros(4, 256, dt=U8), w_q=zeros(130, 256, dt=E4), a_scale=zeros(4, 2, dt=F32),
                                                w_scale=zeros(2, 2, dt=F32), out=zeros(4, 130))),
        "grouped": (bsr.fp8_grouped_gemm_blockscaled,
                    dict(a_q=zeros(4, 256, dt=E4), w_q=zeros(3, 256, 256, dt=U8), a_scale=zeros(4, 2, dt=F32),
                         w_scale=zeros(3, 2, 2, dt=F32), offsets=zeros(4, dt=I32), out=zeros(8, 128),
                         row_index=zeros(8, dt=I32), silu_mul=True)),
        "prefill": (bsr.prefill_fp8, dict(a_bf16=x, w_q=zeros(130, 256, dt=E4), w_scale=zeros(2, 2, dt=F32),
                                          a_q_scratch=zeros(4, 256, dt=U8), a_scale_scratch=zeros(4, 2, dt=F32),
                                          out=zeros(4, 130))),
        "dispatch": (bsr.moe_dispatch, dict(x=x, pos=pos, out=rows)),
        "dispatch_grad": (bsr.moe_dispatch_grad, dict(d_rows=rows, pos=pos, d_x=x)),
        "combine_grad": (bsr.moe_combine_grad, dict(d_out=x, y=rows, pos=pos, weights=wt, d_y=zeros(8, 256), d_weights=zeros(4, 2, dt=F32))),
    }


CASES = [(name, arg) for name, (_, args) in _calls().items() for arg, t in args.items() if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("name", list(_calls()))
def test_right_arguments_are_launched(name, launched):
    fn, args = _calls()[name]
    fn(**args)
    assert len(launched) == (2 if name == "prefill" else 1)


@pytest.mark.parametrize("name, arg", CASES)
def test_each_argument_is_checked_before_any_launch(name, arg, launched):
    """Another element type, another size, strides, another device: each is refused by every argument."""
    fn, args = _calls()[name]
    t = args[arg]
    wrong = {F32: torch.float64, I32: torch.int64, BF: torch.float16, U8: I8, E4: torch.float8_e5m2}[t.dtype]
    bad = [t.view(wrong) if t.element_size() == wrong.itemsize else t.to(wrong),
           torch.cat((t, t[:1])) if t.dtype != E4 else torch.cat((t.view(U8), t[:1].view(U8))).view(E4),
           t.as_subclass(Card1)]
    if t.dim() > 1 and t.shape[-1] > 1:
        bad.append(t.transpose(-1, -2).contiguous().transpose(-1, -2))
    for i, b in enumerate(bad):
        if i == 1 and (name, arg) in GROWS:
            continue  # (that size is the call's own: the others must follow it)
        if i == 3 and b.is_contiguous():
            continue
        with pytest.raises(ValueError):
            fn(**{**args, arg: b})
        assert not launched, (i, launched)


# arguments one more row of which still fits what they are checked against
GROWS = {("dispatch", "out"), ("dispatch_grad", "d_rows")}


class Card1(torch.Tensor):
    """A tensor that says it is on cuda:1."""

    def get_device(self):
        return 1


def test_other_codes_are_refused(launched):
    fn, args = _calls()["gemm"]
    for arg in ("a_q", "w_q"):
        for dt in (I8, torch.bool, torch.float8_e5m2, torch.float8_e4m3fnuz):
            with pytest.raises(ValueError, match=f"{arg}: dtype"):
                fn(**{**args, arg: zeros(*args[arg].shape, dt=U8).view(dt)})
    assert not launched


def test_sizes_past_32_bits_are_refused():
    n = (1 << 32) + 128
    with pytest.raises(ValueError, match="32 bits"):
        bsr.quantize_w_fp8(zeros(0, 128, n), zeros(0, 128, n, dt=U8), zeros(0, 1, n // 128, dt=F32))
    with pytest.raises(ValueError, match="32 bits"):
        bsr.fp8_gemm_blockscaled(zeros(0, n, dt=U8), zeros(0, n, dt=U8), zeros(0, n // 128, dt=F32), zeros(0, n // 128, dt=F32),
                                 zeros(0, 0))
    with pytest.raises(ValueError, match="32 bits"):
        bsr.fp8_grouped_gemm_blockscaled(zeros(0, n, dt=U8), zeros(0, 256, n, dt=U8), zeros(0, n // 128, dt=F32),
                                         zeros(0, 2, n // 128, dt=F32), zeros(1, dt=I32), zeros(0, 256))
    with pytest.raises(ValueError, match="32 bits"):
        bsr.moe_dispatch(zeros(0, n), zeros(0, 2, dt=I32), zeros(0, n))
    with pytest.raises(ValueError, match="32 bits"):
        bsr.moe_combine_grad(zeros(0, n), zeros(0, n), zeros(0, 2, dt=I32), zeros(0, 2, dt=F32), zeros(0, n), zeros(0, 2, dt=F32))


def test_quantizer_needs_both_transposed_or_neither(launched):
    fn, args = _calls()["quantize"]
    for arg in ("w_qt", "w_scale_t"):
        with pytest.raises(ValueError, match="both or neither"):
            fn(**{**args, arg: None})
    fn(**{**args, "w_qt": None, "w_scale_t": None})
    for w in (zeros(2, 128, 192), zeros(2, 2, 2, 128), zeros(128)):
        with pytest.raises(ValueError):
            fn(**{**args, "w_bf16": w})
    assert launched == ["quantize_w_fp8"]


def test_layer_refusals(launched):
    layer = Layer()
    layer()
    assert launched == ["moe_route", "quantize_act", "fp8_grouped_gemm_blockscaled", "quantize_act",
                        "fp8_grouped_gemm_blockscaled", "moe_combine"]
    del launched[:]
    a = layer.args
    for change in (dict(logits=zeros(3, 3, dt=F32)), dict(logits=a["logits"].as_subclass(Card1)), dict(out=a["out"].half()),
                   dict(x_bf16=a["x_bf16"].half()), dict(residual=a["out"].half()), dict(w_down=zeros(3, 128, 192, dt=U8))):
        with pytest.raises(ValueError):
            layer(**change)
        assert not launched, change


@pytest.mark.parametrize("arg", ["x_bf16", "logits", "w_gate_up", "gate_up_scale", "w_down", "down_scale", "out", "residual"])
def test_layer_checks_each_argument_before_any_launch(arg, launched):
    """Another element type, another size in each dimension, strides, another device."""
    layer = Layer()
    t = layer.args.get(arg, layer.args["out"])
    wrong = {F32: torch.float64, BF: torch.float16, U8: I8, E4: torch.float8_e5m2}[t.dtype]
    bad = [t.view(wrong) if t.element_size() == wrong.itemsize else t.to(wrong), t.as_subclass(Card1),
           t.transpose(-1, -2).contiguous().transpose(-1, -2)]
    assert not bad[-1].is_contiguous() or 1 in t.shape[-2:]
    bad += [zeros(*(n + 128 * (i == j) for i, n in enumerate(t.shape)), dt=t.dtype) for j in range(t.dim())]
    for i, b in enumerate(bad):
        if i == 2 and b.is_contiguous():
            continue
        with pytest.raises(ValueError):
            layer(**{arg: b})
        assert not launched, (i, launched)


@pytest.mark.parametrize("other", [dict(h=256), dict(i=128), dict(experts=5)])
def test_layer_refuses_scratch_of_other_sizes(other, launched):
    layer = Layer()
    layer.scratch = Layer(**other).scratch
    with pytest.raises(ValueError, match="scratch"):
        layer()
    assert not launched


@pytest.mark.parametrize("sizes", [dict(h=1 << 23, i=128), dict(h=128, i=1 << 23)])
def test_layer_refuses_widths_past_the_products(sizes, launched):
    """A product ends below 2^23 elements a row; no memory stands behind these tensors."""
    meta = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="meta")  # noqa: E731
    t, e, h, i = 2, 2, sizes["h"], sizes["i"]
    scratch = bsr.MoeScratch(t, e, 1, h, i, device="meta")
    with pytest.raises(ValueError, match=r"2\^23"):
        bsr.moe_prefill_fp8(meta(t, h), meta(t, e, dt=F32), meta(e, 2 * i, h, dt=E4), meta(e, 2 * i // 128, h // 128, dt=F32),
                            meta(e, h, i, dt=E4), meta(e, h // 128, i // 128, dt=F32), meta(t, h), scratch)
    assert not launched


def test_layer_refuses_tokens_past_the_gather(launched):
    """Gathered rows end at 2^32 bytes."""
    meta = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="meta")  # noqa: E731
    t, e, h, i = 1 << 19, 2, 8192, 128
    scratch = bsr.MoeScratch(t, e, 1, h, i, device="meta")
    with pytest.raises(ValueError, match=r"2\^32"):
        bsr.moe_prefill_fp8(meta(t, h), meta(t, e, dt=F32), meta(e, 2 * i, h, dt=E4), meta(e, 2 * i // 128, h // 128, dt=F32),
                            meta(e, h, i, dt=E4), meta(e, h // 128, i // 128, dt=F32), meta(t, h), scratch)
    assert not launched


def test_prefill_refuses_a_width_past_the_product(launched):
    """Before the quantizer runs."""
    meta = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="meta")  # noqa: E731
    k = 1 << 23
    with pytest.raises(ValueError, match=r"2\^23"):
        bsr.prefill_fp8(meta(2, k), meta(4, k, dt=E4), meta(1, k // 128, dt=F32), meta(2, k, dt=E4), meta(2, k // 128, dt=F32),
                        meta(2, 4))
    assert not launched


def test_layer_runs_on_its_tensors_device(monkeypatch):
    """Every step runs with its tensors' device as the current one, whichever is current around the call."""
    current, seen = [0], []

    class device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, current[0] = current[0], self.dev

        def __exit__(self, *_):
            current[0] = self.before

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, current[0])) or bsr.BSR_OK

    monkeypatch.setattr(bsr, "_LIB", Lib())
    monkeypatch.setattr(bsr, "_ptr", lambda t: None)
    monkeypatch.setattr(bsr, "_stream", lambda *a: None)
    monkeypatch.setattr(bsr, "_current_stream", lambda dev: 0)
    monkeypatch.setattr(bsr, "_current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    layer = Layer()
    card = lambda t: t.as_subclass(Card1)  # noqa: E731
    for name, t in vars(layer.scratch).items():
        if isinstance(t, torch.Tensor):
            setattr(layer.scratch, name, card(t))
    layer(**{k: card(t) for k, t in layer.args.items()})
    for name, (fn, args) in _calls().items():
        fn(**{k: card(t) if isinstance(t, torch.Tensor) else t for k, t in args.items()})
    assert len(seen) == 6 + 8 and {dev for _, dev in seen} == {1}, seen
    assert current == [0]


# ---- the oracle ---------------------------------------------------------------

def test_e4m3_table_and_rounding():
    codes = torch.arange(256, dtype=torch.uint8).view(E4).float().numpy()
    assert np.array_equal(codes, fp8.E4M3.astype(np.float32), equal_nan=True)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(2000) * 2.0 ** rng.integers(-12, 9, 2000), fp8.E4M3[:127], -fp8.E4M3[:127],
                        (fp8.E4M3[1:127] + fp8.E4M3[:126]) / 2, [0.0, -0.0, 500.0, -1e9, 2.0 ** -10, -(2.0 ** -10)]]).astype(np.float32)
    x = np.clip(x, -448, 448)
    assert np.array_equal(fp8.e4m3_nearest(x), torch.from_numpy(x).to(E4).view(U8).numpy())
    assert [int(c) for c in fp8.e4m3_nearest(x[:300])] == [oracle.e4m3_encode(float(v)) for v in x[:300]]


def test_products_and_gradients_of_the_oracle():
    """The oracle's sums against torch's, and its gradients against autograd of the forward formulas."""
    rng = np.random.default_rng(2)
    q, s = fp8.quantize_w(rng.standard_normal((200, 256)).astype(np.float32))
    v = torch.from_numpy(q).view(E4).double()
    big = torch.from_numpy(s).double().repeat_interleave(128, 0)[:200].repeat_interleave(128, 1)
    assert np.array_equal(fp8.values_w(q, s), (v * big).numpy())
    t, k, n = 7, 3, 11
    pos = rng.permutation(t * k).reshape(t, k)
    pos[2, 1] = -1
    pos[5] = -1
    x = torch.from_numpy(rng.standard_normal((t, n))).requires_grad_()
    rows = torch.zeros(t * k, n, dtype=torch.float64)
    live = torch.from_numpy(pos >= 0)
    at = torch.from_numpy(pos)[live]
    sent = rows.index_put((at,), x[:, None].expand(t, k, n)[live])
    assert np.array_equal(fp8.dispatch(x.detach().numpy(), pos, rows.numpy()), sent.detach().numpy())
    d = torch.from_numpy(rng.standard_normal((t * k, n)))
    sent.backward(d)
    assert np.allclose(fp8.dispatch_grad(d.numpy(), pos)[0], x.grad.numpy(), rtol=1e-14, atol=1e-14)
    y = d.clone().requires_grad_()
    w = torch.from_numpy(rng.standard_normal((t, k))).requires_grad_()
    out = torch.zeros(t, n, dtype=torch.float64).index_add(0, torch.nonzero(live)[:, 0], w[live][:, None] * y[at])
    d_out = torch.from_numpy(rng.standard_normal((t, n)))
    out.backward(d_out)
    d_y, d_w, _ = fp8.combine_grad(d_out.numpy(), y.detach().numpy(), pos, w.detach().numpy())
    assert np.allclose(d_w, w.grad.numpy(), rtol=1e-13, atol=1e-13)
    named = ~np.isnan(d_y[:, 0])
    assert np.allclose(d_y[named], y.grad.numpy()[named], rtol=1e-14) and not y.grad.numpy()[~named].any()

"""The binding of the expert layers on the CPU: what it refuses before any launch."""
import pytest
import torch

from block_scaled_precision_requant_amd import bsr

I8, I32, F32, U8, BF = torch.int8, torch.int32, torch.float32, torch.uint8, torch.bfloat16


def zeros(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt)


class Layer:
    """Arguments of both layer calls, all right but for where they are."""

    def __init__(self, tokens=4, experts=3, top_k=2, h=64, i=32):
        self.scratch = bsr.MoeScratch(8, experts, top_k, h, i, device="cpu")
        self.x, self.logits, self.out = zeros(tokens, h), zeros(tokens, experts, dt=F32), zeros(tokens, h)
        e = experts
        self.i8 = [zeros(e, 2 * i, h, dt=I8), zeros(e, 2 * i, h // 32, dt=F32), zeros(e, h, i, dt=I8),
                   zeros(e, h, i // 32, dt=F32)]
        self.w4 = [zeros(e, 2 * i, h // 2, dt=U8), zeros(e, 2 * i, h // 32, dt=F32), None,
                   zeros(e, h, i // 2, dt=U8), zeros(e, h, i // 32, dt=F32), None]

    def prefill(self, **change):
        self._call(bsr.moe_prefill, self.i8, change)

    def decode(self, **change):
        self._call(bsr.moe_decode_w4, self.w4, change)

    def _call(self, fn, weights, change):
        a = dict(x=self.x, logits=self.logits, out=self.out, residual=None)
        a.update(change)
        fn(a["x"], a["logits"], *weights, a["out"], self.scratch, residual=a["residual"])


@pytest.fixture
def launched(monkeypatch):
    """Names of the launches that a call comes to, none of which runs."""
    names = []
    monkeypatch.setattr(bsr, "_launch", lambda name, *a: names.append(name))
    for name in ("requant_a_int8", "silu_mul_requant_int8"):
        monkeypatch.setattr(bsr, name, lambda *a, name=name, **k: names.append(name))
    return names


@pytest.mark.parametrize("path", ["prefill", "decode"])
@pytest.mark.parametrize("tokens", [0, 3, 5])
def test_layers_reject_logits_of_other_tokens(path, tokens, launched):
    layer = Layer(tokens=4)
    getattr(layer, path)()
    assert launched[0] == "moe_route" and launched[-1] == "moe_combine"
    del launched[:]
    with pytest.raises(ValueError, match=f"logits: {tokens} tokens, x_bf16 4"):
        getattr(layer, path)(logits=zeros(tokens, 3, dt=F32))
    assert not launched


def _float16_calls():
    ids, pos, off, rows = zeros(4, 2, dt=I32), zeros(4, 2, dt=I32), zeros(4, dt=I32), zeros(8, dt=I32)
    wt, y, w4, s4 = zeros(4, 2, dt=F32), zeros(8, 64), zeros(64, 32, dt=U8), zeros(64, 2, dt=torch.float16)
    e4, es4, x, out = zeros(3, 64, 32, dt=U8), zeros(3, 64, 2, dt=F32), zeros(4, 64), zeros(4, 64)
    a, a_s, w, w_s = zeros(4, 64, dt=I8), zeros(4, 2, dt=F32), zeros(3, 64, 64, dt=I8), zeros(3, 64, 2, dt=F32)
    layer = Layer()
    return [
        ("x_bf16", lambda h: bsr.w4a16_group_gemv(h(x), w4, s4, out)),
        ("out", lambda h: bsr.w4a16_group_gemv(x, w4, s4, h(out))),
        ("x_bf16", lambda h: bsr.w4a16_group_gemv_experts(h(x), e4, es4, off, out)),
        ("out", lambda h: bsr.w4a16_group_gemv_experts(x, e4, es4, off, h(out))),
        ("out", lambda h: bsr.int8_grouped_gemm_blockscaled(a, w, a_s, w_s, off, h(out))),
        ("y", lambda h: bsr.moe_combine(h(y), pos, wt, out)),
        ("residual", lambda h: bsr.moe_combine(y, pos, wt, out, residual=h(out))),
        ("out", lambda h: bsr.moe_combine(y, pos, wt, h(out))),
        ("x_bf16", lambda h: layer.prefill(x=h(layer.x))),
        ("x_bf16", lambda h: layer.decode(x=h(layer.x))),
        ("out", lambda h: layer.prefill(out=h(layer.out))),
        ("residual", lambda h: layer.decode(residual=h(layer.out))),
    ]


@pytest.mark.parametrize("i", range(12))
def test_float16_is_not_read_as_bf16(i, launched):
    """A float16 tensor has a type of its own here (logits and scales are read as such): never raw BF16 bits."""
    what, call = _float16_calls()[i]
    call(lambda t: t)
    call(lambda t: t.view(torch.int16))  # raw bits stay welcome
    call(lambda t: t.view(torch.uint16))
    with pytest.raises(ValueError, match=f"{what}: dtype torch.float16"):
        call(lambda t: t.view(torch.float16))


def test_float16_layer_inputs_are_refused_before_any_launch(launched):
    layer = Layer()
    for change in (dict(x=layer.x.half()), dict(out=layer.out.half()), dict(residual=layer.out.half())):
        for path in (layer.prefill, layer.decode):
            with pytest.raises(ValueError, match="dtype torch.float16"):
                path(**change)
            assert not launched


class Card1(torch.Tensor):
    """A tensor that says it is on cuda:1."""

    def get_device(self):
        return 1


@pytest.mark.parametrize("path, steps", [("prefill", 6), ("decode", 4)])
def test_layers_run_on_their_tensors_device(path, steps, monkeypatch):
    """Every step of a layer runs with its tensors' device as the current one, whichever is current around the call."""
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
    card = lambda t: None if t is None else t.as_subclass(Card1)  # noqa: E731
    layer.i8, layer.w4 = [card(t) for t in layer.i8], [card(t) for t in layer.w4]
    for name, t in vars(layer.scratch).items():
        if isinstance(t, torch.Tensor):
            setattr(layer.scratch, name, card(t))
    getattr(layer, path)(x=card(layer.x), logits=card(layer.logits), out=card(layer.out))
    assert len(seen) == steps and {dev for _, dev in seen} == {1}, seen
    assert current == [0]


@pytest.mark.parametrize("path", ["prefill", "decode"])
def test_layers_reject_logits_on_another_device(path, launched):
    """The router would run on the logits' device and read and write the scratch there, the rest on x_bf16's."""
    layer = Layer()
    with pytest.raises(ValueError, match="logits: on"):
        getattr(layer, path)(logits=layer.logits.as_subclass(Card1))
    assert not launched


def test_route_top_k_past_32_bits_is_refused():
    """Without tokens the ids [0, k] take no memory whatever k is; k = 2^32 + 2 was cut to 2."""
    k = (1 << 32) + 2
    with pytest.raises(ValueError, match="32 bits"):
        bsr.moe_route(zeros(0, 4, dt=F32), zeros(0, k, dt=I32), zeros(0, k, dt=F32), zeros(5, dt=I32), zeros(0, dt=I32),
                      zeros(0, k, dt=I32))


@pytest.mark.parametrize("dtype", [torch.int8, torch.bool, torch.float8_e4m3fn])
def test_zero_points_are_numbers_from_0_to_255(dtype, launched):
    """The kernel reads zero points as unsigned bytes: an int8 -1 would count as 255."""
    x, out = zeros(4, 64), zeros(4, 64)
    w, s, z = zeros(64, 32, dt=U8), zeros(64, 2, dt=F32), zeros(64, 2, dt=U8)
    bsr.w4a16_group_gemv(x, w, s, out, zero=z)
    with pytest.raises(ValueError, match="zero: dtype"):
        bsr.w4a16_group_gemv(x, w, s, out, zero=z.to(dtype))
    e = [t.expand(3, *t.shape).contiguous() for t in (w, s, z)]
    bsr.w4a16_group_gemv_experts(x, e[0], e[1], zeros(4, dt=I32), out, zero=e[2])
    with pytest.raises(ValueError, match="zero: dtype"):
        bsr.w4a16_group_gemv_experts(x, e[0], e[1], zeros(4, dt=I32), out, zero=e[2].to(dtype))


@pytest.mark.parametrize("sizes", [((1 << 32) + 5, 8, 2), (5, (1 << 32) + 8, 2), (5, 8, (1 << 32) + 2), (-1, 8, 2)])
def test_workspace_of_sizes_past_32_bits_is_refused(sizes):
    """A cut token count would name a workspace far too small."""
    with pytest.raises(ValueError, match="32 bits"):
        bsr.moe_route_ws_bytes(*sizes)

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

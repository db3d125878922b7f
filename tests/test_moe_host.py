"""Expert-layer operators on the CPU: the refusals of the C ABI and of the
binding, the router's launch plan, and the oracle against independent forms."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from block_scaled_precision_requant_amd import bsr
from oracle import moe

FAKE = ctypes.c_void_p(1 << 20)       # never dereferenced: every call below fails validation first
INV, NUL, ALI, OK = bsr.BSR_EINVAL, bsr.BSR_ENULL, bsr.BSR_EALIGN, bsr.BSR_OK


def _fake(off):
    return ctypes.c_void_p((1 << 20) + off)


def _call(name, defaults, **change):
    args = dict(defaults)
    assert set(change) <= set(args)
    args.update(change)
    return getattr(bsr.lib(), name)(*args.values())


ROUTE = dict(logits=FAKE, type=2, ld=8, ids=FAKE, weights=FAKE, offsets=FAKE, row_token=FAKE, pos=FAKE, tokens=4,
             experts=8, top_k=2, score=0, renorm=1, scale=1.0, workspace=None, workspace_bytes=0, stream=None)
GROUPED = dict(a=FAKE, w=FAKE, a_s=FAKE, w_s=FAKE, offsets=FAKE, row_index=None, out=FAKE, a_rows=4, rows=4, experts=2,
               n=8, k=64, stream=None)
COMBINE = dict(y=FAKE, pos=FAKE, weights=FAKE, residual=None, out=FAKE, tokens=4, top_k=2, rows=8, n=8, stream=None)
W4 = dict(x=FAKE, w=FAKE, scale=FAKE, scale_type=0, zero=None, group=32, out=FAKE, m=4, n=8, k=64, stream=None)
W4E = dict(x=FAKE, w=FAKE, scale=FAKE, scale_type=0, zero=None, group=32, offsets=FAKE, row_index=None, silu_mul=0,
           out=FAKE, x_rows=4, rows=4, experts=2, n=8, k=64, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(type=3), INV), (dict(type=-1), INV), (dict(score=2), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(experts=0), INV), (dict(experts=1025, ld=1025), INV), (dict(ld=7), INV),
    (dict(top_k=0), INV), (dict(top_k=9), INV), (dict(top_k=17, experts=64, ld=64), INV),
    (dict(tokens=1 << 30, top_k=2), INV), (dict(tokens=10000), NUL), (dict(tokens=10000, workspace=_fake(8)), ALI),
    (dict(tokens=10000, workspace=FAKE, workspace_bytes=16), INV), (dict(offsets=None), NUL),
    (dict(tokens=0, offsets=None), NUL), (dict(logits=None), NUL), (dict(ids=None), NUL), (dict(weights=None), NUL),
    (dict(row_token=None), NUL), (dict(pos=None), NUL), (dict(logits=_fake(2)), ALI), (dict(pos=_fake(2)), ALI),
    (dict(type=0, logits=_fake(1)), ALI), (dict(weights=_fake(1)), ALI), (dict(offsets=_fake(2)), ALI),
    (dict(ids=_fake(2)), ALI), (dict(row_token=_fake(2)), ALI),
])
def test_route_refusals(change, status):
    assert _call("moe_route", ROUTE, **change) == status


@pytest.mark.parametrize("change, status", [
    (dict(k=0), INV), (dict(k=48), INV), (dict(k=1 << 24), INV), (dict(experts=65537), INV), (dict(rows=1 << 31), INV),
    (dict(rows=5), INV), (dict(row_index=FAKE, a_rows=0), INV), (dict(row_index=FAKE, a_rows=1 << 26, k=64), INV), (dict(rows=0), OK), (dict(n=0), OK),
    (dict(experts=0), OK), (dict(a=None), NUL), (dict(w=None), NUL), (dict(a_s=None), NUL), (dict(w_s=None), NUL),
    (dict(offsets=None), NUL), (dict(out=None), NUL), (dict(a=_fake(8)), ALI), (dict(w=_fake(8)), ALI),
    (dict(a_s=_fake(2)), ALI), (dict(w_s=_fake(2)), ALI), (dict(offsets=_fake(2)), ALI),
    (dict(row_index=_fake(2)), ALI), (dict(out=_fake(1)), ALI),
    (dict(rows=(1 << 31) - 1, a_rows=(1 << 31) - 1, n=1 << 20), INV),
])
def test_grouped_refusals(change, status):
    assert _call("int8_grouped_gemm_blockscaled", GROUPED, **change) == status


@pytest.mark.parametrize("change, status", [
    (dict(top_k=0), INV), (dict(top_k=17), INV), (dict(tokens=0), OK), (dict(n=0), OK), (dict(y=None), NUL),
    (dict(pos=None), NUL), (dict(weights=None), NUL), (dict(out=None), NUL), (dict(y=_fake(1)), ALI),
    (dict(pos=_fake(2)), ALI), (dict(weights=_fake(2)), ALI), (dict(residual=_fake(1)), ALI), (dict(out=_fake(1)), ALI),
    (dict(tokens=1 << 26, n=1 << 13), INV),
])
def test_combine_refusals(change, status):
    assert _call("moe_combine", COMBINE, **change) == status


W4_BOTH = [
    (dict(k=0), INV), (dict(k=48), INV), (dict(group=16), INV), (dict(group=64, k=96), INV), (dict(group=256), INV),
    (dict(k=1 << 24), INV), (dict(scale_type=3), INV), (dict(scale_type=-1), INV), (dict(n=0), OK), (dict(x=None), NUL), (dict(w=None), NUL),
    (dict(scale=None), NUL), (dict(out=None), NUL), (dict(x=_fake(8)), ALI), (dict(w=_fake(8)), ALI),
    (dict(scale=_fake(1)), ALI), (dict(scale=_fake(2), scale_type=2), ALI), (dict(out=_fake(1)), ALI),
]


@pytest.mark.parametrize("change, status", W4_BOTH + [(dict(m=0), OK), (dict(m=1 << 31), INV), (dict(m=1 << 25), INV),
                                                      (dict(m=1 << 24, n=1 << 16), INV)])
def test_w4_group_refusals(change, status):
    assert _call("w4a16_group_gemv", W4, **change) == status


# Launches end at 2^32 threads: the last sizes that pass go on to the device check.
NODEV = bsr.BSR_EDEVICE


@pytest.mark.skipif(torch.cuda.is_available(), reason="the sizes that pass would be launched")
@pytest.mark.parametrize("name, defaults, change, status", [
    ("moe_combine", COMBINE, dict(tokens=(1 << 24) - 1, n=2048), NODEV),
    ("moe_combine", COMBINE, dict(tokens=1 << 24, n=2048), INV),
    ("moe_combine", COMBINE, dict(tokens=1 << 23, n=2048, y=_fake(2)), INV),
    ("moe_combine", COMBINE, dict(tokens=1 << 24, n=1), INV),
    ("int8_grouped_gemm_blockscaled", GROUPED, dict(rows=1 << 20, a_rows=1 << 20, experts=1, n=2047 * 128), NODEV),
    ("int8_grouped_gemm_blockscaled", GROUPED, dict(rows=1 << 20, a_rows=1 << 20, experts=1, n=2048 * 128), INV),
    ("int8_grouped_gemm_blockscaled", GROUPED, dict(rows=1, a_rows=1, experts=1, n=(1 << 30) - 16, k=32), NODEV),
    ("int8_grouped_gemm_blockscaled", GROUPED, dict(rows=1, a_rows=1, experts=1, n=1 << 30, k=32), INV),
    ("w4a16_group_gemv", W4, dict(m=1, n=(1 << 30) - 16, k=32), NODEV),
    ("w4a16_group_gemv", W4, dict(m=1, n=1 << 30, k=32), INV),
    ("w4a16_group_gemv_experts", W4E, dict(rows=1, n=1 << 30, k=32), INV),
    ("w4a16_group_gemv_experts", W4E, dict(rows=1, n=1 << 30, k=32, silu_mul=1), NODEV),
])
def test_launch_limits(name, defaults, change, status):
    assert _call(name, defaults, **change) == status


@pytest.mark.parametrize("change, status", W4_BOTH + [
    (dict(rows=0), OK), (dict(experts=0), OK), (dict(rows=5), INV), (dict(experts=65537), INV), (dict(silu_mul=2), INV),
    (dict(row_index=FAKE, x_rows=0), INV),
    (dict(silu_mul=1, n=7), INV), (dict(offsets=None), NUL), (dict(offsets=_fake(2)), ALI),
    (dict(row_index=_fake(2)), ALI), (dict(rows=1 << 31), INV), (dict(x_rows=1 << 25), INV),
])
def test_w4_experts_refusals(change, status):
    assert _call("w4a16_group_gemv_experts", W4E, **change) == status


def test_route_plan_bounds():
    for experts in (1, 8, 64, 1000, 1024):
        for tokens in (0, 1, 31, 64, 65, 255, 4096, 8192, 8193, 100003, 1 << 24, (1 << 31) - 1):
            need = bsr.moe_route_ws_bytes(tokens, experts, 1)
            assert need <= 1024 * experts
            assert (need == 0) == (tokens <= 64)


def test_binding_rejects_shapes_types_and_devices():
    i8, i32, f32, bf = torch.int8, torch.int32, torch.float32, torch.bfloat16
    z = lambda *s, dt: torch.zeros(s, dtype=dt)  # noqa: E731
    a, w = z(4, 64, dt=i8), z(2, 8, 64, dt=i8)
    a_s, w_s = z(4, 2, dt=f32), z(2, 8, 2, dt=f32)
    off, out = z(3, dt=i32), z(4, 8, dt=bf)
    good = dict(a_i8=a, w_i8=w, a_scale=a_s, w_scale=w_s, offsets=off, out=out)
    for change, msg in [(dict(offsets=z(2, dt=i32)), "offsets: shape"), (dict(offsets=z(3, dt=torch.int64)), "int32"),
                        (dict(w_scale=z(2, 8, 3, dt=f32)), "w_scale: shape"), (dict(out=z(4, 7, dt=bf)), "out: shape"),
                        (dict(out=z(4, 8, dt=f32)), "out: dtype"), (dict(row_index=z(3, dt=i32)), "row_index: shape"),
                        (dict(a_i8=z(64, 4, dt=i8).t()), "contiguous"), ({}, "device tensor")]:
        with pytest.raises(ValueError, match=msg):
            bsr.int8_grouped_gemm_blockscaled(**{**good, **change})
    x, wp, sc = z(4, 64, dt=bf), z(8, 32, dt=torch.uint8), z(8, 2, dt=bf)
    good = dict(x_bf16=x, w_packed=wp, scale=sc, out=out)
    for change, msg in [(dict(scale=z(8, 3, dt=bf)), "groups"), (dict(scale=z(7, 2, dt=bf)), "scale: shape"),
                        (dict(scale=z(8, 2, dt=torch.int8)), "scale: dtype"), (dict(zero=z(8, 1, dt=torch.uint8)), "zero"),
                        (dict(w_packed=z(2, 8, 32, dt=torch.uint8), scale=z(2, 8, 2, dt=bf)), "two dimensions"),
                        ({}, "device tensor")]:
        with pytest.raises(ValueError, match=msg):
            bsr.w4a16_group_gemv(**{**good, **change})
    with pytest.raises(ValueError, match="three dimensions"):
        bsr.w4a16_group_gemv_experts(x, wp, sc, off, out)
    with pytest.raises(ValueError, match="out: shape"):
        bsr.w4a16_group_gemv_experts(x, z(2, 8, 32, dt=torch.uint8), z(2, 8, 2, dt=bf), off, out, silu_mul=True)
    ids, wt, ro = z(4, 2, dt=i32), z(4, 2, dt=f32), z(8, dt=i32)
    good = dict(logits=z(4, 2, dt=f32), ids=ids, weights=wt, offsets=off, row_token=ro, pos=ids)
    for change, msg in [(dict(logits=z(2, 4, dt=f32).t()), "logits"), (dict(weights=ids), "weights: dtype"),
                        (dict(row_token=z(7, dt=i32)), "row_token: shape"), (dict(ids=z(8, dt=i32)), "ids: shape"),
                        (dict(logits=z(4, 2, dt=torch.float64)), "logits: dtype"), ({}, "device tensor")]:
        with pytest.raises(ValueError, match=msg):
            bsr.moe_route(**{**good, **change})
    with pytest.raises(ValueError, match="residual: shape"):
        bsr.moe_combine(z(8, 8, dt=bf), ids, wt, out, residual=z(4, 7, dt=bf))
    with pytest.raises(ValueError, match="device tensor"):
        bsr.moe_combine(z(8, 8, dt=bf), ids, wt, out)


def test_binding_rejects_sizes_past_32_bits():
    """Sizes the ABI's 32-bit arguments cannot hold are refused, not cut (views of one element: no memory)."""
    big = 1 << 32

    def view(*shape, dtype=torch.bfloat16):
        return torch.zeros(1, dtype=dtype).expand(shape)
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    logits = torch.empty_strided((2, 4), (big + 4, 1), device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        bsr.moe_route(logits, *[torch.zeros(2, 2, dtype=t) for t in (i32, f32)], torch.zeros(5, dtype=i32),
                      torch.zeros(4, dtype=i32), torch.zeros(2, 2, dtype=i32))
    with pytest.raises(ValueError, match="32 bits"):
        bsr.int8_grouped_gemm_blockscaled(view(1, 32, dtype=torch.int8), view(1, big + 8, 32, dtype=torch.int8),
                                          view(1, 1, dtype=f32), view(1, big + 8, 1, dtype=f32),
                                          torch.zeros(2, dtype=i32), view(1, big + 8))
    with pytest.raises(ValueError, match="32 bits"):
        bsr.moe_combine(view(1, big + 8), torch.zeros(1, 1, dtype=i32), torch.zeros(1, 1), view(1, big + 8))
    with pytest.raises(ValueError, match="32 bits"):
        bsr.w4a16_group_gemv(view(1, 32), view(big + 8, 16, dtype=u8), view(big + 8, 1), view(1, big + 8))
    with pytest.raises(ValueError, match="32 bits"):
        bsr.w4a16_group_gemv_experts(view(big + 1, 32), view(1, 8, 16, dtype=u8), view(1, 8, 1),
                                     torch.zeros(2, dtype=i32), view(1, 8))


def test_oracle_route_by_hand():
    inf, nan = np.inf, np.nan
    x = np.array([[1.0, 3.0, 3.0, 2.0], [-inf] * 4, [nan, -inf, 0.0, -inf], [0.0, inf, -1.0, inf]])
    ids, w, off, tok, pos = moe.route(x, 2)
    assert ids.tolist() == [[1, 2], [-1, -1], [2, -1], [1, 3]]
    assert w.tolist() == [[0.5, 0.5], [0, 0], [1, 0], [0.5, 0.5]]
    assert off.tolist() == [0, 0, 2, 4, 5] and tok.tolist() == [0, 3, 0, 2, 3]
    assert pos.tolist() == [[0, 2], [-1, -1], [3, -1], [1, 4]]
    _, w, _, _, _ = moe.route(np.array([[-200.0, -201.0]]), 2, sigmoid=True)
    np.testing.assert_allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))]], rtol=1e-12)
    _, w, _, _, _ = moe.route(np.array([[0.0, 1.0, 2.0]]), 1, renorm=False, scale=3.0)
    np.testing.assert_allclose(w, [[3 * np.exp(2) / (1 + np.exp(1) + np.exp(2))]], rtol=1e-12)


def test_oracle_products_against_dense_matmul():
    rng = np.random.default_rng(5)
    a, w = rng.integers(-127, 128, (6, 64)).astype(np.int8), rng.integers(-127, 128, (3, 5, 64)).astype(np.int8)
    a_s, w_s = rng.random((6, 2)).astype(np.float32), rng.random((3, 5, 2)).astype(np.float32)
    offsets, index = np.array([1, 3, 3, 6]), np.array([0, 5, 2, -1, 6, 4, 0])
    y, t, cov = moe.grouped(a, w, a_s, w_s, offsets, index, 7)
    ad = a * np.repeat(a_s, 32, axis=1).astype(np.float64)
    wd = w * np.repeat(w_s, 32, axis=2).astype(np.float64)
    assert cov.tolist() == [False, True, True, True, True, True, False]
    for p, e, i in [(1, 0, 5), (2, 0, 2), (5, 2, 4)]:
        np.testing.assert_allclose(y[p], wd[e] @ ad[i], rtol=1e-12, atol=1e-9)
        assert (t[p] >= np.abs(y[p]) * (1 - 1e-12)).all()
    assert not y[[0, 3, 4, 6]].any()
    x = rng.standard_normal((4, 64))
    wp = rng.integers(0, 256, (5, 32)).astype(np.uint8)
    s, z = rng.random((5, 2)), rng.integers(0, 16, (5, 2)).astype(np.uint8)
    y, t = moe.w4_group(x, wp, s, z)
    for j in range(5):
        ref = sum(x[:, k] * s[j, k // 32] * ((int(wp[j, k // 2]) >> (4 * (k % 2))) % 16 - int(z[j, k // 32]))
                  for k in range(64))
        np.testing.assert_allclose(y[:, j], ref, rtol=1e-11, atol=1e-11)


def test_launch_plans(tmp_path):
    """The plans of the streamed kernels, the row-tile bound and the router's workspace, over sizes (host code)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "moe_plan_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", f"-I{root}/block_scaled_precision_requant_amd/csrc",
                    os.path.join(root, "tests", "host", "moe_plan_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    cases, many, gemv = map(int, r.stdout.split()[1:])
    assert cases > 100000 and 0 < many < cases and gemv > 100

"""What the expert-layer operators are measured on: their cases, their inputs,
the plain form of each in elementary torch operations and the definition in 64
bits.

Operators: the router (top-k of the router logits and the order of the routed
rows by expert), the products grouped by expert with int8 operands scaled per 32
elements, the matrix-vector products with 4-bit weights and group scales (dense
and by expert), and the weighted sum that brings the experts' rows back to their
tokens.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token's router logits while a single sequence is decoded: latency only
        dict(name="route_token", op="route", tokens=1, experts=64, top_k=8, type="bf16", score="softmax", renorm=True,
             scale=1.0, padded=0),
        # a serving batch, odd sizes, sigmoid scores with a routing factor
        dict(name="route_batch", op="route", tokens=333, experts=120, top_k=6, type="f32", score="sigmoid", renorm=True,
             scale=2.5, padded=5),
        # a long prefill over many small experts; the padded tokens' rows are masked out
        dict(name="route_prefill", op="route", tokens=16384, experts=256, top_k=8, type="f32", score="softmax",
             renorm=False, scale=1.0, padded=97),
        # one token decoded: eight experts of one row each, weights read once
        dict(name="grouped_token", op="grouped", tokens=1, experts=64, top_k=8, n=4096, k=2048, gather=True, skew=0.0,
             padded=0),
        # a decode batch: every expert has a few rows; the down projection, rows in expert order already
        dict(name="grouped_batch", op="grouped", tokens=48, experts=64, top_k=8, n=2048, k=4096, gather=False, skew=0.5,
             padded=0),
        # a short prefill with unevenly used experts
        dict(name="grouped_prefill", op="grouped", tokens=1537, experts=32, top_k=4, n=4096, k=2048, gather=True,
             skew=1.0, padded=33),
        # a long prefill over a few wide experts, gate and up stacked
        dict(name="grouped_prefill_wide", op="grouped", tokens=4096, experts=8, top_k=2, n=28672, k=4096, gather=True,
             skew=0.3, padded=0),
        # decode of one token through a 4-bit projection, zero points
        dict(name="w4_token", op="w4", rows=1, n=14336, k=4096, group=128, scale="bf16", zero=True),
        # decode of a batch through the down projection, symmetric codes
        dict(name="w4_batch", op="w4", rows=16, n=4096, k=14336, group=32, scale="f16", zero=False),
        # one token through its experts' gate and up projections with the SiLU product
        dict(name="w4_experts_token", op="w4_experts", tokens=1, experts=64, top_k=8, n=4096, k=2048, group=64,
             scale="bf16", zero=True, silu=True, gather=True, skew=0.0, padded=0),
        # a few decoded tokens back from expert order, with the residual stream
        dict(name="combine_token", op="combine", tokens=3, top_k=8, n=4096, residual=True, padded=0),
        # a prefill's rows back from expert order
        dict(name="combine_prefill", op="combine", tokens=4099, top_k=8, n=4096, residual=False, padded=21),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "grouped", "w4", "w4_experts", "combine"])
    if op == "route":
        experts = rng.choice([rng.randint(4, 256), 8, 64, 128, 256])
        tokens = _log(rng, 1, 16384)
        return dict(op=op, tokens=tokens, experts=experts, top_k=rng.randint(1, min(8, experts)),
                    type=rng.choice(["bf16", "f32", "f16"]), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), padded=rng.randint(0, tokens // 8))
    if op == "grouped":
        while True:
            experts = rng.choice([rng.randint(4, 128), 8, 16, 64])
            c = dict(op=op, tokens=_log(rng, 1, 4096), experts=experts, top_k=rng.randint(1, min(8, experts)),
                     n=rng.choice([_log(rng, 256, 28672), 32 * _log(rng, 8, 896)]), k=32 * _log(rng, 8, 256),
                     gather=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]), padded=0)
            c["padded"] = rng.randint(0, c["tokens"] // 8)
            if experts * c["n"] * c["k"] <= 940e6 and c["tokens"] * c["top_k"] * c["n"] * c["k"] <= 9.6e11:
                return c
    if op == "w4":
        k = 256 * _log(rng, 2, 56) + rng.choice([0, 128])
        return dict(op=op, rows=rng.randint(1, 16), n=_log(rng, 512, 14336), k=k, group=rng.choice([32, 64, 128, k]),
                    scale=rng.choice(["bf16", "f16", "f32"]), zero=rng.random() < 0.5)
    if op == "w4_experts":
        experts = rng.choice([rng.randint(4, 64), 8, 64])
        k = 128 * _log(rng, 4, 32)
        tokens = _log(rng, 1, 64)
        return dict(op=op, tokens=tokens, experts=experts, top_k=rng.randint(1, min(8, experts)),
                    n=2 * _log(rng, 128, 2048), k=k, group=rng.choice([32, 64, 128]),
                    scale=rng.choice(["bf16", "f16", "f32"]), zero=rng.random() < 0.5, silu=rng.random() < 0.5,
                    gather=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]), padded=rng.randint(0, tokens // 8))
    tokens = _log(rng, 1, 4099)
    return dict(op=op, tokens=tokens, top_k=rng.randint(1, 8), n=8 * _log(rng, 32, 512), residual=rng.random() < 0.5,
                padded=rng.randint(0, tokens // 8))


# ---- inputs ---------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _logits(g, tokens, experts, padded, skew=0.0):
    """Router logits: unit normal, experts of uneven popularity, padded tokens at -inf."""
    x = _randn(g, tokens, experts) + skew * _randn(g, 1, experts)
    if padded:
        x[torch.randperm(tokens, generator=g, device="cuda")[:padded]] = -math.inf
    return x


def _order(g, c):
    """Routed rows in expert order, as the router leaves them: (offsets [E+1], token of each row
    [T*k] (-1 behind the last), place of each (token, slot) [T, k]; -1 for padded tokens)."""
    t, k, e = c["tokens"], c["top_k"], c["experts"]
    x = _logits(g, t, e, c["padded"], c["skew"])
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k].int()
    ids[torch.isinf(x[:, 0])] = -1
    return _positions(ids, e)


def _positions(ids, experts):
    t, k = ids.shape
    flat = torch.where(ids < 0, experts, ids).reshape(-1)
    key, src = torch.sort(flat, stable=True)
    edges = torch.arange(experts + 1, device=ids.device, dtype=key.dtype)
    offsets = torch.searchsorted(key, edges).int()
    live = key < experts
    row_token = torch.where(live, src // k, -1).int()
    pos = torch.empty_like(flat, dtype=torch.int32)
    pos[src] = torch.where(live, torch.arange(t * k, device=ids.device), -1).int()
    return offsets, row_token, pos.reshape(t, k)


def _int8_rows(x):
    """int8 codes and a scale per 32 elements of the rows of x."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    s = b.abs().amax(-1) / 127
    return torch.round(b / s[..., None]).clamp(-127, 127).to(torch.int8).reshape(x.shape), s


def _w4(g, shape, n, k, group, scale, zero):
    lead = tuple(shape)
    w = torch.randint(0, 256, (*lead, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(*lead, n, k // group, generator=g, device="cuda") + 0.5) * (0.3 / math.sqrt(k))
    z = torch.randint(4, 12, (*lead, n, k // group), generator=g, device="cuda", dtype=torch.uint8) if zero else None
    return w, s.to(TYPES[scale]), z


def _inputs(c, seed):
    g = _gen(seed)
    s = dict(c)
    op = c["op"]
    if op == "route":
        s["logits"] = (2 * _logits(g, c["tokens"], c["experts"], c["padded"])).to(TYPES[c["type"]])
    elif op == "grouped":
        s["offsets"], s["row_token"], _ = _order(g, c)
        rows = c["tokens"] if c["gather"] else c["tokens"] * c["top_k"]
        s["a_i8"], s["a_scale"] = _int8_rows(_randn(g, rows, c["k"]))
        w = torch.empty(c["experts"], c["n"], c["k"], dtype=torch.int8, device="cuda")
        ws = torch.empty(c["experts"], c["n"], c["k"] // 32, device="cuda")
        for e in range(c["experts"]):
            w[e], ws[e] = _int8_rows(_randn(g, c["n"], c["k"]) / math.sqrt(c["k"]))
        s["w_i8"], s["w_scale"] = w, ws
    elif op == "w4":
        s["x"] = _randn(g, c["rows"], c["k"]).to(torch.bfloat16)
        s["w"], s["scale_t"], s["zero_t"] = _w4(g, (), c["n"], c["k"], c["group"], c["scale"], c["zero"])
    elif op == "w4_experts":
        s["offsets"], s["row_token"], _ = _order(g, c)
        s["x"] = _randn(g, c["tokens"] if c["gather"] else c["tokens"] * c["top_k"], c["k"]).to(torch.bfloat16)
        s["w"], s["scale_t"], s["zero_t"] = _w4(g, (c["experts"],), c["n"], c["k"], c["group"], c["scale"], c["zero"])
    else:
        s["pos"] = _order(g, dict(c, experts=16, skew=0.0))[2]
        s["y"] = _randn(g, c["tokens"] * c["top_k"], c["n"]).to(torch.bfloat16)
        s["weights"] = torch.softmax(_randn(g, c["tokens"], c["top_k"]), dim=1)
        s["residual_t"] = _randn(g, c["tokens"], c["n"]).to(torch.bfloat16) if c["residual"] else None
    return s


def prepare(case, seed):
    """Inputs, and the output and scratch tensors that a serving program keeps."""
    s = _inputs(case, seed)
    op = case["op"]

    def full(*shape, dtype=torch.bfloat16, value=0):
        return torch.full(shape, value, dtype=dtype, device="cuda")

    if op == "route":
        t, k = case["tokens"], case["top_k"]
        s["ids"], s["pos"] = full(t, k, dtype=torch.int32), full(t, k, dtype=torch.int32)
        s["weights"] = full(t, k, dtype=torch.float32)
        s["offsets"] = full(case["experts"] + 1, dtype=torch.int32)
        s["row_token"] = full(t * k, dtype=torch.int32, value=-1)
        s["workspace"] = full(1024 * case["experts"], dtype=torch.uint8)
    elif op == "w4":
        s["out"] = full(case["rows"], case["n"])
    elif op == "combine":
        s["out"] = full(case["tokens"], case["n"])
    else:
        s["out"] = full(case["tokens"] * case["top_k"], case["n"] // 2 if case.get("silu") else case["n"])
        s["bounds"] = s["offsets"].tolist()  # what the plain form slices by
    return s


# ---- plain forms ----------------------------------------------------------

def _plain_route(s):
    x = s["logits"].float()
    t, e = x.shape
    k = s["top_k"]
    v, ids = torch.sort(x, dim=1, descending=True, stable=True)
    v, ids = v[:, :k], ids[:, :k].int()
    live = v > -math.inf
    ids = torch.where(live, ids, -1)
    if s["score"] == "softmax":
        top = torch.where(live[:, :1], v[:, :1], 0.0)
        p = torch.exp(v - top)
        total = p.sum(1, keepdim=True) if s["renorm"] else torch.exp(x - top).sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-v))
        total = p.sum(1, keepdim=True) if s["renorm"] else torch.ones_like(p[:, :1])
    weights = torch.where(live, p / torch.where(total > 0, total, 1.0) * s["scale"], 0.0)
    offsets, row_token, pos = _positions(ids, e)
    return ids, weights, offsets, row_token, pos


def _plain_grouped(s):
    out = torch.zeros_like(s["out"])
    for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if lo == hi:
            continue
        rows = s["row_token"][lo:hi].long() if s["gather"] else slice(lo, hi)
        a = s["a_i8"][rows].float().reshape(hi - lo, -1, 32) * s["a_scale"][rows][..., None]
        w = s["w_i8"][e].float().reshape(s["n"], -1, 32) * s["w_scale"][e][..., None]
        out[lo:hi] = (a.reshape(hi - lo, -1) @ w.reshape(s["n"], -1).T).to(out.dtype)
    return out


def _plain_w4_weight(w, scale, zero, group):
    codes = torch.stack((w & 15, w >> 4), dim=-1).float().reshape(w.shape[0], -1, group)
    z = 8.0 if zero is None else zero.float()[..., None]
    return ((codes - z) * scale.float()[..., None]).reshape(w.shape[0], -1)


def _plain_w4(s):
    w = _plain_w4_weight(s["w"], s["scale_t"], s["zero_t"], s["group"])
    return (s["x"].float() @ w.T).to(torch.bfloat16)


def _plain_w4_experts(s):
    out = torch.zeros_like(s["out"])
    half = s["n"] // 2
    for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if lo == hi:
            continue
        x = (s["x"][s["row_token"][lo:hi].long()] if s["gather"] else s["x"][lo:hi]).float()
        y = x @ _plain_w4_weight(s["w"][e], s["scale_t"][e], None if s["zero_t"] is None else s["zero_t"][e],
                                 s["group"]).T
        if s["silu"]:
            gate, up = y[:, :half], y[:, half:]
            y = gate / (1 + torch.exp(-gate)) * up
        out[lo:hi] = y.to(out.dtype)
    return out


def _plain_combine(s):
    live = (s["pos"] >= 0)[..., None]
    y = torch.where(live, s["y"][s["pos"].clamp(min=0).long()].float(), 0.0)
    out = (y * s["weights"][..., None]).sum(1)
    if s["residual_t"] is not None:
        out = out + s["residual_t"].float()
    return out.to(torch.bfloat16)


# ---- one pass -------------------------------------------------------------

def run(s):
    op = s["op"]
    if not own:
        return {"route": _plain_route, "grouped": _plain_grouped, "w4": _plain_w4, "w4_experts": _plain_w4_experts,
                "combine": _plain_combine}[op](s)
    from block_scaled_precision_requant_amd import bsr
    if op == "route":
        bsr.moe_route(s["logits"], s["ids"], s["weights"], s["offsets"], s["row_token"], s["pos"], s["workspace"],
                      score=bsr.SCORE_SOFTMAX if s["score"] == "softmax" else bsr.SCORE_SIGMOID, renorm=s["renorm"],
                      scale=s["scale"])
        return s["ids"], s["weights"], s["offsets"], s["row_token"], s["pos"]
    if op == "grouped":
        bsr.int8_grouped_gemm_blockscaled(s["a_i8"], s["w_i8"], s["a_scale"], s["w_scale"], s["offsets"], s["out"],
                                          row_index=s["row_token"] if s["gather"] else None)
    elif op == "w4":
        bsr.w4a16_group_gemv(s["x"], s["w"], s["scale_t"], s["out"], zero=s["zero_t"])
    elif op == "w4_experts":
        bsr.w4a16_group_gemv_experts(s["x"], s["w"], s["scale_t"], s["offsets"], s["out"], zero=s["zero_t"],
                                     row_index=s["row_token"] if s["gather"] else None, silu_mul=s["silu"])
    else:
        bsr.moe_combine(s["y"], s["pos"], s["weights"], s["out"], residual=s["residual_t"])
    return s["out"]


def _used(c):
    """Experts that have rows, of evenly used ones."""
    return min(c["experts"], max(c["top_k"], round(c["experts"] *
                                                   (1 - (1 - c["top_k"] / c["experts"]) ** (c["tokens"] - c["padded"])))))


def work(c):
    op = c["op"]
    if op == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        return {"bytes": t * e * (4 if c["type"] == "f32" else 2) + 16 * t * k + 4 * (e + 1), "flops": 4 * t * e}
    if op == "grouped":
        rows = (c["tokens"] - c["padded"]) * c["top_k"]
        a_rows = c["tokens"] - c["padded"] if c["gather"] else rows
        return {"bytes": (a_rows + _used(c) * c["n"]) * (c["k"] + c["k"] // 8) + 2 * rows * c["n"],
                "flops": 2 * rows * c["n"] * c["k"]}
    if op == "combine":
        rows = (c["tokens"] - c["padded"]) * c["top_k"]
        return {"bytes": 2 * c["n"] * (rows + c["tokens"] * (2 if c["residual"] else 1)) + 8 * c["tokens"] * c["top_k"],
                "flops": 2 * rows * c["n"]}
    per_group = (4 if c["scale"] == "f32" else 2) + (1 if c["zero"] else 0)
    weight = c["n"] * (c["k"] // 2 + c["k"] // c["group"] * per_group)
    if op == "w4":
        rows, x_rows, used, cols = c["rows"], c["rows"], 1, c["n"]
    else:
        rows = (c["tokens"] - c["padded"]) * c["top_k"]
        x_rows = c["tokens"] - c["padded"] if c["gather"] else rows
        used, cols = _used(c), c["n"] // 2 if c["silu"] else c["n"]
    return {"bytes": used * weight + 2 * x_rows * c["k"] + 2 * rows * cols, "flops": 2 * rows * c["n"] * c["k"]}


# ---- the definition in 64 bits ----------------------------------------------

def _exact_route(s):
    x = s["logits"].double()
    t, e = x.shape
    k = s["top_k"]
    left = x.clone()
    ids = torch.full((t, k), -1, dtype=torch.int64, device=x.device)
    for j in range(k):
        best = left.max(1).values
        at = torch.argmax((left == best[:, None]).int(), dim=1)
        ids[:, j] = torch.where(best > -math.inf, at, -1)
        left[torch.arange(t, device=x.device), at] = -math.inf
    score = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, dim=1))
    w = torch.where(ids >= 0, score.gather(1, ids.clamp(min=0)), 0.0)
    if s["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    hits = torch.zeros(t * k, e, dtype=torch.int32, device=x.device)
    flat = ids.reshape(-1)
    routed = torch.nonzero(flat >= 0)[:, 0]
    hits[routed, flat[routed]] = 1
    count = hits.sum(0)
    offsets = torch.cat((count.new_zeros(1), torch.cumsum(count, 0)))
    rank = torch.cumsum(hits, 0, dtype=torch.int32)
    pos = torch.full((t * k,), -1, dtype=torch.int64, device=x.device)
    pos[routed] = offsets[flat[routed]] + rank[routed, flat[routed]] - 1
    row_token = torch.full((t * k,), -1, dtype=torch.int64, device=x.device)
    row_token[pos[routed]] = routed // k
    return ids.int(), w * s["scale"], offsets.int(), row_token.int(), pos.int().reshape(t, k)


def _exact_product(x, scaled_weight):
    """x [R, K] times the weight given in slices of K, summed in 64 bits."""
    y = 0
    for lo, hi, w in scaled_weight:
        y = y + x[:, lo:hi] @ w.t()
    return y


def _int8_slices(q, s, step=1024):
    k = q.shape[1]
    for lo in range(0, k, step):
        hi = min(k, lo + step)
        yield lo, hi, q[:, lo:hi].double() * torch.repeat_interleave(s[:, lo // 32:hi // 32].double(), 32, dim=1)


def _w4_slices(w, scale, zero, group, step=1024):
    k = 2 * w.shape[1]
    at = torch.arange(k, device=w.device)
    for lo in range(0, k, step):
        i = at[lo:lo + step]
        code = (w[:, i // 2].int() >> (4 * (i % 2))) & 15
        z = 8 if zero is None else zero[:, i // group].int()
        yield lo, lo + len(i), (code - z).double() * scale[:, i // group].double()


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "w4":
        return _exact_product(s["x"].double(), _w4_slices(s["w"], s["scale_t"], s["zero_t"], case["group"]))
    if op == "combine":
        y = torch.cat((s["y"].double(), torch.zeros(1, case["n"], dtype=torch.float64, device="cuda")))
        out = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device="cuda")
        for j in range(case["top_k"]):
            out += s["weights"][:, j:j + 1].double() * y[s["pos"][:, j].long()]
        return out if s["residual_t"] is None else out + s["residual_t"].double()
    cols = case["n"] // 2 if case.get("silu") else case["n"]
    out = torch.zeros(case["tokens"] * case["top_k"], cols, dtype=torch.float64, device="cuda")
    bounds = s["offsets"].tolist()
    for e in range(case["experts"]):
        p = torch.arange(bounds[e], bounds[e + 1], device="cuda")
        if not len(p):
            continue
        i = s["row_token"][p].long() if case["gather"] else p
        if op == "grouped":
            a = s["a_i8"][i].double() * torch.repeat_interleave(s["a_scale"][i].double(), 32, dim=1)
            out[p] = _exact_product(a, _int8_slices(s["w_i8"][e], s["w_scale"][e]))
        else:
            zero = None if s["zero_t"] is None else s["zero_t"][e]
            y = _exact_product(s["x"][i].double(), _w4_slices(s["w"][e], s["scale_t"][e], zero, case["group"]))
            if case["silu"]:
                y = y[:, :cols] * torch.sigmoid(y[:, :cols]) * y[:, cols:]
            out[p] = y
    return out

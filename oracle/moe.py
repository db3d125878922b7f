"""CPU oracle of the expert-layer operators -- TEST INFRASTRUCTURE ONLY.

Plain NumPy from the definitions, in 64 bits; shares no code with the HIP
library.  Products come with the sum of their terms' magnitudes, which the FP32
error bounds scale with (oracle/compare.py).
"""
import numpy as np


def bf16_f64(bits):
    u = np.ascontiguousarray(bits).view(np.uint16).astype(np.uint32) << np.uint32(16)
    return u.view(np.float32).astype(np.float64)


def route(logits, top_k, sigmoid=False, renorm=True, scale=1.0):
    """logits [T, E] float -> ids, weights (float64), offsets, row_token (routed rows only), pos."""
    x = np.asarray(logits, dtype=np.float64)
    t, e = x.shape
    ids = np.full((t, top_k), -1, dtype=np.int32)
    weights = np.zeros((t, top_k))
    for i in range(t):
        cand = [j for j in range(e) if x[i, j] > -np.inf]          # drops -inf and NaN
        cand.sort(key=lambda j: (-x[i, j], j))
        take = cand[:top_k]
        if not take:
            continue
        ids[i, :len(take)] = take
        if sigmoid:
            v = x[i, take]
            # log sigmoid, so that renormalised rows of very negative logits keep their ratios
            logp = np.where(v >= 0, -np.log1p(np.exp(-np.abs(v))), v - np.log1p(np.exp(-np.abs(v))))
            logp = np.where(np.isposinf(v), 0.0, logp)
            p = np.exp(logp - logp.max()) if renorm else np.exp(logp)
            w = p / p.sum() if renorm else p
        else:
            v = x[i, cand]
            with np.errstate(invalid="ignore"):
                p = np.exp(np.where(v == v.max(), 0.0, v - v.max()))
            w = p[:len(take)] / (p[:len(take)].sum() if renorm else p.sum())
        weights[i, :len(take)] = w * scale
    offsets = np.zeros(e + 1, dtype=np.int32)
    row_token, pos = [], np.full((t, top_k), -1, dtype=np.int32)
    for j in range(e):
        offsets[j] = len(row_token)
        for i, s in zip(*np.nonzero(ids == j)):
            pos[i, s] = len(row_token)
            row_token.append(i)
    offsets[e] = len(row_token)
    return ids, weights, offsets, np.array(row_token, dtype=np.int32), pos


def _sources(offsets, row_index, a_rows, rows):
    """[(expert, output rows, operand rows)] with the documented clamps; operand -1: a row of zeros."""
    out = []
    for e in range(len(offsets) - 1):
        lo = min(max(int(offsets[e]), 0), rows)
        hi = min(max(int(offsets[e + 1]), lo), rows)
        if hi > lo:
            p = np.arange(lo, hi)
            i = p if row_index is None else np.asarray(row_index)[p]
            out.append((e, p, np.where((i >= 0) & (i < a_rows), i, -1)))
    return out


def _rows(x, i):
    return np.where((i >= 0)[:, None], x[np.maximum(i, 0)], 0.0) if len(x) else np.zeros((len(i), x.shape[1]))


def grouped(a, w, a_s, w_s, offsets, row_index, rows):
    """(y [rows, N], T [rows, N], covered [rows]) of the grouped int8 product."""
    n = w.shape[1]
    y, t, covered = np.zeros((rows, n)), np.zeros((rows, n)), np.zeros(rows, dtype=bool)
    nb = a.shape[1] // 32
    for e, p, i in _sources(offsets, row_index, len(a), rows):
        ai = _rows(a.astype(np.float64), i).reshape(len(p), nb, 32)
        asc = _rows(a_s.astype(np.float64), i)
        for b in range(nb):
            part = ai[:, b] @ w[e, :, 32 * b:32 * b + 32].astype(np.float64).T
            part *= asc[:, b:b + 1] * w_s[e, :, b].astype(np.float64)
            y[p] += part
            t[p] += np.abs(part)
        covered[p] = True
    return y, t, covered


def w4_weight(w_packed, scale, zero):
    """(codes, zeros, scales) [N, K] float64 of a 4-bit weight; scale already float."""
    codes = np.stack((w_packed & 15, w_packed >> 4), axis=-1).reshape(w_packed.shape[0], -1).astype(np.float64)
    rep = codes.shape[1] // scale.shape[1]
    z = np.full(scale.shape, 8.0) if zero is None else zero.astype(np.float64)
    return codes, np.repeat(z, rep, axis=1), np.repeat(scale.astype(np.float64), rep, axis=1)


def w4_group(x, w_packed, scale, zero=None):
    """(y, T): the product, and the magnitudes |x| * |scale| * (32 + c + z) its FP32 evaluation rounds at."""
    c, z, s = w4_weight(w_packed, scale, zero)
    return x @ (s * (c - z)).T, np.abs(x) @ (np.abs(s) * (32 + c + z)).T


def w4_terms(k, group):
    """Roundings of one output relative to T: the sums over a group inside the matrix core (group products each
    for P and X, which T's terms cover together), (16 + z) * X taken off (1), the scale (1), one addition per
    group, at most 16 partial sums of the waves (16)."""
    group = k if group == 0 else group
    return group + k // group + 18


def w4_experts(x, w_packed, scale, zero, offsets, row_index, rows):
    n = w_packed.shape[1]
    y, t, covered = np.zeros((rows, n)), np.zeros((rows, n)), np.zeros(rows, dtype=bool)
    for e, p, i in _sources(offsets, row_index, len(x), rows):
        y[p], t[p] = w4_group(_rows(x, i), w_packed[e], scale[e], None if zero is None else zero[e])
        covered[p] = True
    return y, t, covered


def silu_mul(y, t, terms):
    """(out, B): SiLU(gate) * up of the halves of y, and how far FP32 halves that are off by terms * 2^-24 * t
    can take it: |silu'| <= 1.1, |silu(g)| <= |g|, and 8 roundings of the epilogue itself."""
    h = y.shape[1] // 2
    g, u = y[:, :h], y[:, h:]
    d = (terms + 2) * 2.0 ** -24 * t
    dg, du = d[:, :h], d[:, h:]
    sg = g / (1 + np.exp(-np.clip(g, -700, 700)))
    out = sg * u
    return out, 1.1 * dg * (np.abs(u) + du) + np.abs(sg) * du + 8 * 2.0 ** -24 * np.abs(out)


def combine(y, pos, weights, residual=None):
    """(out, T) of the weighted sum."""
    rows, n = y.shape
    t, k = pos.shape
    out = np.zeros((t, n)) if residual is None else residual.copy()
    mag = np.abs(out)
    for i in range(t):
        for j in range(k):
            if 0 <= pos[i, j] < rows:
                term = float(weights[i, j]) * y[pos[i, j]]
                out[i] += term
                mag[i] += np.abs(term)
    return out, mag

"""Plain 64-bit forms of the 8-bit operators (test infrastructure; shares no code with the
HIP path): rows of codes with one scale, the norm with an 8-bit output, scored selection,
products of codes and the experts' FFN over them.

A product's error bound comes with it where a rounding to codes lies inside: the codes of
values within `border` of a rounding border may be one step off, and nothing else may.
"""
from __future__ import annotations

import numpy as np


def quant_rows(v: np.ndarray):
    """Codes (as float64) and scales of the rows of v, and v in units of its scale."""
    top = np.abs(v).max(axis=-1)
    scale = top / 127.0
    units = np.divide(v * 127.0, top[..., None], out=np.zeros_like(v), where=top[..., None] > 0)
    return np.rint(units), scale, units


def norm(x: np.ndarray, residual, weight: np.ndarray, eps: float):
    """(v, n): the sum and the normed rows, float64."""
    v = x.astype(np.float64) + (0.0 if residual is None else residual.astype(np.float64))
    n = v / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps) * weight.astype(np.float64)
    return v, n


def linear(a, a_scale, w, w_scale) -> np.ndarray:
    """a [M, K], w [N, K] codes with their rows' scales -> [M, N] float64."""
    prod = a.astype(np.float64) @ w.astype(np.float64).T   # integers below 2^53: exact
    return prod * a_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)[None, :]


def scores(logits: np.ndarray, sigmoid: bool) -> np.ndarray:
    """float64 scores [T, E]; -inf logits score 0, NaN counts as -inf, +inf share a softmax."""
    out = np.zeros(logits.shape)
    for t, row in enumerate(logits.astype(np.float64)):
        row = np.where(np.isnan(row), -np.inf, row)
        if sigmoid:
            neg = np.exp(-np.abs(row))
            out[t] = np.where(row >= 0, 1.0, neg) / (1.0 + neg)
        elif np.isposinf(row).any():
            out[t] = np.isposinf(row) / np.isposinf(row).sum()
        elif np.isfinite(row).any():
            p = np.exp(row - row[np.isfinite(row)].max())
            out[t] = p / p.sum()
    return out


def _first(values, n, allowed):
    """Indices of the n largest allowed values, in order, the lowest index among equals."""
    got = []
    for _ in range(n):
        best = None
        for i, v in enumerate(values):
            if allowed[i] and i not in got and (best is None or v > values[best]):
                best = i
        got.append(best)
    return got


def route_scored(logits, bias, k, sigmoid=False, n_groups=1, topk_groups=1, top2=True,
                 renormalise=True, scale=1.0):
    """(topk_idx [T, k], topk_w [T, k] float64) by the written rule."""
    T, E = logits.shape
    s = scores(logits, sigmoid)
    with np.errstate(invalid="ignore"):
        choice = s.astype(np.float32) + (np.float32(0) if bias is None else bias.astype(np.float32))
    choice = np.where(np.isnan(choice), np.float32(-np.inf), choice).astype(np.float32)
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    gs = E // n_groups
    for t in range(T):
        allowed = [True] * E
        if topk_groups < n_groups:
            worth = []
            for g in range(n_groups):
                part = np.sort(choice[t, g * gs:(g + 1) * gs])[::-1]
                with np.errstate(invalid="ignore"):
                    v = np.float32(part[0] + part[1]) if top2 else part[0]
                worth.append(np.float32(-np.inf) if np.isnan(v) else v)
            keep = _first(worth, topk_groups, [True] * n_groups)
            allowed = [e // gs in keep for e in range(E)]
        idx[t] = _first(choice[t], k, allowed)
        w[t] = s[t, idx[t]]
        if renormalise:
            w[t] = w[t] / max(w[t].sum(), 1e-30)
    return idx, w * scale


#: An fp32 h differs from the exact one by less than this share (int32 -> fp32, four scale
#: products, exp2, 1 + exp2, reciprocal, two products: 12 roundings of at most 2^-23 with the
#: hardware functions' 1 ulp, and the exponent's rounding times |z| <= 32 of the tests).
H_SHARE = 12 * 2.0 ** -23 + 32 * 2.0 ** -23


def expert_ffn(x, x_scale, gate, up, down):
    """(out, bound): the FFN of rows of codes x by (codes, scales) matrices, with h held as
    codes, and how far fp32 h can move each output by codes that cross a rounding border."""
    g, u = linear(x, x_scale, *gate), linear(x, x_scale, *up)
    h = g / (1.0 + np.exp(-g)) * u
    q, s, units = quant_rows(h)
    out = linear(q, s, *down)
    wd = np.abs(down[0].astype(np.float64) * down[1].astype(np.float64)[:, None])
    # two shares: h's own error and its row maximum's, in code units at most 127 each
    near = np.abs(np.abs(units - np.trunc(units)) - 0.5) <= 2 * H_SHARE * np.abs(units) + 1e-12
    bound = (near * s[:, None]) @ wd.T + np.abs(out) * H_SHARE
    return out, bound


def layer(x, x_scale, idx, w, mats, sh_mats):
    """(expert_out [T*k, H] by assignment, its bound, shared_out or None, its bound, y)."""
    T, k = idx.shape
    H = mats[2][0].shape[1]
    out, bound = np.zeros((T * k, H)), np.zeros((T * k, H))
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        part = [(m[0][e], m[1][e]) for m in mats]
        out[t * k + j], bound[t * k + j] = expert_ffn(x[t], x_scale[t], *part)
    y = (out.reshape(T, k, H) * w[:, :, None]).sum(1)
    sh, sh_bound = None, None
    if sh_mats is not None:
        sh, sh_bound = expert_ffn(x, x_scale, *[(m[0][0], m[1][0]) for m in sh_mats])
        y = y + sh
    return out, bound, sh, sh_bound, y

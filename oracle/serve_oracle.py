"""Plain 64-bit forms of the operators of a step that serves several requests at once (test
infrastructure; shares no code with the HIP path): the 4-bit layer over given selections, the
projection with an adapter for each row, and log probabilities of rows of logits."""
from __future__ import annotations

import numpy as np

from .moe_oracle import dequant, swiglu_ffn


def batch_layer(x: np.ndarray, idx: np.ndarray, w: np.ndarray, mats, shared, gate) -> np.ndarray:
    """x [T, H], the selection idx, w [T, k], mats (gate, up, down) 4-bit sets, shared three more
    or None, gate [T] or None -> y [T, H], nothing rounded."""
    x = x.astype(np.float64)
    y = np.zeros((x.shape[0], x.shape[1]))

    def ffn(rows, of, e):
        return swiglu_ffn(rows, *[dequant(m.codes[e], m.scales[e], m.biases[e]) for m in of])

    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        y[t] += ffn(x[t], mats, e) * w[t, j][:, None]
    if shared is not None:
        sh = ffn(x, shared, 0)
        y += sh if gate is None else sh * gate.astype(np.float64)[:, None]
    return y


def linear_lora(a, a_scale, w, w_scale, A, B, scales, adapter):
    """(out, size): codes a [M, K], w [N, K] with their rows' scales, adapters A [n, R, K],
    B [n, N, R] with scales [n], adapter [M] (outside 0 .. n - 1: none) -> out [M, N]; and the
    sum of the magnitudes of the adapters' products, which bounds their roundings."""
    a = a.astype(np.float64)
    out = a @ w.astype(np.float64).T * w_scale.astype(np.float64)
    size = np.zeros_like(out)
    for m, j in enumerate(adapter):
        if 0 <= j < len(A):
            Aj, Bj, s = A[j].astype(np.float64), B[j].astype(np.float64), float(scales[j])
            out[m] += s * (Bj @ (Aj @ a[m]))
            size[m] = abs(s) * (np.abs(Bj) @ (np.abs(Aj) @ np.abs(a[m])))
    sa = a_scale.astype(np.float64)[:, None]
    return out * sa, size * np.abs(sa)


def logprobs(z: np.ndarray, targets, n: int):
    """(logprob [T], entropy [T], top_idx [T, n], top_logprob [T, n]) of logits z [T, V].  A target
    outside 0 .. V - 1 gives 0; a row of -inf alone has log probabilities -inf and entropy 0; a
    row with a NaN or +inf has NaN for all of them.  NaN counts as -inf in the order."""
    z = z.astype(np.float64)
    T, V = z.shape
    lp, ent = np.zeros(T), np.zeros(T)
    idx, top = np.zeros((T, n), np.int32), np.zeros((T, n))
    for t in range(T):
        row = z[t]
        best = np.max(np.where(np.isnan(row), -np.inf, row))
        if np.isnan(row).any() or best == np.inf:
            all_lp, ent[t] = np.full(V, np.nan), np.nan
        elif best == -np.inf:
            all_lp = row
        else:
            all_lp = row - best - np.log(np.exp(row - best).sum())
            p = np.exp(all_lp)
            ent[t] = -(p[p > 0] * all_lp[p > 0]).sum()
        order = np.argsort(-np.where(np.isnan(row), -np.inf, row), kind="stable")[:n]
        idx[t], top[t] = order, all_lp[order]
        if targets is not None:
            lp[t] = all_lp[targets[t]] if 0 <= targets[t] < V else 0.0
    return lp, ent, idx, top

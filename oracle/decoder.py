"""Plain 64-bit oracle of the 8-bit decoder-layer operators: the norm with its
8-bit output, the shared projection in 8 bits beside the adapters, and a whole
MoE layer.  Per-token and per-expert loops in numpy, written from the formulas
in include/mlora.h; shares no code with the HIP path.

The functions that end in ``_mag`` give, beside each value, the sum of the
magnitudes of the terms it is made of: what a rounding-error bound multiplies.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import numpy as np

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


def rms_norm(x, weight, eps, residual=None) -> Tuple[np.ndarray, np.ndarray]:
    """(h, v): h = x + residual, v = h * weight / sqrt(mean(h^2) + eps)."""
    h = x if residual is None else x + residual
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight


def row_scale(v) -> np.ndarray:
    """Scale of each row in 8 bits: the largest magnitude over 448, 1 for zeros."""
    top = np.abs(v).max(1) if v.shape[1] else np.zeros(v.shape[0])
    return np.where(top == 0, 1.0, np.maximum(top / E4M3_MAX, SCALE_MIN))


def linear_fp8_mag(x8, x_scale, W8, w_scale, x, ids, A: Sequence[np.ndarray],
                   B: Sequence[np.ndarray], ranks: Sequence[int],
                   slice_sizes: Sequence[int]) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """y = (x8 xs)(W8 ws)^T + the adapter's delta per token, with the term
    magnitudes of the base product and of the delta; A[i] [n_sl * r, K]
    slice-major, B[i] [N, r]."""
    xd, Wd = x8 * x_scale[:, None], W8 * w_scale[:, None]
    y, mag = xd @ Wd.T, np.abs(xd) @ np.abs(Wd).T
    dmag = np.zeros_like(y)
    for m in range(x.shape[0]):
        i = int(ids[m])
        if i < 0 or i >= len(ranks) or ranks[i] == 0:
            continue
        r, n0 = ranks[i], 0
        for s, n in enumerate(slice_sizes):
            a, b = A[i][s * r:(s + 1) * r], B[i][n0:n0 + n]
            y[m, n0:n0 + n] += b @ (a @ x[m])
            dmag[m, n0:n0 + n] += np.abs(b) @ (np.abs(a) @ np.abs(x[m]))
            n0 += n
    return y, mag, dmag


def route(x, router, topk: int, renormalize: bool) -> Tuple[np.ndarray, np.ndarray]:
    """Chosen experts [M, topk] (largest logit first, ties to the lowest
    expert) and their weights."""
    logits = x @ router.T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :topk]
    e = np.exp(logits - logits.max(1, keepdims=True))
    w = np.take_along_axis(e / e.sum(1, keepdims=True), ids, 1)
    return ids, w / w.sum(1, keepdims=True) if renormalize else w


def moe_layer_mag(x, ids, weights, W_gu, W_d, token_ids, adapters: Optional[List],
                  enabled, step: float, unit: float) -> Tuple[np.ndarray, np.ndarray]:
    """(out, bound): the layer's output for a given routing, and a bound on
    the error of a computation that rounds h to half a `step` relative and
    every sum of products to `unit` of the sum of its terms' magnitudes.
    adapters: None or (A_gu, B_gu, A_d, B_d), the hidden-side stacks with one
    or E expert slots."""
    M, H = x.shape
    I = W_d.shape[2]
    out, bound = np.zeros((M, H)), np.zeros((M, H))
    for m in range(M):
        l = int(token_ids[m]) if adapters is not None else -1
        if l >= 0 and (l >= len(enabled) or not enabled[l]):
            l = -1
        for e, c in zip(ids[m], weights[m]):
            gu, mag = W_gu[e] @ x[m], np.abs(W_gu[e]) @ np.abs(x[m])
            if l >= 0:
                A_gu, B_gu, A_d, B_d = adapters
                a, b = A_gu[l, e if A_gu.shape[1] > 1 else 0], B_gu[l, e]
                gu = gu + b @ (a @ x[m])
                mag = mag + np.abs(b) @ (np.abs(a) @ np.abs(x[m]))
            g, u, dg, du = gu[:I], gu[I:], unit * mag[:I], unit * mag[I:]
            s = g / (1 + np.exp(-g))
            h = c * s * u
            # |silu'| <= 1.1
            dh = c * (1.1 * dg * (np.abs(u) + du) + np.abs(s) * du) + (step + unit) * np.abs(h)
            out[m] += W_d[e] @ h
            bound[m] += np.abs(W_d[e]) @ (dh + unit * np.abs(h))
            if l >= 0:
                a, b = A_d[l, e], B_d[l, e if B_d.shape[1] > 1 else 0]
                out[m] += b @ (a @ h)
                bound[m] += np.abs(b) @ (np.abs(a) @ (dh + unit * np.abs(h)))
    return out, bound

"""Plain 64-bit oracle of the experts' base products and of rows in 8-bit
integers: loops in numpy, written from the formulas in include/mlora.h; shares
no code with the HIP path."""
from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

INT8_MAX = 127.0
SCALE_MIN = 2.0 ** -126


def group(topk_ids, E: int) -> Tuple[np.ndarray, np.ndarray]:
    """(pairs, offsets): pair indices m * topk + k by ascending expert, equal
    experts in their own order, ids outside [0, E) last; where each expert's
    begin, and the end of the last."""
    shares = [[] for _ in range(E + 1)]
    for f, e in enumerate(np.asarray(topk_ids).reshape(-1)):
        shares[e if 0 <= e < E else E].append(f)
    pairs = [f for share in shares for f in share]
    offsets = np.cumsum([0] + [len(share) for share in shares[:E]])
    return np.array(pairs, dtype=np.int32), offsets.astype(np.int32)


def grouped_linear_mag(topk_ids, x, W, pair_rows: bool, x_scale=None,
                       w_scale=None) -> Tuple[np.ndarray, np.ndarray]:
    """y[f] = W[e] x[r] (with the scales) for every pair f whose expert e lies in
    [0, E), NaN for the others, and the sums of the terms' magnitudes."""
    M, topk = np.asarray(topk_ids).shape
    E, N, _ = W.shape
    y, mag = np.full((M * topk, N), np.nan), np.full((M * topk, N), np.nan)
    ids = np.asarray(topk_ids).reshape(-1)
    for e in range(E):
        f = np.flatnonzero(ids == e)
        if f.size == 0:
            continue
        r = f if pair_rows else f // topk
        y[f], mag[f] = x[r] @ W[e].T, np.abs(x[r]) @ np.abs(W[e]).T
        if x_scale is not None:         # after the sums: those of integers are exact here too
            scale = x_scale[r][:, None] * w_scale[e][None, :]
            y[f], mag[f] = y[f] * scale, mag[f] * scale
    return y, mag


def row_scale_int8(v) -> np.ndarray:
    """Scale of each row: the largest magnitude over 127 rounded to fp32, 1 for
    zeros, at least the smallest normal number."""
    top = np.abs(v).max(1)
    return np.where(top == 0, 1.0, np.maximum((top / INT8_MAX).astype(np.float32).astype(np.float64), SCALE_MIN))


def quantize_int8(v, scale: Optional[np.ndarray] = None) -> Tuple[np.ndarray, np.ndarray]:
    """(q, scale): v / scale to the nearest integer, ties to even.  v holds fp32
    values: a quotient that is no tie lies further from one than the rounding of
    its 53 bits (v - (n + 1/2) scale is a multiple of 2^-25 of the scale)."""
    s = row_scale_int8(v) if scale is None else scale
    return np.rint(v / s[:, None]), s

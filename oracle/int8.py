"""8-bit rows and products, in exact arithmetic (test infrastructure).

    quantize: amax = max |x_i|, scale = amax / 127, q_i = round-half-even(127 x_i / amax), on fractions;
    product:  Y[r, o] = (sum_i xq[r, i] wq[o, i]) * xs[r] * ws[o], the sum in int64, the rest in float64.

Pins (tests/test_oracle_int8_rows.py): hand-worked ties and rows; the half-step bound; a naive product loop.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def quantize_row(x):
    """(q int list, scale float64) of one row of finite or non-finite values."""
    x = [float(v) for v in x]
    if not all(np.isfinite(x)):
        return [0] * len(x), float("nan")
    amax = max(abs(v) for v in x)
    if amax == 0.0:
        return [0] * len(x), 0.0
    top = Fraction(amax)
    return [round(Fraction(v) * 127 / top) for v in x], float(Fraction(amax) / 127)   # round(): halves to even


def quantize(x):
    rows = [quantize_row(r) for r in np.asarray(x, np.float64).reshape(-1, np.shape(x)[-1])]
    return np.array([r[0] for r in rows], np.int8), np.array([r[1] for r in rows], np.float64)


def gemm(xq, xs, wq, ws):
    """float64 [M, m]."""
    acc = np.asarray(xq, np.int64) @ np.asarray(wq, np.int64).T
    return acc.astype(np.float64) * np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)


def gemm_grouped(xq, xs, wq, ws, offsets, order, pairs_per_row, y):
    """y float64 [pairs, m] with the rows of the routed pairs filled in (the others as they were)."""
    y = np.array(y, np.float64)
    for e in range(len(offsets) - 1):
        for j in range(offsets[e], offsets[e + 1]):
            p = order[j]
            t = p // pairs_per_row
            y[p] = gemm(xq[t:t + 1], xs[t:t + 1], wq[e], ws[e])[0]
    return y

"""e4m3 rows, layers and products with a scale for each block of 128 (test infrastructure).

    quantize: amax = max |x_i| of a block, scale = amax / 448, q_i = the e4m3 value nearest to 448 x_i / amax, ties to the
              even code. The step of a value is the number of borders between neighbouring magnitudes that lie below it, each
              comparison 896 |x| against (v_k + v_{k+1}) amax multiplied out; both sides are exact in float64 for values of up to
              48 significant bits (a product of two binary32).
    product:  Y[r, o] = sum_b xs[r, b] ws[o / 128, b] sum_{i in b} xq[r, i] wq[o, i], in float64.

Pins (tests/test_oracle_fp8.py): the type's values from its definition, fractions, hand-worked ties, a naive product loop.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def magnitudes():
    """The type's values from 0 to 448 by code: i / 512 below code 8, then 8 to a binade."""
    return np.array([c * 2.0 ** -9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10) for c in range(127)])


def codes_near(v, amax):
    """Codes (uint8) of the e4m3 values nearest to 448 v / amax; v float64 [..., k], amax > 0 broadcast against it."""
    m = magnitudes()
    a = 896.0 * np.abs(v)
    code = np.zeros(np.broadcast(v, amax).shape, np.int64)
    for k in range(126):
        border = (m[k] + m[k + 1]) * amax
        code += (a > border) | ((a == border) & (k % 2 == 1))
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def values(codes):
    """float64 values of e4m3 codes (NaN where the code is one)."""
    c = np.asarray(codes, np.uint8)
    m = np.append(magnitudes(), np.nan)[c & 0x7F]
    return np.where(c & 0x80, -m, m)


def _blocked(x, axis):
    pad = -x.shape[axis] % BLOCK
    widths = [(0, 0)] * x.ndim
    widths[axis] = (0, pad)
    return np.pad(x, widths)


def quantize(x, block_rows=1):
    """(codes uint8 [rows, n], scales float64 [rows / block_rows, n / 128], rounded up)."""
    x = np.asarray(x, np.float64)
    rows, n = x.shape
    p = _blocked(x, 1)
    if block_rows != 1:
        p = _blocked(p, 0)
    b = p.reshape(p.shape[0] // block_rows, block_rows, p.shape[1] // BLOCK, BLOCK).transpose(0, 2, 1, 3)
    good = np.isfinite(b).all((2, 3))
    amax = np.abs(np.where(good[:, :, None, None], b, 0.0)).max((2, 3))
    codes = codes_near(np.where(good[:, :, None, None], b, 0.0), np.where(amax > 0, amax, 1.0)[:, :, None, None])
    codes = np.where(good[:, :, None, None], codes, 0).astype(np.uint8)
    return codes.transpose(0, 2, 1, 3).reshape(p.shape)[:rows, :n], np.where(good, amax / 448.0, np.nan)


def block_sums(xq, wq):
    """sum over each block of the inner axis: float64 [M, m, blocks], of values (not codes)."""
    x, w = _blocked(np.asarray(xq, np.float64), 1), _blocked(np.asarray(wq, np.float64), 1)
    x, w = x.reshape(x.shape[0], -1, BLOCK), w.reshape(w.shape[0], -1, BLOCK)
    return np.stack([x[:, b] @ w[:, b].T for b in range(x.shape[1])], 2)


def scale_products(xs, ws, m):
    """xs[r, b] * ws[o / 128, b]: float64 [M, m, blocks]."""
    owner = np.arange(m) // BLOCK
    return np.asarray(xs, np.float64)[:, None, :] * np.asarray(ws, np.float64)[owner][None]


def gemm(xq, xs, wq, ws):
    return (block_sums(xq, wq) * scale_products(xs, ws, len(wq))).sum(2)


def gemm_grouped(xq, xs, wq, ws, offsets, order, pairs_per_row, y):
    """y float64 [pairs, m] with the rows of the routed pairs filled in (the others as they were)."""
    y = np.array(y, np.float64)
    for e in range(len(offsets) - 1):
        p = np.asarray(order[offsets[e]:offsets[e + 1]], np.int64)
        if len(p):
            t = p // pairs_per_row
            y[p] = gemm(xq[t], xs[t], wq[e], ws[e])
    return y

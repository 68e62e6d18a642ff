"""Root-mean-square norm with the residual's addition and 8-bit outputs (test infrastructure).

    h = round(x + residual), r = 1 / sqrt(mean h^2 + eps), v = h w;  y = v r, or the steps of v by rows (int8) or by 128
    values (e4m3) with the scales amax r / 127 or amax r / 448.

All in float64; the sum x + residual is rounded to binary32 and then to the residual's type, as the operator defines it. Pins
(tests/test_oracle_fp8.py): hand-worked rows, fractions for the steps.
"""
from __future__ import annotations

import numpy as np

from . import fp8


def round_to(v, kind):
    """float64 values rounded to "float32", "float16" or "bfloat16", halves to even."""
    v = np.asarray(v, np.float64)
    with np.errstate(over="ignore"):
        if kind == "float32":
            return v.astype(np.float32).astype(np.float64)
        if kind == "float16":
            return v.astype(np.float16).astype(np.float64)
    fine = np.isfinite(v) & (v != 0)
    e = np.frexp(np.where(fine, v, 1.0))[1] - 1
    step = np.ldexp(1.0, np.maximum(e, -126) - 7)
    r = np.rint(np.where(fine, v, 0.0) / step) * step
    r = np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, r), r)
    return np.where(fine, r, v)


def steps127(v):
    """(whole numbers nearest to 127 v / amax row by row, halves to even, amax): float64 [rows, n] of finite values, on fractions."""
    from fractions import Fraction
    amax = np.abs(v).max(1)
    rows = [[round(Fraction(float(t)) * 127 / Fraction(float(a))) if a else 0 for t in r] for r, a in zip(v, amax)]
    return np.array(rows, np.int64).reshape(v.shape), amax


def rms_norm(x, w, residual=None, eps=1e-6, kind=None):
    """(h, r [rows], v = h w) of float64 rows; kind: the residual's type."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = round_to(round_to(h + np.asarray(residual, np.float64), "float32"), kind)
    mean = (h * h).mean(1) + eps
    r = np.where(mean > 0, 1.0 / np.sqrt(np.where(mean > 0, mean, 1.0)), 0.0)
    return h, np.where(np.isfinite(h).all(1), r, np.nan), h * np.asarray(w, np.float64)

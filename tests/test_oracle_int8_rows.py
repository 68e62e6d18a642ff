"""Pins of the 8-bit oracle: ties, zero and non-finite rows, the half-step bound, a naive product loop."""
import numpy as np

from oracle import int8 as o


def test_ties_by_hand():
    # amax 254: 127 x / 254 = x / 2, so odd x are exact halves
    q, s = o.quantize_row([254.0, 1.0, 3.0, 5.0, -1.0, -3.0, 2.0])
    assert q == [127, 0, 2, 2, 0, -2, 1] and s == 2.0
    assert o.quantize_row([0.0, -0.0]) == ([0, 0], 0.0)
    q, s = o.quantize_row([1.0, float("inf")])
    assert q == [0, 0] and np.isnan(s)


def test_half_step_bound():
    x = np.random.default_rng(5).normal(size=(4, 97)).astype(np.float32).astype(np.float64)
    q, s = o.quantize(x)
    assert np.all(np.abs(x - q * s[:, None]) <= s[:, None] * (0.5 + 1e-12))
    assert np.all(np.abs(q).max(axis=1) == 127)


def test_product_loop():
    rng = np.random.default_rng(6)
    xq, wq = rng.integers(-128, 128, (3, 32)), rng.integers(-128, 128, (5, 32))
    xs, ws = rng.random(3), rng.random(5)
    y = o.gemm(xq, xs, wq, ws)
    for r in range(3):
        for c in range(5):
            assert y[r, c] == sum(int(a) * int(b) for a, b in zip(xq[r], wq[c])) * xs[r] * ws[c]
    w3 = np.stack([wq, -wq])
    out = o.gemm_grouped(xq, xs, w3, np.stack([ws, ws]), [0, 1, 3], [2, 0, 1], 1, np.full((3, 5), 9.0))
    assert np.array_equal(out[2], y[2]) and np.array_equal(out[0], -y[0]) and np.array_equal(out[1], -y[1])
    out = o.gemm_grouped(xq[:1], xs[:1], w3, np.stack([ws, ws]), [0, 1, 1], [1, 0], 2, np.full((2, 5), 9.0))
    assert np.array_equal(out[1], y[0]) and np.all(out[0] == 9.0)

"""Pins of the e4m3 and norm oracles: the type's definition, fractions, hand-worked ties, naive loops."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import fp8, norm


def test_magnitudes_are_the_type():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.values(codes), want, equal_nan=True)
    assert fp8.magnitudes()[-1] == 448 and np.all(np.diff(fp8.magnitudes()) > 0)


def _nearest(v, amax):
    """By fractions: the nearest magnitude, ties to the even code."""
    t = abs(Fraction(float(v))) * 448 / Fraction(float(amax))
    best = min(range(127), key=lambda c: (abs(Fraction(float(fp8.magnitudes()[c])) - t), c % 2))
    return best


@pytest.mark.parametrize("bits", [8, 11, 24, 48])
def test_codes_against_fractions(bits):
    rng = np.random.default_rng(bits)
    v = rng.integers(1, 1 << bits, 300).astype(np.float64) * 2.0 ** rng.integers(-12, 1, 300)
    v[0] = v.max() * 2
    v[1:120] = np.ldexp(np.round(v[1:120] * 64 / v[0]) / 64, int(np.log2(v[0])))   # some on the borders
    amax = np.abs(v).max()
    assert [int(c) for c in fp8.codes_near(v, amax)] == [_nearest(a, amax) for a in v]
    assert np.array_equal(fp8.codes_near(-v, amax), fp8.codes_near(v, amax) | 0x80)


def test_ties_by_hand():
    # amax 448: the quotient is the value itself. 1.0625 lies between 1 (code 56) and 1.125 (57): to 56; 1.1875 between 57 and 58: to 58
    v = np.array([448.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 432.0, 464.0 - 32])
    assert fp8.codes_near(v, 448.0).tolist() == [126, 56, 58, 0, 2, 126, 126]


def test_quantize_blocks_of_rows_and_layers():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(130, 300))
    q, s = fp8.quantize(x)
    assert q.shape == x.shape and s.shape == (130, 3)
    for r, b in ((0, 0), (7, 1), (129, 2)):
        part = x[r, 128 * b:128 * b + 128]
        amax = np.abs(part).max()
        assert s[r, b] == amax / 448 and q[r, 128 * b:128 * b + 128].tolist() == fp8.codes_near(part, amax).tolist()
    ql, sl = fp8.quantize(x, 128)
    assert sl.shape == (2, 3) and sl[1, 2] == np.abs(x[128:, 256:]).max() / 448
    assert ql[129, 299] == fp8.codes_near(x[129:, 299:], np.abs(x[128:, 256:]).max())[0, 0]
    x[5, 200], x[6, 0], x[7] = np.inf, np.nan, 0.0
    q, s = fp8.quantize(x)
    assert np.isnan(s[5, 1]) and np.isnan(s[6, 0]) and not s[7].any() and np.isfinite(s[5, [0, 2]]).all()
    assert not q[5, 128:256].any() and not q[6, :128].any() and not q[7].any()


def test_products_against_a_loop():
    rng = np.random.default_rng(1)
    M, m, n = 3, 131, 150
    xq, wq = rng.normal(size=(M, n)), rng.normal(size=(m, n))
    xs, ws = rng.random((M, 2)), rng.random((2, 2))
    y = fp8.gemm(xq, xs, wq, ws)
    for r, o in ((0, 0), (1, 127), (2, 128), (2, 130)):
        want = sum(xq[r, i] * wq[o, i] * xs[r, i // 128] * ws[o // 128, i // 128] for i in range(n))
        assert abs(y[r, o] - want) < 1e-12
    wq, ws = rng.normal(size=(2, m, n)), rng.random((2, 2, 2))
    z = fp8.gemm_grouped(xq, xs, wq, ws, [0, 1, 3], [5, 0, 3, 1, 2, 4], 2, np.full((6, m), 9.0))
    assert np.allclose(z[5], fp8.gemm(xq[2:], xs[2:], wq[0], ws[0])[0]) and np.allclose(z[0], fp8.gemm(xq[:1], xs[:1], wq[1], ws[1])[0])
    assert (z[[1, 2, 4]] == 9).all()


def test_rounding_to_types():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(2)
    v = (rng.normal(size=4000) * 2.0 ** rng.integers(-150, 120, 4000)).astype(np.float32)
    v[:6] = [0.0, -0.0, np.inf, -np.inf, 3.4e38, 1e-45]
    for kind in ("float16", "bfloat16"):
        want = torch.from_numpy(v).to(getattr(torch, kind)).double().numpy()
        assert np.array_equal(norm.round_to(v.astype(np.float64), kind), want)


def test_norm_by_hand():
    h, r, v = norm.rms_norm(np.array([[3.0, 4.0], [0.0, 0.0]]), np.array([2.0, -1.0]), eps=0.0)
    assert r[0] == pytest.approx(1 / np.sqrt(12.5)) and r[1] == 0 and v[0].tolist() == [6.0, -4.0]
    h, r, v = norm.rms_norm(np.array([[1.0, 2.0]]), np.ones(2), np.array([[2.0 ** -9, 0.0]]), kind="bfloat16")
    assert h.tolist() == [[1.0, 2.0]]                        # 1 + 2^-9 is no bfloat16
    q, amax = norm.steps127(np.array([[127.0, 0.5, -1.5, 2.5]]))
    assert q.tolist() == [[127, 0, -2, 2]] and amax[0] == 127

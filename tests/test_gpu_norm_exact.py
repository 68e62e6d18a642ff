"""rms_norm where its decisions are closest: int8 ties of products with 48 significant bits, values that only a
large weight brings back into the range, the borders of the steps and the values beside them."""
import numpy as np
import pytest

from gpu_common import device, say
from oracle import fp8
from test_gpu_norm import _check
from trellis_coded_gemv_amd import binding as tg

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-6))


def _int8(torch, x, w):
    x, w = torch.from_numpy(x.astype(np.float32)).to("cuda"), torch.from_numpy(w.astype(np.float32)).to("cuda")
    q, s = tg.rms_norm(x, w, out_dtype=torch.int8)
    torch.cuda.synchronize()
    for r in range(len(x)):
        _check(torch, x[r:r + 1], w, None, EPS, "int8", q[r:r + 1], s[r:r + 1], None)


def test_int8_ties_of_long_products():
    """A row of odd multiples of c whose largest is 254 c: 127 h / hmax is an odd number of halves. With c of 16 bits and weights of
    24, the 254 |h w| that the decision compares have 55 bits, more than binary64 holds. Half of the rows lie elsewhere in binary32."""
    device()
    import torch
    say("norm int8 ties")
    rng = np.random.default_rng(1)
    odd = np.arange(1, 254, 2)
    odd = np.r_[odd, -odd]
    for weight in rng.integers(1 << 23, 1 << 24, 6) | 1:
        c = rng.integers(1 << 15, 1 << 16, 10) | 1
        x = np.c_[254 * c, odd[None] * c[:, None]].astype(np.float64)
        assert np.array_equal(x.astype(np.float32).astype(np.float64), x)
        x[5:] *= 2.0 ** -70
        _int8(torch, x, np.full(x.shape[1], weight * 2.0 ** -23))


def test_int8_products_one_unit_from_a_tie():
    """a = odd c. Weights a and a + 1 beside a tie of a * a: (a - 1) (a + 1) is one unit below it; weights a + 2 and a + 1 beside
    a (a + 2): (a + 1) (a + 1) is one above. One unit is 2^-48 of the product at the least."""
    device()
    import torch
    say("norm int8 beside ties")
    rng = np.random.default_rng(2)
    for odd in (1, 3, 85, 101, 125, 127, 129, 251, 253):
        for c in rng.integers(1 << 15, 1 << 16, 4) | 1:
            a = odd * int(c)
            _int8(torch, np.array([[254.0 * c, a - 1, -(a - 1), a, -a]]), np.array([a, a + 1, a + 1, a, a]) * 2.0 ** -20)
            _int8(torch, np.array([[254.0 * c, a + 1, -(a + 1), a, -a]]), np.array([a + 2, a + 1, a + 1, a + 2, a + 2]) * 2.0 ** -20)


@pytest.mark.parametrize("out", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [2, 13, 304, 4100])
def test_weights_that_bring_small_values_back(n, out):
    """Values that the norm alone takes below binary32's normal range, with weights up to 2^127: every output keeps its bits, on rows of
    every scale."""
    dev = device()
    import torch
    say("norm small values, large weights", n, out)
    rng = np.random.default_rng(n)
    rows = []
    for row in (0, 60, 100, -60, -110):                             # the row's largest values
        h = np.ldexp(1 + rng.random(n), row - rng.integers(90, 149, n))
        h[0] = np.ldexp(1.0, row)
        rows.append(h * rng.choice([-1, 1], n))
    x = torch.from_numpy(np.array(rows).astype(np.float32))
    w = np.ldexp(1 + rng.random(n), rng.integers(60, 127, n))
    w[0], w[1] = 1.0, 1.3 * 2.0 ** 127
    x[0, 1] = 2.0 ** -130
    w = torch.from_numpy(w.astype(np.float32))
    y = tg.rms_norm(x.to(dev), w.to(dev), eps=0.0, out_dtype=getattr(torch, out))
    torch.cuda.synchronize()
    for r in range(len(x)):
        _check(torch, x[r:r + 1].to(dev), w.to(dev), None, 0.0, out, y[r:r + 1], None, None)


@pytest.mark.parametrize("out", ["float32", "float16"])
def test_zeros_beside_values_whose_norm_leaves_binary32(out):
    """Pieces of zeros in a row of subnormal values, whose 1 / sqrt(mean) is beyond binary32: zeros stay zeros."""
    dev = device()
    import torch
    say("norm zeros beside subnormal values", out)
    x = torch.zeros(2, 400)
    x[0, 5], x[1, 300:] = 2.0 ** -149, -(2.0 ** -140)
    w = torch.linspace(0.5, 1.5, 400)
    y = tg.rms_norm(x.to(dev), w.to(dev), eps=0.0, out_dtype=getattr(torch, out))
    torch.cuda.synchronize()
    for r in range(2):
        _check(torch, x[r:r + 1].to(dev), w.to(dev), None, 0.0, out, y[r:r + 1], None, None)


def _neighbours(torch, v):
    """v, and the values of its type one last place above and below in magnitude."""
    bits = v.view(torch.int32 if v.dtype == torch.float32 else torch.int16)
    return [v, (bits + 1).view(v.dtype), (bits - 1).view(v.dtype)]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("out", ["int8", "float8_e4m3fn"])
def test_every_border_and_its_neighbours(out, dtype):
    """Every border of two steps and the values of the type one last place beside it, at scales that are powers of two or not; every row compared."""
    dev = device()
    import torch
    say("norm borders and neighbours", out, dtype)
    t = getattr(torch, dtype)
    m = fp8.magnitudes()
    top, mid = (127.0, np.arange(0.5, 127)) if out == "int8" else (448.0, (m[1:] + m[:-1]) / 2)
    rows = []
    for scale in (1.0, 2.0 ** -5, 3.0, 2.0 ** 5 / 3):
        border = torch.from_numpy(mid * scale).to(t)
        for v in _neighbours(torch, border):
            rows += [torch.cat([torch.full((1,), top * scale, dtype=t), v]), torch.cat([torch.full((1,), -top * scale, dtype=t), -v])]
    x = torch.stack(rows)
    parts = [torch.cat([x[:, :1], p, x[:, :1].expand(-1, 127 - p.shape[1])], 1) for p in x[:, 1:].split(127, 1)]   # each 128 values with the largest among them
    x = torch.cat(parts, 1).contiguous().to(dev)
    for w in (1.0, 1.0 + 2.0 ** -7, 1.0 + 3 * 2.0 ** -5):
        w = torch.full((x.shape[1],), w, dtype=t, device=dev)
        got = tg.rms_norm(x, w, out_dtype=getattr(torch, out))
        torch.cuda.synchronize()
        for r in range(x.shape[0]):
            _check(torch, x[r:r + 1], w, None, EPS, out, got[0][r:r + 1], got[1][r:r + 1], None)

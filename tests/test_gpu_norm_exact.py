"""rms_norm where its decisions are closest: int8 ties of products with 48 significant bits."""
import numpy as np
import pytest

from gpu_common import device, say
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

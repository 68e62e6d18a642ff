"""The routing and 8-bit entry points at the ends of their documented ranges."""
import pytest

from gpu_common import device, say
from trellis_coded_gemv_amd import binding as tg

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24
TOL = (1 + STEP) ** 3 - 1            # three roundings to binary32


def _ints(torch, dev, shape, seed):
    return torch.randint(-128, 128, shape, generator=torch.Generator(device=dev).manual_seed(seed), device=dev, dtype=torch.int8)


def _near(y, ref):
    assert bool(((y.double() - ref).abs() <= TOL * ref.abs()).all())


def test_most_tokens():
    """2^24 tokens of two experts: the larger logit's, the first of equal ones; its score is s or 1 - s of the difference."""
    dev = device()
    import torch
    say("largest route")
    l = torch.randint(-3, 4, (1 << 24, 2), generator=torch.Generator(device=dev).manual_seed(1), device=dev).float()
    sel, w = tg.moe_route(l, 1, renormalize=False)
    assert torch.equal(sel[:, 0], (l[:, 1] > l[:, 0]).int())
    ref = torch.sigmoid((l[:, 0] - l[:, 1]).abs().double())
    assert bool(((w[:, 0].double() - ref).abs() <= STEP * (1 + 1e-6) * ref).all())


@pytest.mark.parametrize("pairs,experts", [(1 << 24, 1024), ((1 << 24) - 4097, 256), (1 << 24, 1)])
def test_most_pairs(pairs, experts):
    dev = device()
    import torch
    say("largest group", pairs, experts)
    sel = torch.randint(-1, experts, (pairs,), generator=torch.Generator(device=dev).manual_seed(2), device=dev, dtype=torch.int32)
    off, order = tg.moe_group(sel, experts)
    last = torch.where(sel < 0, torch.full_like(sel, experts), sel)
    assert torch.equal(order.long(), torch.sort(last, stable=True).indices)
    assert torch.equal(off[1:].long(), torch.bincount(last.long(), minlength=experts + 1)[:experts].cumsum(0)) and int(off[0]) == 0


@pytest.mark.parametrize("rows,n", [(1 << 24, 4), (3, 1 << 22), ((1 << 24) - 1, 1)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_most_rows_and_values(rows, n, dtype):
    """Steps by binary64 quotients, off by less than 2^-44: they decide every step but exact halves, where either neighbour passes."""
    dev = device()
    import torch
    say("largest quantize", rows, n, dtype)
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.randn((rows, n), generator=g, device=dev).to(getattr(torch, dtype))
    q, s = tg.int8_quantize(x)
    for a in range(0, rows, 1 << 22):
        xd = x[a:a + (1 << 22)].double()
        amax = xd.abs().amax(1, keepdim=True)
        one = torch.where(amax > 0, amax, torch.ones_like(amax))     # a row of zeros has steps 0
        t = xd * 127.0 / one
        exact = 254.0 * xd.abs() / one
        sure = (exact - exact.round()).abs() > 2.0 ** -40            # twice the quotient is no whole number: no half
        sure |= exact.round().remainder(2.0) == 0                    # or an even one: a whole step
        part = q[a:a + (1 << 22)].double()
        assert bool((part == t.round())[sure].all()) and bool(((part - t).abs() <= 0.5 + 1e-9).all())
        ref = amax[:, 0] / 127.0
        assert bool(((s[a:a + (1 << 22)].double() - ref).abs() <= STEP * ref).all())


@pytest.mark.parametrize("M,m,n", [(1 << 20, 17, 16), (1, 1 << 22, 16), (3, (1 << 22) - 1, 32), ((1 << 20) - 7, 250, 16), (1 << 16, 4100, 16)])
def test_most_rows_and_outputs(M, m, n):
    dev = device()
    import torch
    say("largest int8 gemm", M, m, n)
    g = torch.Generator(device=dev).manual_seed(4)
    xq, wq = _ints(torch, dev, (M, n), 5), _ints(torch, dev, (m, n), 6)
    xs, ws = torch.rand(M, generator=g, device=dev) + 0.5, torch.rand(m, generator=g, device=dev) + 0.5
    y = tg.int8_gemm(tg.Int8Layer(wq, ws), xq, xs)
    step = max(1, (1 << 28) // m)
    for a in range(0, M, step):
        _near(y[a:a + step], (xq[a:a + step].double() @ wq.double().t()) * xs[a:a + step].double()[:, None] * ws.double())


def test_largest_row_stride():
    """Layer rows 2^23 bytes apart: the last of a tile's 256 lies 2^31 bytes behind its first. One byte more is refused."""
    dev = device()
    import torch
    say("largest int8 row stride")
    m, n, M = 300, 272, 300
    wide = torch.empty(m, 1 << 23, dtype=torch.int8, device=dev)
    wide[:, :n] = _ints(torch, dev, (m, n), 7)
    g = torch.Generator(device=dev).manual_seed(8)
    ws = torch.rand(m, generator=g, device=dev) + 0.5
    for rows in (1, 40, M, 3000):
        xq, xs = _ints(torch, dev, (rows, n), 9), torch.rand(rows, generator=g, device=dev) + 0.5
        y = tg.int8_gemm(tg.Int8Layer(wide[:, :n], ws), xq, xs)
        _near(y, (xq.double() @ wide[:, :n].double().t()) * xs.double()[:, None] * ws.double())
    far = torch.empty(2 * ((1 << 23) + 16), dtype=torch.int8, device=dev).view(2, -1)[:, :n]
    with pytest.raises(tg.TgError):
        tg.int8_gemm(tg.Int8Layer(far, ws[:2]), xq, xs)


@pytest.mark.parametrize("m,n", [(16, 16), (33, 48)])
def test_most_pairs_of_most_experts(m, n):
    dev = device()
    import torch
    say("largest int8 grouped", m, n)
    pairs, experts = 1 << 20, 1024
    g = torch.Generator(device=dev).manual_seed(10)
    sel = torch.randint(0, experts, (pairs,), generator=g, device=dev, dtype=torch.int32)
    sel[::1000] = -1
    xq, wq = _ints(torch, dev, (pairs // 8, n), 11), _ints(torch, dev, (experts, m, n), 12)
    xs, ws = torch.rand(pairs // 8, generator=g, device=dev) + 0.5, torch.rand(experts, m, generator=g, device=dev) + 0.5
    y = tg.int8_gemm_grouped(tg.Int8Experts(wq, ws), xq, xs, *tg.moe_group(sel, experts), 8)
    assert not bool(y[::1000].any())
    for a in range(0, pairs, 1 << 17):
        e, t = sel[a:a + (1 << 17)].long(), torch.arange(a, a + (1 << 17), device=dev) // 8
        there = e >= 0
        ref = (wq[e].double() * xq[t].double()[:, None, :]).sum(2) * xs[t].double()[:, None] * ws[e].double()
        _near(y[a:a + (1 << 17)][there], ref[there])

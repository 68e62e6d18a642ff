"""Every kernel of the 8-bit products against exact sums: each tile shape, whole and in each number of parts of its inner axis, dense and
over ragged experts, every output type."""
import pytest

from gpu_common import device, say
from int8_shapes import DENSE, GROUPED, plan
from trellis_coded_gemv_amd import binding as tg

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24                   # an output: three roundings to binary32, and one more to a 16-bit type
TOL = {"float32": (1 + STEP) ** 3 - 1, "float16": (1 + STEP) ** 3 * (1 + 2.0 ** -11) - 1, "bfloat16": (1 + STEP) ** 3 * (1 + 2.0 ** -8) - 1}


def _operands(torch, dev, rows, weights, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    q = lambda s: torch.randint(-128, 128, s, generator=g, device=dev, dtype=torch.int8)
    r = lambda s: torch.rand(s, generator=g, device=dev) * 0.01 + 0.001
    n = weights[-1]
    return q((rows, n + 16))[:, :n], r(rows), q(weights), r(weights[:-1])


def _near(torch, y, xq, xs, wq, ws, dtype):
    """Sums of 8-bit products are below 2^53: binary64 holds them exactly."""
    ref = (xq.double() @ wq.double().t()) * xs.double()[:, None] * ws.double()
    bound = TOL[dtype] * ref.abs() + (2.0 ** -25 if dtype == "float16" else 0.0)
    bad = ~((y.double() - ref).abs() <= bound)
    assert not bool(bad.any()), bad.nonzero()[0].tolist()


@pytest.mark.parametrize("M,m,n", DENSE)
def test_dense(M, m, n):
    dev = device()
    import torch
    say("int8 shapes dense", M, m, n, plan(M, m, n))
    xq, xs, wq, ws = _operands(torch, dev, M, (m, n), M + m + n)
    L = tg.Int8Layer(wq, ws)
    work = tg.int8_workspace(L, M)
    for dtype in ("float32", "bfloat16", "float16"):
        Y = torch.full((M + 1, m + 3), 9.0, dtype=getattr(torch, dtype), device=dev)
        tg.int8_gemm(L, xq, xs, Y=Y[:M, :m], ws=work)
        torch.cuda.synchronize()
        _near(torch, Y[:M, :m], xq, xs, wq, ws, dtype)
        assert bool((Y[M] == 9).all()) and bool((Y[:, m:] == 9).all())
    assert not bool(work[256:256 + 4096].any())                      # counters back at zero


@pytest.mark.parametrize("pairs,m,n,experts,top_k", GROUPED)
@pytest.mark.parametrize("shared", [True, False])
def test_grouped(pairs, m, n, experts, top_k, shared):
    """One crowded expert, one without pairs, some pairs that no expert has."""
    dev = device()
    import torch
    say("int8 shapes grouped", pairs, m, n, experts, top_k, shared, plan(pairs, m, n, experts))
    ppr = top_k if shared else 1
    xq, xs, wq, ws = _operands(torch, dev, pairs // ppr, (experts, m, n), pairs + m + n)
    g = torch.Generator(device=dev).manual_seed(pairs)
    sel = torch.randint(0, experts, (pairs,), generator=g, device=dev, dtype=torch.int32)
    if experts > 2:
        sel[torch.rand(pairs, generator=g, device=dev) < 0.2] = 1
        sel[sel == 2] = 0
    sel[torch.rand(pairs, generator=g, device=dev) < 0.03] = -1
    off, order = tg.moe_group(sel, experts)
    E = tg.Int8Experts(wq, ws)
    rows = torch.arange(pairs, device=dev) // ppr
    for dtype in ("float32", "bfloat16", "float16"):
        Y = torch.full((pairs + 1, m + 5), 9.0, dtype=getattr(torch, dtype), device=dev)
        tg.int8_gemm_grouped(E, xq, xs, off, order, ppr, Y=Y[:pairs, :m])
        torch.cuda.synchronize()
        assert bool((Y[pairs] == 9).all()) and bool((Y[:, m:] == 9).all()) and bool((Y[:pairs, :m][sel < 0] == 9).all())
        for e in range(experts):
            p = (sel == e).nonzero()[:, 0]
            if len(p):
                _near(torch, Y[p, :m], xq[rows[p]], xs[rows[p]], wq[e], ws[e], dtype)
        own = tg.int8_gemm_grouped(E, xq, xs, off, order, ppr, out_dtype=getattr(torch, dtype))
        assert torch.equal(own[sel >= 0], Y[:pairs, :m][sel >= 0]) and not bool(own[sel < 0].any())

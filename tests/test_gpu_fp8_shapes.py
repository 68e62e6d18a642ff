"""Every kernel of the e4m3 products against the oracle, on a choice of rows and outputs, and twice with the same bits."""
import numpy as np
import pytest

from fp8_shapes import DENSE16, DENSE32, GROUPED16, GROUPED32, plan
from gpu_common import device, say
from oracle import fp8 as oracle
from test_gpu_fp8 import _bound, _f8, _operands
from trellis_coded_gemv_amd import binding as tg

pytestmark = pytest.mark.gpu


def _pick(rng, count, most):
    """The ends, the borders of tiles and some between."""
    return np.unique(np.r_[0, count - 1, np.arange(127, count, 128)[:most // 2], rng.integers(0, count, most // 2)].clip(0, count - 1))


def _check(torch, y, rows, xq, xs, wq, ws, outs, dtype):
    """y's rows and outs against the oracle; xq, xs: those rows'."""
    nb = xs.shape[1]
    sums = oracle.block_sums(oracle.values(xq), oracle.values(wq[outs]))
    scales = xs.astype(np.float64)[:, None, :] * ws.astype(np.float64)[outs // 128][None]
    ref = (sums * scales).sum(2)
    got = y[torch.from_numpy(rows).to(y.device)][:, torch.from_numpy(outs).to(y.device)].double().cpu().numpy()
    assert np.isfinite(got).all() and nb == sums.shape[2]
    over = np.abs(got - ref) - _bound(sums, scales, ref, dtype)
    assert over.max() <= 0, float(over.max())


@pytest.mark.parametrize("M,m,n,dtype", [c + (("float16", "bfloat16")[i % 2],) for i, c in enumerate(DENSE16)] + [c + ("float32",) for c in DENSE32])
def test_dense(M, m, n, dtype):
    dev = device()
    import torch
    say("fp8 shapes", M, m, n, dtype, plan(M, m, n, 0, 0 if dtype == "float32" else 2))
    rng = np.random.default_rng(M + m + n)
    xq, xs, wq, ws = _operands(rng, M, m, n)
    L = tg.Fp8Layer(_f8(torch, wq, dev), torch.from_numpy(ws).to(dev))
    X, S = _f8(torch, xq, dev), torch.from_numpy(xs).to(dev)
    work = tg.fp8_workspace(L, M)
    y = tg.fp8_gemm(L, X, S, out_dtype=getattr(torch, dtype), ws=work)
    z = tg.fp8_gemm(L, X, S, out_dtype=getattr(torch, dtype), ws=work)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and bool(y.isfinite().all())
    assert not work[256:256 + 4096].any()                            # the counters are zero between calls
    rows, outs = _pick(rng, M, 24), _pick(rng, m, 40)
    _check(torch, y, rows, xq[rows], xs[rows], wq, ws, outs, dtype)


@pytest.mark.parametrize("pairs,m,n,experts,top_k,dtype", [c + (("bfloat16", "float16")[i % 2],) for i, c in enumerate(GROUPED16)] + [c + ("float32",) for c in GROUPED32])
def test_grouped(pairs, m, n, experts, top_k, dtype):
    dev = device()
    import torch
    say("fp8 grouped shapes", pairs, m, n, experts, top_k, dtype, plan(pairs, m, n, experts, 0 if dtype == "float32" else 2))
    rng = np.random.default_rng(pairs + m + n)
    sel = np.argsort(rng.random((pairs // top_k, experts)) + 0.3 * rng.random(experts), 1)[:, :top_k].astype(np.int32)
    sel[rng.random(sel.shape) < 0.05] = -1
    for per_pair in (False, True):
        ppr = 1 if per_pair else top_k
        xq, xs, wq, ws = _operands(rng, pairs // ppr, m, n, (experts,))
        offsets, order = tg.moe_group(torch.from_numpy(sel).to(dev), experts)
        E = tg.Fp8Experts(_f8(torch, wq, dev), torch.from_numpy(ws).to(dev))
        X, S = _f8(torch, xq, dev), torch.from_numpy(xs).to(dev)
        y = tg.fp8_gemm_grouped(E, X, S, offsets, order, ppr, out_dtype=getattr(torch, dtype))
        z = tg.fp8_gemm_grouped(E, X, S, offsets, order, ppr, out_dtype=getattr(torch, dtype))
        torch.cuda.synchronize()
        assert torch.equal(y, z) and bool(y.isfinite().all())
        of, od = offsets.cpu().numpy(), order.cpu().numpy()
        assert not y[torch.from_numpy(od[of[-1]:]).long().to(dev)].any()
        outs = _pick(rng, m, 40)
        for e in np.unique(np.r_[0, experts - 1, rng.integers(0, experts, 6)]):
            p = od[of[e]:of[e + 1]]
            if len(p):
                p = p[_pick(rng, len(p), 12)]
                _check(torch, y, p.astype(np.int64), xq[p // ppr], xs[p // ppr], wq[e], ws[e], outs, dtype)

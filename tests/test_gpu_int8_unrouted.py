"""int8_gemm_grouped over pairs without an expert: rows of an output that the call makes are zero there, a caller's own are
left as they were; a whole block over masked experts stays finite."""
import numpy as np
import pytest

from gpu_common import device, say
from oracle import int8 as oracle
from trellis_coded_gemv_amd import binding as tg

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24                   # an output: three roundings to binary32, and one more to a 16-bit type
TOL = {"float32": (1 + STEP) ** 3 - 1, "float16": (1 + STEP) ** 3 * (1 + 2.0 ** -11) - 1, "bfloat16": (1 + STEP) ** 3 * (1 + 2.0 ** -8) - 1}


def _leave_nan(torch, dev, shape, dtype):
    """Freed memory of the size that the next output takes, full of NaN."""
    held = [torch.full(shape, float("nan"), dtype=dtype, device=dev) for _ in range(3)]
    torch.cuda.synchronize()
    del held


CASES = [  # tokens, experts, top_k, m, n, share of pairs without an expert
    (1, 8, 1, 16, 16, 1.0), (1, 128, 8, 96, 256, 0.5), (3, 4, 2, 130, 272, 0.3), (64, 128, 8, 128, 512, 0.2), (300, 8, 3, 256, 640, 0.1),
    (300, 2, 1, 515, 128, 1.0), (700, 16, 6, 300, 272, 0.9), (513, 3, 2, 1031, 1024, 0.02), (40, 1024, 8, 33, 64, 0.3), (600, 1, 1, 260, 400, 0.5),
    (700, 64, 4, 64, 128, 0.5), (200, 300, 3, 40, 80, 0.0)]


@pytest.mark.parametrize("tokens,experts,top_k,m,n,share", CASES)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_rows_without_an_expert(tokens, experts, top_k, m, n, share, dtype):
    dev = device()
    import torch
    say("int8 unrouted", tokens, experts, top_k, m, n, share, dtype)
    rng = np.random.default_rng(tokens + experts + m)
    t = getattr(torch, dtype)
    sel = rng.integers(0, experts, tokens * top_k)
    sel[rng.random(sel.size) < share] = -1
    sel[rng.random(sel.size) < share / 4] = experts
    xq = rng.integers(-128, 128, (tokens, n)).astype(np.int8)
    wq = rng.integers(-128, 128, (experts, m, n)).astype(np.int8)
    xs, ws = ((rng.random(s) * 0.02 + 0.001).astype(np.float32) for s in (tokens, (experts, m)))
    E = tg.Int8Experts(torch.from_numpy(wq).to(dev), torch.from_numpy(ws).to(dev))
    off, order = tg.moe_group(torch.from_numpy(sel.astype(np.int32)).to(dev), experts)
    X = torch.from_numpy(xq).to(dev), torch.from_numpy(xs).to(dev)
    own = torch.full((sel.size, m), 9.0, dtype=t, device=dev)
    tg.int8_gemm_grouped(E, *X, off, order, top_k, Y=own)
    _leave_nan(torch, dev, (sel.size, m), t)
    y = tg.int8_gemm_grouped(E, *X, off, order, top_k, out_dtype=t).double().cpu().numpy()
    own = own.double().cpu().numpy()
    for p, e in enumerate(sel):
        if 0 <= e < experts:
            ref = oracle.gemm(xq[p // top_k:p // top_k + 1], xs[p // top_k:p // top_k + 1], wq[e], ws[e])[0]
            assert np.all(np.abs(y[p] - ref) <= TOL[dtype] * np.abs(ref) + (2.0 ** -25 if dtype == "float16" else 0.0)), p
            assert np.array_equal(own[p], y[p]), p
        else:
            assert not y[p].any() and (own[p] == 9).all(), p


def _block(torch, x, logits, gu, dn, top_k):
    """Route, group, quantise, gate/up, silu * up, quantise, down, combine, every output the calls' own."""
    tokens, hidden = x.shape
    sel, w = tg.moe_route(logits, top_k, renormalize=False)
    off, order = tg.moe_group(sel, gu.experts)
    h = tg.int8_gemm_grouped(gu, *tg.int8_quantize(x), off, order, pairs_per_row=top_k)
    a = (torch.nn.functional.silu(h[:, :dn.n]) * h[:, dn.n:]).half()
    y = tg.int8_gemm_grouped(dn, *tg.int8_quantize(a), off, order)
    return (y.view(tokens, top_k, hidden) * w[..., None]).sum(1)


def test_block_over_masked_experts():
    """Tokens with fewer available experts than slots (one with none), over memory that held NaN: the same outputs as over clean memory,
    zeros for the token without experts."""
    dev = device()
    import torch
    say("int8 block over masked experts")
    g = torch.Generator().manual_seed(61)
    tokens, experts, top_k, hidden, inter = 70, 16, 4, 256, 96
    gu = tg.Int8Experts.from_dense((torch.randn(experts, 2 * inter, hidden, generator=g) * 0.06).to(dev))
    dn = tg.Int8Experts.from_dense((torch.randn(experts, hidden, inter, generator=g) * 0.1).to(dev))
    x = torch.randn(tokens, hidden, generator=g).half().to(dev)
    logits = torch.randn(tokens, experts, generator=g).to(dev)
    logits[5] = float("-inf")
    logits[11:20, 3:] = float("-inf")
    logits[69, 1:] = float("-inf")
    first = _block(torch, x, logits, gu, dn, top_k)
    for _ in range(3):
        for shape in ((tokens * top_k, 2 * inter), (tokens * top_k, hidden)):
            _leave_nan(torch, dev, shape, torch.float32)
        y = _block(torch, x, logits, gu, dn, top_k)
        assert bool(y.isfinite().all()) and torch.equal(y, first) and not bool(y[5].any())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _block(torch, x, logits, gu, dn, top_k)
    for _ in range(4):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        assert torch.equal(_block(torch, x, logits, gu, dn, top_k), first)
        torch.cuda.synchronize()


def test_offsets_that_fall():
    """Lists that overlap, as no grouping makes them: whatever products are missing, nothing outside the output is written."""
    dev = device()
    import torch
    say("int8 grouped falling offsets")
    g = torch.Generator().manual_seed(62)
    pairs, experts, m, n = 300, 40, 70, 64
    E = tg.Int8Experts.from_dense(torch.randn(experts, m, n, generator=g).to(dev))
    q, s = tg.int8_quantize(torch.randn(pairs, n, generator=g).to(dev))
    order = torch.randperm(pairs, generator=g).to(torch.int32).to(dev)
    for offsets in ([0, pairs] * 20 + [0], [pairs, 0] * 20 + [pairs], list(range(40, -1, -1)), [pairs] * 41, [-1] * 41):
        off = torch.tensor(offsets, dtype=torch.int32, device=dev)
        Y = torch.full((pairs + 2, m + 4), 9.0, device=dev)
        tg.int8_gemm_grouped(E, q, s, off, order, Y=Y[1:-1, 2:-2])
        y = tg.int8_gemm_grouped(E, q, s, off, order)
        torch.cuda.synchronize()
        assert bool((Y[0] == 9).all()) and bool((Y[-1] == 9).all()) and bool((Y[:, :2] == 9).all()) and bool((Y[:, -2:] == 9).all())
        if offsets[-1] <= 0 and max(offsets) <= 0:                   # every pair is behind the last expert's
            assert not bool(y.any())

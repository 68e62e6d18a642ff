"""int8_quantize, int8_gemm and int8_gemm_grouped on the GPU against the exact oracle."""
import numpy as np
import pytest

from gpu_common import device, say
from oracle import int8 as oracle
from oracle import route as route_oracle
from trellis_coded_gemv_amd import binding as tg

pytestmark = pytest.mark.gpu

# An output is the exact sum rounded to binary32 and two products rounded in binary32, each by at most 2^-24 relative;
# a 16-bit output is rounded once more, by half a step of its type (and, below fp16's normal range, by 2^-25 at most).
STEP = 2.0 ** -24
TOL = {"float32": (1 + STEP) ** 3 - 1, "float16": (1 + STEP) ** 3 * (1 + 2.0 ** -11) - 1, "bfloat16": (1 + STEP) ** 3 * (1 + 2.0 ** -8) - 1}


def _near(y, ref, dtype):
    y = y.double().cpu().numpy()
    assert np.isfinite(y).all()
    bound = TOL[dtype] * np.abs(ref) + (2.0 ** -25 if dtype == "float16" else 2.0 ** -149)
    assert np.all(np.abs(y - ref) <= bound), float((np.abs(y - ref) - bound).max())


@pytest.mark.parametrize("rows,n,pad", [(1, 1, 0), (3, 7, 0), (1, 16, 0), (5, 64, 1), (4, 100, 8), (2, 255, 0), (2, 257, 3), (3, 2048, 0),
                                        (2, 8192, 16), (1, 8192, 0), (300, 130, 0), (2, 14336, 0), (1, 14337, 0), (1, 40000, 0), (2, 70001, 5),
                                        (600, 4104, 0), (66000, 8, 0), (65537, 3, 1)])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_quantize_is_exact(rows, n, pad, dtype):
    dev = device()
    import torch
    say("quantize", rows, n, pad, dtype)
    rng = np.random.default_rng(rows * 7 + n)
    x = torch.from_numpy((rng.normal(size=(rows, n + pad)) * 3).astype(np.float32)).to(getattr(torch, dtype))
    x[0, 0] = 127.0                     # with halves on the grid: exact ties in the first row, whose amax is 127
    x[0, : n // 2] = (x[0, : n // 2].float() * 2).round().clamp(-254, 254).to(x.dtype) / 2
    if pad:
        x[:, n:] = float("nan")         # between the rows: never read
    xv = x.to(dev)[:, :n]
    q = torch.full((rows, n + 5), 99, dtype=torch.int8, device=dev)
    scales = torch.full((rows + 2,), 99.0, device=dev)
    tg.int8_quantize(xv, q=q[:, :n], scales=scales[1:-1])
    torch.cuda.synchronize()
    # the oracle works on fractions: of many rows, it takes the ends and some between
    pick = np.arange(rows) if rows <= 300 else np.unique(np.r_[0, rows - 1, 65534, 65535, 65536, rng.integers(0, rows, 8)].clip(0, rows - 1))
    qr, sr = oracle.quantize(x[pick, :n].double().numpy())
    got = q.cpu().numpy()
    assert np.array_equal(got[pick, :n], qr) and (got[:, n:] == 99).all()
    s = scales.double().cpu().numpy()
    assert s[0] == s[-1] == 99 and np.all(np.abs(s[1:-1][pick] - sr) <= STEP * sr)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("n", [24, 9000])
def test_quantize_special_rows(dtype, n):
    """Zero rows, NaN and infinity, one value, the type's largest and smallest values."""
    dev = device()
    import torch
    say("quantize special", dtype, n)
    t = getattr(torch, dtype)
    fi = torch.finfo(t)
    x = torch.randn(9, n, generator=torch.Generator().manual_seed(1)).to(t)
    x[0] = 0
    x[1, n - 1] = float("nan")
    x[2, 5] = float("-inf")
    x[3] = 0
    x[3, n - 2] = -2.5
    x[4, 3] = fi.max
    x[5] = 0
    x[5, :4] = torch.tensor([fi.smallest_normal, -fi.smallest_normal / 2, fi.smallest_normal / 4, 0]).to(t)
    x[6] = -0.0
    x[7] = fi.max
    x[8] *= fi.tiny
    q, s = tg.int8_quantize(x.to(dev))
    torch.cuda.synchronize()
    qr, sr = oracle.quantize(x.double().numpy())
    assert np.array_equal(q.cpu().numpy(), qr)
    s = s.double().cpu().numpy()
    assert np.array_equal(np.isnan(s), np.isnan(sr)) and np.isnan(sr).sum() == 2
    ok = ~np.isnan(sr)
    assert np.all(np.abs(s[ok] - sr[ok]) <= STEP * sr[ok] + 2.0 ** -150)


def test_quantize_shapes_and_strided_views():
    dev = device()
    import torch
    say("quantize shapes")
    x = torch.randn(4, 6, 32, generator=torch.Generator().manual_seed(2)).half().to(dev)
    q, s = tg.int8_quantize(x)
    assert q.shape == x.shape and s.shape == (4, 6)
    q1, s1 = tg.int8_quantize(x[1, 2])
    assert torch.equal(q1, q[1, 2]) and float(s1) == float(s[1, 2])
    qt, st = tg.int8_quantize(x.transpose(0, 1))
    assert torch.equal(qt, q.transpose(0, 1)) and torch.equal(st, s.t())
    qc, sc = tg.int8_quantize(x[:, :, 0].float().t())               # columns: the innermost stride is not one
    qd, sd = tg.int8_quantize(x[:, :, 0].float().t().contiguous())
    assert torch.equal(qc, qd) and torch.equal(sc, sd)


def _operands(rng, M, m, n, extreme=False):
    lo, hi = (-128, 128)
    xq = rng.integers(lo, hi, (M, n)).astype(np.int8)
    wq = rng.integers(lo, hi, (m, n)).astype(np.int8)
    if extreme:
        xq[:], wq[:] = -128, -128
    xs = (rng.random(M) * 0.02 + 0.001).astype(np.float32)
    ws = (rng.random(m) * 0.02 + 0.001).astype(np.float32)
    return xq, xs, wq, ws


def _padded(torch, a, dev, pad, fill):
    wide = np.full((a.shape[0], a.shape[1] + pad), fill, a.dtype)
    wide[:, :a.shape[1]] = a
    return torch.from_numpy(wide).to(dev)[:, :a.shape[1]]


GEMM = [  # M, m, n, pads of x, w and y
    (1, 1, 16, 0, 0, 0), (1, 128, 256, 0, 0, 0), (1, 100, 48, 16, 32, 0), (1, 1000, 2064, 0, 0, 0), (2, 33, 80, 0, 16, 3),
    (15, 130, 272, 16, 0, 4), (16, 64, 512, 0, 0, 0), (17, 65, 1040, 0, 0, 1), (31, 256, 768, 0, 0, 0), (33, 515, 144, 0, 0, 2),
    (61, 384, 4096, 0, 0, 0), (64, 256, 14336, 0, 0, 0), (65, 257, 320, 16, 16, 7), (100, 300, 1264, 0, 0, 0), (128, 256, 128, 0, 0, 0),
    (129, 512, 640, 0, 0, 8), (200, 1000, 2000, 0, 48, 0), (255, 255, 256, 0, 0, 0), (256, 256, 1024, 0, 0, 0), (257, 513, 1040, 0, 0, 0),
    (300, 770, 384, 0, 0, 2), (512, 1024, 2048, 0, 0, 0), (777, 1281, 400, 32, 0, 5), (1030, 260, 16, 0, 0, 0), (2048, 528, 144, 0, 0, 0)]


@pytest.mark.parametrize("M,m,n,px,pw,py", GEMM)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_gemm_matches_oracle(M, m, n, px, pw, py, dtype):
    dev = device()
    import torch
    say("int8 gemm", M, m, n, px, pw, py, dtype)
    rng = np.random.default_rng(M * 31 + m + n)
    xq, xs, wq, ws = _operands(rng, M, m, n)
    L = tg.Int8Layer(_padded(torch, wq, dev, pw, 55), torch.from_numpy(ws).to(dev))
    X = _padded(torch, xq, dev, px, 77)
    wide = torch.full((M + 2, m + py), 9.0, dtype=getattr(torch, dtype), device=dev)
    work = tg.int8_workspace(L, M)
    for _ in range(2):                                              # the workspace serves call after call
        tg.int8_gemm(L, X, torch.from_numpy(xs).to(dev), Y=wide[1:-1, :m], ws=work)
        torch.cuda.synchronize()
        _near(wide[1:-1, :m], oracle.gemm(xq, xs, wq, ws), dtype)
        assert bool((wide[0] == 9).all()) and bool((wide[-1] == 9).all()) and bool((wide[:, m:] == 9).all())


LARGE = [  # one or more products for each tile shape and for split inner axes; odd sizes, ends inside a step
    (3001, 4001, 4112), (1500, 5003, 2064), (301, 20001, 1040), (1030, 9000, 272), (100, 30001, 1040), (515, 4099, 2064), (260, 4100, 4112),
    (150, 28674, 144), (61, 4096, 14336), (64, 4097, 14352), (1, 28672, 8192), (1, 28673, 176), (256, 4096, 14336), (2050, 300, 20000)]


def _device_ref(torch, xq, xs, wq, ws):
    """The exact sums by binary64 products on the device (below 2^53), and their scaled values in binary64."""
    return (xq.double() @ wq.double().t()) * xs.double()[:, None] * ws.double()


def _near_on_device(torch, y, ref, dtype):
    bound = TOL[dtype] * ref.abs() + (2.0 ** -25 if dtype == "float16" else 2.0 ** -149)
    assert bool((y.double() - ref).abs().le(bound).all())


@pytest.mark.parametrize("M,m,n", LARGE)
def test_gemm_large_tiles(M, m, n):
    dev = device()
    import torch
    say("int8 gemm large", M, m, n)
    g = torch.Generator(device=dev).manual_seed(M + m + n)
    q = lambda *s: torch.randint(-128, 128, s, generator=g, device=dev, dtype=torch.int8)
    xq, wq = q(M, n + 16)[:, :n], q(m, n)
    xs, ws = torch.rand(M, generator=g, device=dev) * 0.01 + 0.001, torch.rand(m, generator=g, device=dev) * 0.01 + 0.001
    L = tg.Int8Layer(wq, ws)
    work = tg.int8_workspace(L, M)
    ref = _device_ref(torch, xq, xs, wq, ws)
    first = None
    for dtype in ("float32", "bfloat16", "float16", "float32"):
        Y = torch.full((M + 1, m + 3), 9.0, dtype=getattr(torch, dtype), device=dev)
        tg.int8_gemm(L, xq, xs, Y=Y[:M, :m], ws=work)
        torch.cuda.synchronize()
        _near_on_device(torch, Y[:M, :m], ref, dtype)
        assert bool((Y[M] == 9).all()) and bool((Y[:, m:] == 9).all())
        if dtype == "float32":
            assert first is None or torch.equal(first, Y)            # the same bits, however the parts arrive
            first = Y
    assert not bool(work[256:256 + 4096].any())                      # counters back at zero


LARGE_GROUPED = [(4000, 4100, 4112, 2, 2), (1000, 2100, 272, 3, 3), (3000, 5000, 2064, 2, 1), (300, 1540, 2064, 16, 2), (2048, 1536, 2048, 128, 8),
                 (60, 9000, 1040, 3, 4), (1000, 600, 144, 12, 8), (8192, 260, 768, 200, 8), (30, 33, 528, 1000, 6)]


@pytest.mark.parametrize("tokens,m,n,experts,top_k", LARGE_GROUPED)
@pytest.mark.parametrize("shared", [True, False])
def test_grouped_large_tiles(tokens, m, n, experts, top_k, shared):
    """Each tile shape over ragged groups: an even routing with one crowded expert, some without pairs, some ids that are no expert."""
    dev = device()
    import torch
    say("int8 grouped large", tokens, m, n, experts, top_k, shared)
    g = torch.Generator(device=dev).manual_seed(tokens + m + n)
    q = lambda *s: torch.randint(-128, 128, s, generator=g, device=dev, dtype=torch.int8)
    pairs, ppr = tokens * top_k, top_k if shared else 1
    sel = torch.randint(-1, experts, (pairs,), generator=g, device=dev, dtype=torch.int32)
    if experts > 3:
        sel[torch.rand(pairs, generator=g, device=dev) < 0.2] = 1
        sel[sel == 2] = 3
    off, order = tg.moe_group(sel, experts)
    xq, wq = q(pairs // ppr, n), q(experts, m, n)
    xs = torch.rand(pairs // ppr, generator=g, device=dev) * 0.01 + 0.001
    ws = torch.rand(experts, m, generator=g, device=dev) * 0.01 + 0.001
    Y = torch.full((pairs, m), 9.0, device=dev)
    tg.int8_gemm_grouped(tg.Int8Experts(wq, ws), xq, xs, off, order, ppr, Y=Y)
    torch.cuda.synchronize()
    rows = torch.arange(pairs, device=dev) // ppr
    for e in range(-1, experts):
        p = (sel == e).nonzero()[:, 0]
        if e < 0:
            assert bool((Y[p] == 9).all())
        elif len(p):
            _near_on_device(torch, Y[p], _device_ref(torch, xq[rows[p]], xs[rows[p]], wq[e], ws[e]), "float32")


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_largest_sums(M):
    """-128 * -128 over the longest axis: 2^31 - 2^18, still inside int32."""
    dev = device()
    import torch
    say("int8 gemm largest sums", M)
    n = 131056
    xq = torch.full((M, n), -128, dtype=torch.int8, device=dev)
    L = tg.Int8Layer(torch.full((20, n), -128, dtype=torch.int8, device=dev), torch.ones(20, device=dev))
    y = tg.int8_gemm(L, xq, torch.ones(M, device=dev))
    torch.cuda.synchronize()
    assert bool((y == float(128 * 128 * n)).all())


def test_gemm_scales_carry_nan_and_zero():
    """A row whose scale is NaN (a non-finite token) gives NaN outputs in its row alone; a zero scale gives zeros."""
    dev = device()
    import torch
    say("int8 gemm scales")
    x = torch.randn(5, 64, generator=torch.Generator().manual_seed(3)).to(dev)
    x[1, 7], x[3] = float("inf"), 0.0
    q, s = tg.int8_quantize(x)
    L = tg.Int8Layer.from_dense(torch.randn(40, 64, generator=torch.Generator().manual_seed(4)).to(dev))
    y = tg.int8_gemm(L, q, s)
    torch.cuda.synchronize()
    assert bool(y[1].isnan().all()) and bool((y[3] == 0).all()) and bool(y[[0, 2, 4]].isfinite().all())


@pytest.mark.parametrize("lead,dtype", [((), "float16"), ((1,), "float16"), ((3, 5), "bfloat16"), ((200,), "float32")])
def test_int8_linear_equals_its_two_calls(lead, dtype):
    dev = device()
    import torch
    say("int8 linear", lead, dtype)
    g = torch.Generator().manual_seed(8)
    L = tg.Int8Layer.from_dense(torch.randn(300, 512, generator=g).to(dev))
    x = torch.randn(*lead, 512, generator=g).to(getattr(torch, dtype)).to(dev)
    y = tg.Int8Linear(L)(x)
    assert y.shape == lead + (300,) and y.dtype == torch.float32
    xq, xs = oracle.quantize(x.reshape(-1, 512).double().cpu().numpy())
    got_q, got_s = tg.int8_quantize(x.reshape(-1, 512))
    assert np.array_equal(got_q.cpu().numpy(), xq)
    _near(y.reshape(-1, 300), oracle.gemm(xq, got_s.cpu().numpy(), L.q.cpu().numpy(), L.scales.cpu().numpy()), "float32")


GROUPED = [  # tokens, experts, top_k, m, n, pairs_per_row == top_k
    (1, 8, 1, 16, 16, True), (1, 128, 8, 96, 256, True), (3, 4, 2, 130, 272, False), (20, 60, 4, 65, 48, True), (64, 128, 8, 128, 512, True),
    (130, 5, 2, 257, 144, False), (300, 8, 3, 256, 640, True), (300, 2, 1, 515, 128, True), (700, 16, 6, 300, 272, False), (513, 3, 2, 512, 1024, True),
    (40, 1024, 8, 32, 64, True), (600, 1, 1, 260, 400, False)]


def _grouped_ref(xq, xs, wq, ws, off, order, ppr, pairs, m):
    ref = np.full((pairs, m), 9.0)
    acc = {}
    for e in range(len(off) - 1):
        p = order[off[e]:off[e + 1]]
        if len(p):
            ref[p] = oracle.gemm(xq[p // ppr], xs[p // ppr], wq[e], ws[e])
    return ref


@pytest.mark.parametrize("tokens,experts,top_k,m,n,shared", GROUPED)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_grouped_matches_oracle(tokens, experts, top_k, m, n, shared, dtype):
    """Ragged groups (empty ones, one very long one), ids that are no expert, rows without an expert left as they were."""
    dev = device()
    import torch
    say("int8 grouped", tokens, experts, top_k, m, n, shared, dtype)
    rng = np.random.default_rng(tokens * 13 + experts + m)
    sel = rng.integers(-1, experts, (tokens, top_k))
    if experts > 4:
        sel[rng.random(sel.shape) < 0.4] = 3                       # one crowded expert
        sel[sel == 2] = 1                                          # one empty one
    off, order = route_oracle.group(sel, experts)
    pairs, ppr = tokens * top_k, top_k if shared else 1
    rows = pairs // ppr
    xq = rng.integers(-128, 128, (rows, n)).astype(np.int8)
    wq = rng.integers(-128, 128, (experts, m, n)).astype(np.int8)
    xs = (rng.random(rows) * 0.02 + 0.001).astype(np.float32)
    ws = (rng.random((experts, m)) * 0.02 + 0.001).astype(np.float32)
    E = tg.Int8Experts(torch.from_numpy(wq).to(dev), torch.from_numpy(ws).to(dev))
    got_off, got_order = tg.moe_group(torch.from_numpy(sel.astype(np.int32)).to(dev), experts)
    Y = torch.full((pairs, m), 9.0, dtype=getattr(torch, dtype), device=dev)
    tg.int8_gemm_grouped(E, torch.from_numpy(xq).to(dev), torch.from_numpy(xs).to(dev), got_off, got_order, ppr, Y=Y)
    torch.cuda.synchronize()
    _near(Y, _grouped_ref(xq, xs, wq, ws, off, order, ppr, pairs, m), dtype)


def test_grouped_cuts_bad_offsets_and_pairs():
    """Offsets outside [0, pairs] and entries of order outside it write nothing and read nothing out of range."""
    dev = device()
    import torch
    say("int8 grouped bad offsets")
    g = torch.Generator().manual_seed(9)
    E = tg.Int8Experts.from_dense(torch.randn(3, 40, 64, generator=g).to(dev))
    q, s = tg.int8_quantize(torch.randn(6, 64, generator=g).to(dev))
    off = torch.tensor([-5, 2, 1, 1 << 30], dtype=torch.int32, device=dev)         # expert 0: 0..2, 1: none, 2: 1..6
    order = torch.tensor([0, 3, 6, -1, 1 << 30, 5], dtype=torch.int32, device=dev)
    Y = torch.full((6, 40), 9.0, device=dev)
    tg.int8_gemm_grouped(E, q, s, off, order, Y=Y)
    torch.cuda.synchronize()
    ref = lambda e, p: oracle.gemm(q[p:p + 1].cpu().numpy(), s[p:p + 1].cpu().numpy(), E.q[e].cpu().numpy(), E.scales[e].cpu().numpy())
    _near(Y[0:1], ref(0, 0), "float32")
    _near(Y[5:6], ref(2, 5), "float32")
    assert bool((Y[[1, 2, 4]] == 9).all())                                          # pair 3 is listed for two experts: either's


def test_grouped_chain_equals_expert_by_expert():
    """A whole block over many tokens: router logits (8-bit layer), route, group, quantise, gate/up, silu * up, quantise, down, combine --
    against the same block with dense products expert by expert on the dequantised values."""
    dev = device()
    import torch
    say("int8 moe chain")
    g = torch.Generator().manual_seed(21)
    tokens, experts, top_k, hidden, inter = 70, 16, 4, 256, 96
    router = tg.Int8Linear(tg.Int8Layer.from_dense((torch.randn(experts, hidden, generator=g) * 0.1).to(dev)))
    gu = tg.Int8Experts.from_dense((torch.randn(experts, 2 * inter, hidden, generator=g) * 0.06).to(dev))
    dn = tg.Int8Experts.from_dense((torch.randn(experts, hidden, inter, generator=g) * 0.1).to(dev))
    x = torch.randn(tokens, hidden, generator=g).half().to(dev)
    sel, w = tg.moe_route(router(x), top_k)
    off, order = tg.moe_group(sel, experts)
    xq, xs = tg.int8_quantize(x)
    h = tg.int8_gemm_grouped(gu, xq, xs, off, order, pairs_per_row=top_k)
    a = (torch.nn.functional.silu(h[:, :inter]) * h[:, inter:]).half()
    aq, as_ = tg.int8_quantize(a)
    y = (tg.int8_gemm_grouped(dn, aq, as_, off, order).view(tokens, top_k, hidden) * w[..., None]).sum(1)
    torch.cuda.synchronize()
    deq = lambda q, s: q.double().cpu() * s.double().cpu()[..., None]
    X, GU, DN, A = deq(xq, xs), deq(gu.q, gu.scales), deq(dn.q, dn.scales), deq(aq, as_)
    S, W = sel.cpu(), w.double().cpu()
    hr = torch.stack([GU[S[t, i]] @ X[t] for t in range(tokens) for i in range(top_k)])
    assert torch.allclose(h.double().cpu(), hr, rtol=TOL["float32"] + 1e-12, atol=1e-12)
    yr = torch.stack([sum(W[t, i] * (DN[S[t, i]] @ A[t * top_k + i]) for i in range(top_k)) for t in range(tokens)])
    # the combine's products and sums of top_k terms in binary32, relative to the terms' sizes
    size = torch.stack([sum(W[t, i].abs() * (DN[S[t, i]] @ A[t * top_k + i]).abs() for i in range(top_k)) for t in range(tokens)])
    assert bool(((y.double().cpu() - yr).abs() <= (TOL["float32"] + (top_k + 1) * STEP) * 1.001 * size + 1e-12).all())

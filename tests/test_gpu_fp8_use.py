"""The norm and e4m3 operators as a program uses them: one behind the other, in captured graphs, on named streams, with shared
workspaces, at the ends of their ranges."""
import numpy as np
import pytest

from gpu_common import device, rel_err, say
from oracle import fp8 as oracle
from oracle import int8 as int8_oracle
from test_gpu_fp8 import HALF, STEP, _codes, _f8
from trellis_coded_gemv_amd import binding as tg
from trellis_coded_gemv_amd import inputs

pytestmark = pytest.mark.gpu


def _host(t):
    return t.double().cpu().numpy()


def _product_bound(xq, xs, wq, ws, dtype, ref):
    """Of any e4m3 values: 128 additions to a block's sum, each off by 2^-23 of the sum of magnitudes (32-bit outputs), or eight products
    aligned to the largest of them, each off by 2^-10 of it at most (16-bit outputs); the scales' product and the sums' additions."""
    most = oracle.gemm(np.abs(xq), xs, np.abs(wq), ws)
    rel, least = HALF[dtype]
    each = 128 * 2.0 ** -23 if dtype == "float32" else 8 * 2.0 ** -10 + 2.0 ** -16
    return (each + (xs.shape[1] + 10) * STEP) * most * (1 + rel) + rel * np.abs(ref) + least


def _check_product(y, xq, xs, wq, ws, dtype="float32"):
    a, s, w, t = _host(xq.float()), _host(xs), _host(wq.float()), _host(ws)
    ref = oracle.gemm(a, s, w, t)
    assert np.all(np.abs(_host(y) - ref) <= _product_bound(a, s, w, t, dtype, ref))


@pytest.mark.parametrize("rows", [1, 5, 200])
def test_norm_in_front_of_every_kind_of_layer(rows):
    """One residual stream, its norm in the form that each kind of layer reads."""
    dev = device()
    import torch
    say("norm in front of layers", rows)
    g = torch.Generator().manual_seed(rows)
    n, m = 512, 384
    x, stream = torch.randn(rows, n, generator=g).to(dev), torch.randn(rows, n, generator=g).bfloat16().to(dev)
    w = (torch.rand(n, generator=g) + 0.5).to(dev)
    dense = torch.randn(m, n, generator=g) / 16

    q, s, total = tg.rms_norm(x, w, residual=stream, out_dtype=torch.float8_e4m3fn)
    F = tg.Fp8Layer.from_dense(dense.to(dev))
    _check_product(tg.fp8_gemm(F, q, s), q, s, F.q, F.scales)

    q, s, again = tg.rms_norm(x, w, residual=stream, out_dtype=torch.int8)
    assert torch.equal(total, again)
    I = tg.Int8Layer.from_dense(dense.to(dev))
    y = tg.int8_gemm(I, q, s)
    ref = int8_oracle.gemm(q.cpu().numpy(), s.cpu().numpy(), I.q.cpu().numpy(), I.scales.cpu().numpy())
    assert np.all(np.abs(_host(y) - ref) <= 4 * STEP * np.abs(ref) + 2.0 ** -149)

    h, again = tg.rms_norm(x, w, residual=stream, out_dtype=torch.float16)
    assert torch.equal(total, again) and h.dtype == torch.float16
    arr = inputs.make_layer(256, n, 3, 5)
    from oracle import gemv as trellis_oracle
    y = tg.TrellisLinear(tg.DeviceLayer(arr, dev)).forward(h)
    bits = h.cpu().numpy().view(np.uint16)
    for r in {0, rows - 1}:
        assert rel_err(y[r].cpu().numpy(), trellis_oracle.gemv(arr, bits[r])) <= 1e-3


def test_linear():
    """Fp8Linear is its quantiser and its product; its workspace grows with the rows and serves smaller counts again."""
    dev = device()
    import torch
    say("fp8 linear")
    g = torch.Generator().manual_seed(3)
    n, m = 4112, 300
    L = tg.Fp8Layer.from_dense((torch.randn(m, n, generator=g) / 64).to(dev))
    f, half = tg.Fp8Linear(L), tg.Fp8Linear(L, out_dtype=torch.bfloat16)
    first = None
    for shape in ((n,), (3, n), (2, 40, n), (700, n), (1, n), (61, n)):
        x = torch.randn(*shape, generator=g).half().to(dev)
        y = f(x)
        q, s = tg.fp8_quantize(x.reshape(-1, n))
        assert y.shape == shape[:-1] + (m,) and y.dtype == torch.float32
        assert torch.equal(y.reshape(-1, m), tg.fp8_gemm(L, q, s))
        assert half(x).dtype == torch.bfloat16 and torch.equal(half(x).reshape(-1, m), tg.fp8_gemm(L, q, s, out_dtype=torch.bfloat16))
        first = y if first is None else first
        _check_product(y.reshape(-1, m)[:8], q[:8], s[:8], L.q, L.scales)
    with pytest.raises(ValueError):
        f(torch.zeros(3, n + 16, device=dev))


def _silu_mul(torch, gu):
    g, u = gu.float().chunk(2, -1)
    return torch.nn.functional.silu(g) * u


def _block(torch, x, stream, w, router, gate_up, down, top_k, out_dtype):
    """Norm, routing and experts of a mixture-of-experts layer over many tokens; every intermediate, for the checks."""
    h, total = tg.rms_norm(x, w, residual=stream, out_dtype=torch.float32)
    q, s, _ = tg.rms_norm(x, w, residual=stream, out_dtype=torch.float8_e4m3fn)
    sel, weights = tg.moe_route(h @ router, top_k)
    offsets, order = tg.moe_group(sel, gate_up.experts)
    gu = tg.fp8_gemm_grouped(gate_up, q, s, offsets, order, pairs_per_row=top_k, out_dtype=out_dtype)
    a = _silu_mul(torch, gu)
    q2, s2 = tg.fp8_quantize(a)
    d = tg.fp8_gemm_grouped(down, q2, s2, offsets, order, out_dtype=out_dtype)
    y = (d.float().view(len(x), top_k, -1) * weights[..., None]).sum(1)
    return dict(total=total, q=q, s=s, sel=sel, gu=gu, q2=q2, s2=s2, d=d, y=y)


@pytest.mark.parametrize("tokens", [1, 7, 300])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_expert_block(tokens, dtype):
    dev = device()
    import torch
    say("fp8 expert block", tokens, dtype)
    g = torch.Generator().manual_seed(tokens)
    hidden, inter, experts, top_k = 272, 144, 12, 3
    rnd = lambda *s: torch.randn(*s, generator=g)
    x, stream, w = rnd(tokens, hidden).to(dev), rnd(tokens, hidden).half().to(dev), (torch.rand(hidden, generator=g) + 0.5).to(dev)
    router = (rnd(hidden, experts) / 8).to(dev)
    up = tg.Fp8Experts.from_dense((rnd(experts, 2 * inter, hidden) / 16).to(dev))
    down = tg.Fp8Experts.from_dense((rnd(experts, hidden, inter) / 12).to(dev))
    r = _block(torch, x, stream, w, router, up, down, top_k, getattr(torch, dtype))
    torch.cuda.synchronize()
    sel = r["sel"].cpu().numpy()
    for e in range(experts):
        p = np.flatnonzero(sel.reshape(-1) == e)
        if len(p):
            at, tok = torch.from_numpy(p).to(dev), torch.from_numpy(p // top_k).to(dev)
            _check_product(r["gu"][at], r["q"].float()[tok], r["s"][tok], up.q[e], up.scales[e], dtype)
            _check_product(r["d"][at], r["q2"].float()[at], r["s2"][at], down.q[e], down.scales[e], dtype)


def test_captured_graph():
    """A captured step replayed on changing inputs, with eager work and synchronisation between, gives the eager results' bits."""
    dev = device()
    import torch
    say("fp8 captured graph")
    g = torch.Generator().manual_seed(1)
    tokens, hidden, inter, experts, top_k = 24, 4112, 144, 12, 3
    rnd = lambda *s: torch.randn(*s, generator=g).to(dev)
    w, router = rnd(hidden).abs() + 0.5, rnd(hidden, experts) / 64
    up, down = tg.Fp8Experts.from_dense(rnd(experts, 2 * inter, hidden) / 64), tg.Fp8Experts.from_dense(rnd(experts, hidden, inter) / 12)
    L = tg.Fp8Layer.from_dense(rnd(700, hidden) / 64)               # a split inner axis: the workspace's counters are in use
    lin = tg.Fp8Linear(L)
    x, stream = rnd(tokens, hidden), rnd(tokens, hidden).bfloat16()

    def run():
        r = _block(torch, x, stream, w, router, up, down, top_k, torch.float32)
        return [r["total"], r["q"].view(torch.uint8), r["s"], r["gu"], r["d"], lin(x), lin(r["total"])]
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        x.copy_(rnd(tokens, hidden) * (i + 1))
        stream.copy_(rnd(tokens, hidden))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, run()):
            assert torch.equal(a, b)


def test_two_graphs_share_a_workspace():
    dev = device()
    import torch
    say("fp8 two graphs, one workspace")
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dev)
    layers = [tg.Fp8Layer.from_dense(rnd(m, n) / 64) for m, n in ((1024, 8192), (300, 4112))]
    ints = tg.Int8Layer.from_dense(rnd(512, 8192) / 64)
    rows = [(tg.fp8_quantize(rnd(M, L.n))) for M, L in zip((61, 17), layers)]
    iq = tg.int8_quantize(rnd(33, 8192))
    size = max([tg.fp8_workspace(L, len(r[0])).numel() for L, r in zip(layers, rows)] + [tg.int8_workspace(ints, 33).numel()])
    ws = torch.zeros(size, dtype=torch.uint8, device=dev)
    calls = [lambda: tg.fp8_gemm(layers[0], *rows[0], ws=ws), lambda: tg.fp8_gemm(layers[1], *rows[1], ws=ws, out_dtype=torch.float16),
             lambda: tg.int8_gemm(ints, *iq, ws=ws)]
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(c())
        graphs.append(graph)
    for i in (0, 1, 2, 1, 0, 0, 2, 2, 1):
        outs[i].fill_(7)
        graphs[i].replay()
        assert torch.equal(calls[(i + 1) % 3](), want[(i + 1) % 3])
        assert torch.equal(outs[i], want[i])


def test_streams():
    """A named stream orders a call behind that stream's work; calls on two streams with a workspace each do not disturb each other."""
    dev = device()
    import torch
    say("fp8 streams")
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dev)
    L = tg.Fp8Layer.from_dense(rnd(512, 4096) / 64)
    x, w = rnd(48, 4096), rnd(4096).abs() + 0.5
    E = tg.Fp8Experts.from_dense(rnd(4, 128, 4096) / 64)
    sel = torch.randint(0, 4, (48, 1), generator=g).int().to(dev)

    def chain(stream=None, ws=None):
        q, s = tg.rms_norm(x, w, out_dtype=torch.float8_e4m3fn, stream=stream)
        q2, s2 = tg.fp8_quantize(x, stream=stream)
        offsets, order = tg.moe_group(sel, 4, stream=stream)
        return [tg.fp8_gemm(L, q, s, ws=ws, stream=stream), tg.fp8_gemm_grouped(E, q2, s2, offsets, order, stream=stream), tg.Fp8Linear(L)(x, stream=stream)]
    want = chain()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    wa, wb = tg.fp8_workspace(L, 48), tg.fp8_workspace(L, 48)
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        got.append(chain(a, wa))
        got.append(chain(b.cuda_stream, wb))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(p, q) for p, q in zip(r, want))
    with torch.cuda.stream(a):
        other = chain()
    a.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(other, want))


def _near_rows(torch, y, xq, xs, wq, ws, outs):
    """Outputs `outs` (their layer rows wq, and the scales of each output's block ws [outs, blocks]) of values whose block sums are exact."""
    sums = oracle.block_sums(oracle.values(xq), oracle.values(wq))
    scales = xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None]
    ref = (sums * scales).sum(2)
    assert np.all(np.abs(_host(y) - ref) <= (sums.shape[2] + 10) * STEP * (np.abs(sums) * scales).sum(2))


def test_offsets_beyond_32_bits():
    """Layers, rows and outputs of more than 2^32 bytes, and rows far apart."""
    dev = device()
    import torch
    say("fp8 wide offsets")
    rng = np.random.default_rng(9)
    m, n = 540000, 8192                                             # a layer of 4.4 GB
    wq = torch.full((m, n), 0x38, dtype=torch.uint8, device=dev)    # ones
    outs = np.array([0, 127, 128, 262143, 524287, 524288, 524289, m - 2, m - 1])
    codes = _codes(rng, (len(outs), n))
    wq[torch.from_numpy(outs).to(dev)] = torch.from_numpy(codes).to(dev)
    blocks = (m + 127) // 128
    ws = torch.rand(blocks, n // 128, device=dev) * 0.01 + 0.001
    L = tg.Fp8Layer(wq.view(torch.float8_e4m3fn), ws)
    for M in (1, 300):
        xq, xs = _codes(rng, (M, n)), (rng.random((M, n // 128)) * 0.01 + 0.001).astype(np.float32)
        y = tg.fp8_gemm(L, _f8(torch, xq, dev), torch.from_numpy(xs).to(dev))
        at = torch.from_numpy(outs).to(dev)
        _near_rows(torch, y[:, at], xq, xs, codes, ws[at // 128].cpu().numpy(), outs)
        del y
    E = tg.Fp8Experts(wq[:524288].view(8, 65536, n).view(torch.float8_e4m3fn), ws[:4096].view(8, 512, n // 128).contiguous())
    xq, xs = _codes(rng, (3, n)), (rng.random((3, n // 128)) * 0.01 + 0.001).astype(np.float32)
    y = tg.fp8_gemm_grouped(E, _f8(torch, xq, dev), torch.from_numpy(xs).to(dev), *tg.moe_group(torch.tensor([0, 7, 7], dtype=torch.int32, device=dev), 8))
    at = torch.from_numpy(outs[4:5]).to(dev)                        # the last output of the last expert
    _near_rows(torch, y[1:, at - 7 * 65536], xq[1:], xs[1:], codes[4:5], ws[at // 128].cpu().numpy(), outs[4:5])
    del L, E, wq, y
    wide = torch.zeros(3, 1 << 31, dtype=torch.float16, device=dev)[:, :5000]     # rows 4 GiB apart
    rows = torch.randn(3, 5000, generator=torch.Generator().manual_seed(1)).half().to(dev)
    wide.copy_(rows)
    w = torch.rand(5000, device=dev).half()
    for out in (torch.float16, torch.int8, torch.float8_e4m3fn):
        for a, b in zip(tg.rms_norm(wide, w, residual=wide, out_dtype=out), tg.rms_norm(rows, w, residual=rows, out_dtype=out)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for a, b in zip(tg.fp8_quantize(wide), tg.fp8_quantize(rows)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_ends_of_the_ranges():
    dev = device()
    import torch
    say("fp8 ends of ranges")
    rng = np.random.default_rng(10)
    n = 131056                                                      # the longest inner axis of a product
    xq, wq = _codes(rng, (2, n)), _codes(rng, (40, n))
    xs, ws = (rng.random((2, 1024)) * 0.01).astype(np.float32), (rng.random((1, 1024)) * 0.01).astype(np.float32)
    y = tg.fp8_gemm(tg.Fp8Layer(_f8(torch, wq, dev), torch.from_numpy(ws).to(dev)), _f8(torch, xq, dev), torch.from_numpy(xs).to(dev))
    _near_rows(torch, y, xq, xs, wq, np.repeat(ws, 40, 0), np.arange(40))
    x = torch.randn(1, 1 << 22, generator=torch.Generator().manual_seed(1))      # the longest row of the quantiser
    q, s = tg.fp8_quantize(x.to(dev))
    for at in (0, 77 * 128, (1 << 22) - 128):
        c, t = oracle.quantize(x[:, at:at + 128].double().numpy())
        assert np.array_equal(q[:, at:at + 128].contiguous().view(torch.uint8).cpu().numpy(), c)
        assert abs(float(s[0, at // 128]) - t[0, 0]) <= STEP * t[0, 0]
    sel = torch.from_numpy(rng.permutation(1024).astype(np.int32)).to(dev)       # as many experts as there may be, a pair each
    xq, xs = _codes(rng, (1024, 32)), (rng.random((1024, 1)) * 0.01).astype(np.float32)
    wq, ws = _codes(rng, (1024, 33, 32)), (rng.random((1024, 1, 1)) * 0.01).astype(np.float32)
    E = tg.Fp8Experts(_f8(torch, wq, dev), torch.from_numpy(ws).to(dev))
    y = tg.fp8_gemm_grouped(E, _f8(torch, xq, dev), torch.from_numpy(xs).to(dev), *tg.moe_group(sel, 1024))
    e = sel.cpu().numpy()
    ref = np.einsum("pi,poi->po", oracle.values(xq), oracle.values(wq)[e]) * xs * ws[e][:, 0]
    assert np.all(np.abs(_host(y) - ref) <= 12 * STEP * np.abs(ref))
    one = tg.fp8_gemm_grouped(E, _f8(torch, xq, dev), torch.from_numpy(xs).to(dev), *tg.moe_group(torch.full((1024,), 1023, dtype=torch.int32, device=dev), 1024))
    ref = oracle.gemm(oracle.values(xq), xs, oracle.values(wq[1023]), ws[1023])
    assert np.all(np.abs(_host(one) - ref) <= 12 * STEP * np.abs(ref))


def test_workspace_refusals_on_the_device():
    dev = device()
    import torch
    say("fp8 workspace refusals")
    L = tg.Fp8Layer.from_dense(torch.randn(1024, 8192, device=dev))
    q, s = tg.fp8_quantize(torch.randn(61, 8192, device=dev))
    with pytest.raises(tg.TgError):
        tg.fp8_gemm(L, q, s, ws=torch.zeros(4096, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError):
        tg.fp8_gemm(L, q, s, ws=torch.zeros(1 << 26, dtype=torch.uint8, device=dev)[::2])
    with pytest.raises(ValueError):
        tg.fp8_gemm(L, q, s, Y=torch.zeros(61, 1024, device=dev), out_dtype=torch.float16)
    with pytest.raises(ValueError):
        tg.fp8_gemm(L, q, s.t().contiguous().t())                   # a row's scales apart
    with pytest.raises(tg.TgError):
        tg.fp8_gemm(L, q[:1].expand(61, 8192), s)                   # rows that share their memory


def test_experts_from_dense_on_a_stream():
    """Made on a named stream while the current one still writes memory that it has given back."""
    dev = device()
    import torch
    say("fp8 experts from dense on a stream")
    weight = torch.randn(4, 1024, 2048, generator=torch.Generator().manual_seed(6)).to(dev)
    want = tg.Fp8Experts.from_dense(weight)
    a, big = torch.cuda.Stream(), torch.randn(4096, 4096, device=dev)
    torch.cuda.synchronize()
    for stream in (a, a.cuda_stream, a):
        given_back = [torch.empty(4, 1024, 2048, dtype=torch.uint8, device=dev), torch.empty(4, 8, 16, device=dev)]
        for _ in range(4):
            big @ big                                               # the writes below come after this
        for t in given_back:
            t.fill_(77)
        del given_back, t
        E = tg.Fp8Experts.from_dense(weight, stream=stream)
        a.synchronize()
        q, s = E.q.view(torch.uint8).clone(), E.scales.clone()
        assert torch.equal(q, want.q.view(torch.uint8)) and torch.equal(s, want.scales)

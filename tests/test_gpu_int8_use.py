"""The routing and 8-bit entry points as programs use them: in captured graphs that are replayed, on other streams, two
graphs over one workspace, together with the trellis-coded block, and over tensors beyond 32-bit offsets."""
import numpy as np
import pytest

from gpu_common import REL_TOL, device, rel_err, say
from oracle import moe
from trellis_coded_gemv_amd import binding as tg
from trellis_coded_gemv_amd import inputs

pytestmark = pytest.mark.gpu


def _capture(torch, fn):
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            fn()
    torch.cuda.synchronize()
    return g


def _layer(torch, dev, m, n, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    return tg.Int8Layer(torch.randint(-128, 128, (m, n), generator=g, device=dev, dtype=torch.int8), torch.rand(m, generator=g, device=dev) + 0.5)


def _rows(torch, dev, M, n, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randint(-128, 128, (M, n), generator=g, device=dev, dtype=torch.int8), torch.rand(M, generator=g, device=dev) + 0.5


@pytest.mark.parametrize("M,m,n", [(1, 4096, 14336), (61, 4096, 14336), (256, 4096, 14336), (600, 8000, 4112)])
def test_graph_gemm(M, m, n):
    """Replays with eager work on the same workspace between them (split inner axes leave their counters at zero)."""
    dev = device()
    import torch
    say("graph int8 gemm", M, m, n)
    L = _layer(torch, dev, m, n, 1)
    xq, xs = _rows(torch, dev, M, n, 2)
    other = _layer(torch, dev, 512, 2048, 3)
    oq, os_ = _rows(torch, dev, 40, 2048, 4)
    ws = torch.zeros(max(tg.int8_workspace(L, M).numel(), tg.int8_workspace(other, 40).numel()), dtype=torch.uint8, device=dev)
    ref, oref = tg.int8_gemm(L, xq, xs, ws=ws).clone(), tg.int8_gemm(other, oq, os_, ws=ws).clone()
    Y = torch.empty_like(ref)
    g = _capture(torch, lambda: tg.int8_gemm(L, xq, xs, Y=Y, ws=ws))
    for r in range(4):
        Y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, ref), r
        assert torch.equal(tg.int8_gemm(other, oq, os_, ws=ws), oref)
        torch.cuda.synchronize()


def test_two_graphs_share_a_workspace_on_one_stream():
    dev = device()
    import torch
    say("two graphs, one workspace")
    A, B = _layer(torch, dev, 4096, 14336, 5), _layer(torch, dev, 1024, 8192, 6)
    a, b = _rows(torch, dev, 64, 14336, 7), _rows(torch, dev, 64, 8192, 8)
    ws = torch.zeros(max(tg.int8_workspace(A, 64).numel(), tg.int8_workspace(B, 64).numel()), dtype=torch.uint8, device=dev)
    ra, rb = tg.int8_gemm(A, *a, ws=ws).clone(), tg.int8_gemm(B, *b, ws=ws).clone()
    ya, yb = torch.empty_like(ra), torch.empty_like(rb)
    ga, gb = _capture(torch, lambda: tg.int8_gemm(A, *a, Y=ya, ws=ws)), _capture(torch, lambda: tg.int8_gemm(B, *b, Y=yb, ws=ws))
    for _ in range(3):
        ya.zero_()
        yb.zero_()
        ga.replay()
        gb.replay()
        ga.replay()
        torch.cuda.synchronize()
        assert torch.equal(ya, ra) and torch.equal(yb, rb)


def test_first_linear_call_under_capture():
    """The workspace of a layer first used (or first used with so many rows) inside a capture is the graph's: eager calls before
    the first replay and between replays have their own."""
    dev = device()
    import torch
    say("int8 linear first called under capture")
    L = _layer(torch, dev, 4096, 14336, 21)
    xs = [torch.randn(r, 14336, generator=torch.Generator().manual_seed(22 + r)).half().to(dev) for r in (61, 128)]
    refs = [tg.Int8Linear(L)(x).clone() for x in xs]
    lin, outs = tg.Int8Linear(L), [torch.empty_like(r) for r in refs]
    graphs = []
    for x, out, ref in zip(xs, outs, refs):
        graphs.append(_capture(torch, lambda: out.copy_(lin(x))))
        assert torch.equal(lin(x), ref)                              # before its graph has run
    for _ in range(3):
        for x, out, ref, g in zip(xs, outs, refs, graphs):
            out.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref) and torch.equal(lin(x), ref)


def test_workspace_refused():
    dev = device()
    import torch
    L = _layer(torch, dev, 64, 2048, 30)
    xq, xs = _rows(torch, dev, 4, 2048, 31)
    need = tg.int8_workspace(L, 4).numel()
    with pytest.raises(ValueError, match="contiguous"):
        tg.int8_gemm(L, xq, xs, ws=torch.zeros(1, dtype=torch.uint8, device=dev).expand(2 * need))
    with pytest.raises(tg.TgError):
        tg.int8_gemm(L, xq, xs, ws=torch.zeros(need - 256, dtype=torch.uint8, device=dev))


def _block(torch, x, router, gu, dn, top_k, out):
    """Router, groups, both expert products and the combine of a block over many tokens."""
    tokens, hidden = x.shape
    inter = dn.n
    sel, w = tg.moe_route(router(x), top_k, sigmoid=True, n_group=4, topk_group=2, group_top=2)
    off, order = tg.moe_group(sel, gu.experts)
    xq, xs = tg.int8_quantize(x)
    h = tg.int8_gemm_grouped(gu, xq, xs, off, order, pairs_per_row=top_k)
    a = (torch.nn.functional.silu(h[:, :inter]) * h[:, inter:]).half()
    aq, as_ = tg.int8_quantize(a)
    y = tg.int8_gemm_grouped(dn, aq, as_, off, order, out_dtype=torch.bfloat16)
    torch.mul(y.view(tokens, top_k, hidden), w[..., None], out=out)


@pytest.mark.parametrize("tokens", [1, 300])
def test_graph_block(tokens):
    dev = device()
    import torch
    say("graph int8 block", tokens)
    g = torch.Generator().manual_seed(31)
    experts, top_k, hidden, inter = 16, 4, 512, 192
    router = tg.Int8Linear(tg.Int8Layer.from_dense((torch.randn(experts, hidden, generator=g) * 0.1).to(dev)))
    gu = tg.Int8Experts.from_dense((torch.randn(experts, 2 * inter, hidden, generator=g) * 0.06).to(dev))
    dn = tg.Int8Experts.from_dense((torch.randn(experts, hidden, inter, generator=g) * 0.1).to(dev))
    x = torch.randn(tokens, hidden, generator=g).half().to(dev)
    ref, out = (torch.empty(tokens, top_k, hidden, device=dev) for _ in range(2))
    _block(torch, x, router, gu, dn, top_k, ref)
    graph = _capture(torch, lambda: _block(torch, x, router, gu, dn, top_k, out))
    x2 = torch.randn(tokens, hidden, generator=g).half().to(dev)
    ref2 = torch.empty_like(ref)
    _block(torch, x2, router, gu, dn, top_k, ref2)
    x1 = x.clone()
    for r in range(4):
        out.fill_(float("nan"))
        x.copy_(x2 if r % 2 else x1)                                # new values under the same graph
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref2 if r % 2 else ref), r
        _block(torch, x2, router, gu, dn, top_k, torch.empty_like(ref))
        torch.cuda.synchronize()


def test_named_stream():
    """A call on a stream other than the current one: what it allocates belongs to that stream, and the result is the same."""
    dev = device()
    import torch
    say("int8 and route on a named stream")
    L = _layer(torch, dev, 4096, 14336, 9)
    x = torch.randn(50, 14336, generator=torch.Generator().manual_seed(10)).half().to(dev)
    l = torch.randn(500, 128, generator=torch.Generator().manual_seed(11)).to(dev)
    lin = tg.Int8Linear(L)
    ref = lin(x).clone()
    sel, w = tg.moe_route(l, 8)
    off, order = tg.moe_group(sel, 128)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for _ in range(5):
            junk = torch.empty(50, 4096, device=dev).fill_(7.0)     # work and memory of the current stream in between
            del junk
            y = lin.forward(x, stream=stream)
            sel2, w2 = tg.moe_route(l, 8, stream=stream)
            off2, order2 = tg.moe_group(sel2, 128, stream=stream)
        s.synchronize()
        assert torch.equal(y, ref) and torch.equal(sel2, sel) and torch.equal(w2, w) and torch.equal(off2, off) and torch.equal(order2, order)
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with a workspace of its own."""
    dev = device()
    import torch
    say("int8 and route on two streams at once")
    L = _layer(torch, dev, 4096, 14336, 40)
    rows = [_rows(torch, dev, 61, 14336, 41 + i) for i in range(2)]
    refs = [tg.int8_gemm(L, *r).clone() for r in rows]
    logits = [torch.randn(3000, 256, generator=torch.Generator().manual_seed(43 + i)).to(dev) for i in range(2)]
    routed = [tg.moe_route(l, 8) for l in logits]
    grouped = [tg.moe_group(r[0], 256) for r in routed]
    ws = [tg.int8_workspace(L, 61) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = []
        for i, st in enumerate(streams):
            y = tg.int8_gemm(L, *rows[i], ws=ws[i], stream=st)
            sel, w = tg.moe_route(logits[i], 8, stream=st)
            got.append((y, sel, w) + tuple(tg.moe_group(sel, 256, stream=st)))
        for st in streams:
            st.synchronize()
        for i in range(2):
            want = (refs[i],) + tuple(routed[i]) + tuple(grouped[i])
            assert all(torch.equal(a, b) for a, b in zip(got[i], want))


def test_expanded_inputs_refused():
    """Rows that all lie at one place (a broadcast view) are no layout of these entry points."""
    dev = device()
    import torch
    L = _layer(torch, dev, 64, 256, 50)
    xq, xs = _rows(torch, dev, 1, 256, 51)
    with pytest.raises(tg.TgError):
        tg.int8_gemm(L, xq.expand(4, 256), torch.ones(4, device=dev))
    with pytest.raises(tg.TgError):
        tg.int8_quantize(torch.ones(1, 64, device=dev).expand(4, 64))
    with pytest.raises(tg.TgError):
        tg.moe_route(torch.ones(1, 64, device=dev).expand(4, 64), 2)
    with pytest.raises(ValueError):
        tg.int8_gemm(L, xq.expand(4, 256).contiguous(), torch.ones(1, device=dev).expand(4))


def test_route_feeds_the_trellis_block():
    """Router logits of an 8-bit layer -> moe_route -> trellis_moe_block, token by token, against the oracles; a masked router
    leaves slots without an expert, which the block skips."""
    dev = device()
    import torch
    say("route -> trellis moe block")
    wl = inputs.MoEWorkload(experts=8, tokens=3)
    gu = [wl.layer(e, w) for e in range(8) for w in ("gate", "up")]
    dn = [wl.layer(e, "down") for e in range(8)]
    gut = tg.LayerTable([tg.DeviceLayer(a, dev) for a in gu], dev)
    dnt = tg.LayerTable([tg.DeviceLayer(a, dev) for a in dn], dev)
    g = torch.Generator().manual_seed(12)
    router = tg.Int8Linear(tg.Int8Layer.from_dense((torch.randn(8, wl.hidden, generator=g) * 0.05).to(dev)))
    bits = inputs.make_x(wl.hidden, 4321, rows=3)
    x = tg.fp16_tensor(bits, dev)
    logits = router(x)
    logits[2, 2:] = float("-inf")                                   # two experts left for the third token
    sel, w = tg.moe_route(logits, 3)
    for t in range(3):
        y = tg.trellis_moe_block(gut, dnt, sel[t], w[t], x[t])
        torch.cuda.synchronize()
        ids, ws = sel[t].tolist(), w[t].double().tolist()
        assert (ids[2] == -1 and ws[2] == 0.0) == (t == 2)
        ref = moe.moe_block(gu, dn, [i for i in ids if i >= 0], [v for i, v in zip(ids, ws) if i >= 0], bits[t])
        assert rel_err(y.cpu().numpy(), ref) <= REL_TOL


def test_offsets_beyond_32_bits():
    """Weights and outputs of more than 4 GiB: the last rows are addressed as the first."""
    dev = device()
    import torch
    say("int8 beyond 4 GiB: weights")
    m, n = 300000, 16384                                            # 4.9e9 weights
    g = torch.Generator(device=dev).manual_seed(13)
    wq = torch.empty(m, n, dtype=torch.int8, device=dev)
    for i in range(0, m, 50000):
        wq[i:i + 50000] = torch.randint(-128, 128, (min(50000, m - i), n), generator=g, device=dev, dtype=torch.int8)
    ws = torch.rand(m, generator=g, device=dev) + 0.5
    xq, xs = _rows(torch, dev, 3, n, 14)
    y = tg.int8_gemm(tg.Int8Layer(wq, ws), xq, xs)
    E = tg.Int8Experts(wq.view(3, 100000, n), ws.view(3, 100000))
    sel = torch.tensor([2, 0, 2], dtype=torch.int32, device=dev)
    ye = tg.int8_gemm_grouped(E, xq, xs, *tg.moe_group(sel, 3))
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, 99999, 100000, 262143, 262144, 299998, 299999], device=dev)
    ref = (xq.double() @ wq[at].double().t()) * xs.double()[:, None] * ws[at].double()
    tol = (1 + 2.0 ** -24) ** 3 - 1
    assert bool(((y[:, at].double() - ref).abs() <= tol * ref.abs() + 1e-300).all())
    assert torch.equal(ye[0], y[0, 200000:]) and torch.equal(ye[1], y[1, :100000]) and torch.equal(ye[2], y[2, 200000:])
    del wq, E, y, ye
    torch.cuda.empty_cache()
    say("int8 beyond 4 GiB: outputs and activations")
    M, m, n = 70000, 66000, 16                                      # 4.6e9 outputs
    L = _layer(torch, dev, m, n, 15)
    xq, xs = _rows(torch, dev, M, n, 16)
    y = tg.int8_gemm(L, xq, xs, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 255, 256, 65535, 65536, 69999], device=dev)
    ref = (xq[rows].double() @ L.q.double().t()) * xs[rows].double()[:, None] * L.scales.double()
    assert bool(((y[rows].double() - ref).abs() <= ((1 + 2.0 ** -24) ** 3 * (1 + 2.0 ** -8) - 1) * ref.abs()).all())
    say("quantize beyond 4 GiB")
    del y
    torch.cuda.empty_cache()
    x = torch.zeros(2, 1 << 31, dtype=torch.bfloat16, device=dev)[:, :4096]     # rows 4 GiB apart
    x[1] = torch.randn(4096, generator=torch.Generator().manual_seed(17)).bfloat16().to(dev)
    q, s = tg.int8_quantize(x)
    q1, s1 = tg.int8_quantize(x[1].clone())
    assert torch.equal(q[1], q1) and float(s[1]) == float(s1) and not bool(q[0].any()) and float(s[0]) == 0.0


def test_same_inputs_twice_give_the_same_bits():
    dev = device()
    import torch
    say("int8 determinism")
    L = _layer(torch, dev, 4096, 14336, 18)
    xq, xs = _rows(torch, dev, 200, 14336, 19)
    ws = tg.int8_workspace(L, 200)
    first = tg.int8_gemm(L, xq, xs, ws=ws).clone()
    for _ in range(5):
        assert torch.equal(tg.int8_gemm(L, xq, xs, ws=ws), first)
    l = torch.randn(3000, 256, generator=torch.Generator().manual_seed(20)).to(dev)
    b = torch.zeros(256, device=dev)
    s0, w0 = tg.moe_route(l, 8, bias=b, sigmoid=True, n_group=8, topk_group=4, group_top=2)
    for _ in range(3):
        s, w = tg.moe_route(l, 8, bias=b, sigmoid=True, n_group=8, topk_group=4, group_top=2)
        assert torch.equal(s, s0) and torch.equal(w, w0)
    assert np.isfinite(w0.cpu().numpy()).all()

"""Refusals of the routing and 8-bit entry points: every call here fails a host check, so nothing reaches a device."""
import pytest

from trellis_coded_gemv_amd import binding as tg

A16 = 0x10000          # fake device addresses: never dereferenced


def _route(**kw):
    d = dict(tokens=4, experts=64, top_k=8, logits=A16, dtype=0, ld=64, bias=A16, n_group=8, topk_group=4, group_top=2,
             flags=3, scale=1.0, sel=A16, weights=A16, stream=None)
    d.update(kw)
    return tg.lib().moe_route(*d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), -2), (dict(tokens=(1 << 24) + 1), -2), (dict(experts=0), -2), (dict(experts=1025, ld=2048), -2),
    (dict(top_k=0), -8), (dict(top_k=65, experts=128, ld=128, topk_group=8), -8), (dict(top_k=33), -8),
    (dict(dtype=3), -8), (dict(dtype=-1), -8), (dict(ld=63), -8), (dict(n_group=0), -8), (dict(n_group=7), -8),
    (dict(n_group=128, experts=128, ld=128), -8), (dict(topk_group=0), -8), (dict(topk_group=9), -8), (dict(topk_group=1, top_k=9), -8),
    (dict(group_top=0), -8), (dict(group_top=3), -8), (dict(flags=4), -8), (dict(scale=float("nan")), -8),
    (dict(scale=float("inf")), -8), (dict(logits=0), -1), (dict(sel=0), -1), (dict(weights=0), -1),
    (dict(logits=A16 + 2), -4), (dict(logits=A16 + 1, dtype=1), -4), (dict(bias=A16 + 2), -4), (dict(sel=A16 + 1), -4),
    (dict(weights=A16 + 2), -4)])
def test_route_refusals(kw, status):
    assert _route(**kw) == status


@pytest.mark.parametrize("args,status", [
    ((0, 8, A16, A16, A16), -2), (((1 << 24) + 1, 8, A16, A16, A16), -2), ((8, 0, A16, A16, A16), -2),
    ((8, 1025, A16, A16, A16), -2), ((8, 8, 0, A16, A16), -1), ((8, 8, A16, 0, A16), -1), ((8, 8, A16, A16, 0), -1),
    ((8, 8, A16 + 2, A16, A16), -4), ((8, 8, A16, A16 + 2, A16), -4), ((8, 8, A16, A16, A16 + 1), -4)])
def test_group_refusals(args, status):
    assert tg.lib().moe_group(*args, None) == status


def _quantize(**kw):
    d = dict(rows=4, n=100, x=A16, dtype=1, ldx=100, q=A16, ldq=112, scales=A16, stream=None)
    d.update(kw)
    return tg.lib().int8_quantize(*d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), -2), (dict(rows=(1 << 24) + 1), -2), (dict(n=0), -2), (dict(n=(1 << 22) + 1), -2), (dict(dtype=3), -8),
    (dict(ldx=99), -8), (dict(ldq=99), -8), (dict(x=0), -1), (dict(q=0), -1), (dict(scales=0), -1), (dict(x=A16 + 1), -4),
    (dict(x=A16 + 2, dtype=0), -4), (dict(scales=A16 + 2), -4)])
def test_quantize_refusals(kw, status):
    assert _quantize(**kw) == status


def _gemm(**kw):
    d = dict(M=4, m=100, n=128, xq=A16, ldx=128, xs=A16, wq=A16, ldw=128, wscales=A16, Y=A16, out=0, ldy=100, ws=A16,
             ws_bytes=1 << 40, stream=None)
    d.update(kw)
    return tg.lib().int8_gemm(*d.values())


def _grouped(**kw):
    d = dict(pairs=8, experts=4, m=100, n=128, xq=A16, ldx=128, xs=A16, ppr=2, wq=A16, wscales=A16, offsets=A16, order=A16,
             Y=A16, out=0, ldy=100, stream=None)
    d.update(kw)
    return tg.lib().int8_gemm_grouped(*d.values())


SHARED = [(dict(m=0), -2), (dict(m=(1 << 22) + 1, ldy=1 << 23), -2), (dict(n=0), -2), (dict(n=120), -2),
          (dict(n=131072, ldx=131072), -2), (dict(ldx=112), -8), (dict(ldx=136), -8), (dict(ldy=99), -8), (dict(out=3), -8),
          (dict(xq=0), -1), (dict(xs=0), -1), (dict(wq=0), -1), (dict(wscales=0), -1), (dict(Y=0), -1),
          (dict(xq=A16 + 8), -4), (dict(wq=A16 + 8), -4), (dict(xs=A16 + 2), -4), (dict(wscales=A16 + 2), -4),
          (dict(Y=A16 + 2), -4), (dict(Y=A16 + 1, out=2), -4)]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(M=0), -2), (dict(M=(1 << 20) + 1), -2), (dict(ldw=112), -8), (dict(ldw=136), -8), (dict(ldw=(1 << 23) + 16), -8), (dict(ws=0), -5),
    (dict(ws_bytes=255), -5), (dict(ws=A16 + 16), -4)])
def test_gemm_refusals(kw, status):
    assert _gemm(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(pairs=0), -2), (dict(pairs=(1 << 20) + 2), -2), (dict(experts=0), -2), (dict(experts=1025), -2), (dict(ppr=0), -8),
    (dict(ppr=3), -8), (dict(offsets=0), -1), (dict(order=0), -1), (dict(offsets=A16 + 2), -4), (dict(order=A16 + 1), -4)])
def test_grouped_refusals(kw, status):
    assert _grouped(**kw) == status


def test_workspace_sizes():
    L = tg.lib()
    for M, m, n in ((1, 1, 16), (64, 4096, 14336), (4096, 28672, 8192), (1 << 20, 1 << 18, 131056), (1 << 16, 1 << 22, 16)):
        size = L.tg_int8_workspace_size(M, m, n)
        assert size >= 256 and size % 256 == 0
    for M, m, n in ((0, 1, 16), (1, 0, 16), (1, 1, 8), (1, 1, 131072), ((1 << 20) + 1, 1, 16), (1 << 20, 1 << 22, 16)):
        assert L.tg_int8_workspace_size(M, m, n) == 0


def test_binding_refuses_host_tensors_and_wrong_layouts():
    torch = pytest.importorskip("torch")
    f, i8, i32 = torch.float32, torch.int8, torch.int32
    with pytest.raises(ValueError):
        tg.moe_route(torch.zeros(2, 8), 2)                                    # host memory
    with pytest.raises(ValueError):
        tg.moe_route(torch.zeros(2, 8, dtype=torch.float64), 2)
    with pytest.raises(ValueError):
        tg.moe_route(torch.zeros(8, 2, dtype=f).t(), 2)                       # experts not neighbours
    with pytest.raises(ValueError):
        tg.moe_route(torch.zeros(2, 8), 2, bias=torch.zeros(7))
    with pytest.raises(ValueError):
        tg.moe_group(torch.zeros(4, dtype=torch.int64), 8)
    with pytest.raises(ValueError):
        tg.int8_quantize(torch.zeros(0, 8))
    with pytest.raises(ValueError):
        tg.int8_quantize(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        tg.Int8Layer(torch.zeros(4, 16, dtype=f), torch.zeros(4))
    with pytest.raises(ValueError):
        tg.Int8Layer(torch.zeros(4, 16, dtype=i8), torch.zeros(3))
    with pytest.raises(ValueError):
        tg.Int8Experts(torch.zeros(2, 4, 16, dtype=i8)[:, :, :8], torch.zeros(2, 4))

    class Fake:                                                               # a layer's fields without a device
        m, n, ldw, experts = 4, 16, 16, 2
        q, scales = torch.zeros(4, 16, dtype=i8), torch.zeros(4)
    with pytest.raises(ValueError):
        tg.int8_gemm(Fake, torch.zeros(2, 32, dtype=i8), torch.zeros(2))
    with pytest.raises(ValueError):
        tg.int8_gemm(Fake, torch.zeros(2, 16, dtype=i8), torch.zeros(3))
    with pytest.raises(ValueError):
        tg.int8_gemm(Fake, torch.zeros(2, 16, dtype=i8), torch.zeros(2))      # host memory
    with pytest.raises(ValueError):
        tg.int8_gemm_grouped(Fake, torch.zeros(2, 16, dtype=i8), torch.zeros(2), torch.zeros(3, dtype=i32), torch.zeros(3, dtype=i32))
    with pytest.raises(ValueError):
        tg.int8_gemm_grouped(Fake, torch.zeros(2, 16, dtype=i8), torch.zeros(2), torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32))

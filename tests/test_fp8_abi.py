"""Refusals of the norm and e4m3 entry points: every call here fails a host check, so nothing reaches a device."""
import pytest

from trellis_coded_gemv_amd import binding as tg

A16 = 0x10000          # fake device addresses: never dereferenced


def _norm(**kw):
    d = dict(rows=4, n=100, x=A16, dtype=1, ldx=100, residual=A16, rdtype=0, ldr=100, total=A16, ldt=100, weight=A16, wdtype=2,
             eps=1e-6, y=A16, out=4, ldy=100, scales=A16, lds=1, stream=None)
    d.update(kw)
    return tg.lib().rms_norm(*d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), -2), (dict(rows=(1 << 24) + 1), -2), (dict(n=0), -2), (dict(n=32769, ldx=40000, ldr=40000, ldt=40000, ldy=40000, lds=400), -2),
    (dict(dtype=3), -8), (dict(dtype=-1), -8), (dict(rdtype=3), -8), (dict(wdtype=4), -8), (dict(out=5), -8), (dict(out=-1), -8),
    (dict(ldx=99), -8), (dict(ldr=99), -8), (dict(ldt=99), -8), (dict(ldy=99), -8), (dict(lds=0), -8), (dict(lds=0, out=3), -8),
    (dict(n=129, ldx=129, ldr=129, ldt=129, ldy=129, lds=1), -8), (dict(eps=-1.0), -8), (dict(eps=float("nan")), -8), (dict(eps=float("inf")), -8),
    (dict(x=0), -1), (dict(total=0), -1), (dict(weight=0), -1), (dict(y=0), -1), (dict(scales=0), -1), (dict(scales=0, out=3), -1),
    (dict(x=A16 + 1), -4), (dict(residual=A16 + 2), -4), (dict(total=A16 + 2), -4), (dict(weight=A16 + 1), -4),
    (dict(y=A16 + 1, out=1), -4), (dict(y=A16 + 2, out=0), -4), (dict(scales=A16 + 2), -4)])
def test_norm_refusals(kw, status):
    assert _norm(**kw) == status


def _quantize(**kw):
    d = dict(rows=4, n=200, x=A16, dtype=1, ldx=200, block_rows=1, q=A16 + 1, ldq=200, scales=A16, lds=2, stream=None)
    d.update(kw)
    return tg.lib().fp8_quantize(*d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), -2), (dict(rows=(1 << 24) + 1), -2), (dict(n=0), -2), (dict(n=(1 << 22) + 1), -2),
    (dict(rows=1 << 17, n=1 << 22, ldx=1 << 22, ldq=1 << 22, lds=1 << 15), -2), (dict(dtype=3), -8), (dict(block_rows=0), -8),
    (dict(block_rows=64), -8), (dict(ldx=199), -8), (dict(ldq=199), -8), (dict(lds=1), -8), (dict(x=0), -1), (dict(q=0), -1),
    (dict(scales=0), -1), (dict(x=A16 + 1), -4), (dict(x=A16 + 2, dtype=0), -4), (dict(scales=A16 + 2), -4)])
def test_quantize_refusals(kw, status):
    assert _quantize(**kw) == status


def _gemm(**kw):
    d = dict(M=4, m=100, n=144, xq=A16, ldx=144, xs=A16, ldxs=2, wq=A16, ldw=144, wscales=A16, Y=A16, out=0, ldy=100, ws=A16,
             ws_bytes=1 << 40, stream=None)
    d.update(kw)
    return tg.lib().fp8_gemm(*d.values())


def _grouped(**kw):
    d = dict(pairs=8, experts=4, m=100, n=144, xq=A16, ldx=144, xs=A16, ldxs=2, ppr=2, wq=A16, wscales=A16, offsets=A16, order=A16,
             Y=A16, out=0, ldy=100, stream=None)
    d.update(kw)
    return tg.lib().fp8_gemm_grouped(*d.values())


SHARED = [(dict(m=0), -2), (dict(m=(1 << 22) + 1, ldy=1 << 23), -2), (dict(n=0), -2), (dict(n=136), -2),
          (dict(n=131072, ldx=131072), -2), (dict(ldx=128), -8), (dict(ldx=152), -8), (dict(ldxs=1), -8), (dict(ldy=99), -8), (dict(out=3), -8),
          (dict(xq=0), -1), (dict(xs=0), -1), (dict(wq=0), -1), (dict(wscales=0), -1), (dict(Y=0), -1),
          (dict(xq=A16 + 8), -4), (dict(wq=A16 + 8), -4), (dict(xs=A16 + 2), -4), (dict(wscales=A16 + 2), -4),
          (dict(Y=A16 + 2), -4), (dict(Y=A16 + 1, out=2), -4)]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(M=0), -2), (dict(M=(1 << 20) + 1), -2), (dict(ldw=128), -8), (dict(ldw=152), -8), (dict(ldw=(1 << 23) + 16), -8), (dict(ws=0), -5),
    (dict(ws_bytes=255), -5), (dict(ws=A16 + 16), -4), (dict(out=tg.TG_ZERO_UNROUTED), -8)])
def test_gemm_refusals(kw, status):
    assert _gemm(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(pairs=0), -2), (dict(pairs=(1 << 20) + 2), -2), (dict(experts=0), -2), (dict(experts=1025), -2), (dict(ppr=0), -8),
    (dict(ppr=3), -8), (dict(offsets=0), -1), (dict(order=0), -1), (dict(offsets=A16 + 2), -4), (dict(order=A16 + 1), -4),
    (dict(out=tg.TG_ZERO_UNROUTED | 3), -8), (dict(out=0x200), -8), (dict(out=-1), -8)])
def test_grouped_refusals(kw, status):
    assert _grouped(**kw) == status


def test_workspace_sizes():
    L = tg.lib()
    for M, m, n in ((1, 1, 16), (64, 4096, 14336), (4096, 28672, 8192), (1 << 20, 1 << 18, 131056), (1 << 16, 1 << 22, 16)):
        size = L.tg_fp8_workspace_size(M, m, n)
        assert size >= 256 and size % 256 == 0
    for M, m, n in ((0, 1, 16), (1, 0, 16), (1, 1, 8), (1, 1, 131072), ((1 << 20) + 1, 1, 16), (1 << 20, 1 << 22, 16)):
        assert L.tg_fp8_workspace_size(M, m, n) == 0


def test_binding_refuses_host_tensors_and_wrong_layouts():
    torch = pytest.importorskip("torch")
    f, i32, e = torch.float32, torch.int32, torch.float8_e4m3fn
    z = lambda *shape, dtype=f: torch.zeros(*shape, dtype=dtype)

    class Fake:                                                               # a layer's fields without a device
        m, n, ldw, experts = 4, 144, 144, 2
        q, scales = z(4, 144, dtype=e), z(1, 2)
    xq, xs = z(2, 144, dtype=e), z(2, 2)
    calls = [
        lambda: tg.rms_norm(z(2, 8), z(8)),                                   # host memory
        lambda: tg.rms_norm(z(2, 8, dtype=torch.float64), z(8)),
        lambda: tg.rms_norm(z(2, 8), z(7)), lambda: tg.rms_norm(z(2, 8), z(16)[::2]), lambda: tg.rms_norm(z(2, 8), z(8, dtype=i32)),
        lambda: tg.rms_norm(z(0, 8), z(8)), lambda: tg.rms_norm(z(2, 8), z(8), out_dtype=torch.uint8),
        lambda: tg.rms_norm(z(2, 8), z(8), residual=z(2, 7)), lambda: tg.rms_norm(z(2, 8), z(8), residual=z(2, 8, dtype=i32)),
        lambda: tg.rms_norm(z(2, 8), z(8), total=z(2, 8)),
        lambda: tg.fp8_quantize(z(0, 8)), lambda: tg.fp8_quantize(z(2, 8)), lambda: tg.fp8_quantize(z(2, 8, dtype=torch.int32)),
        lambda: tg.fp8_quantize(z(2, 8), block_rows=64), lambda: tg.fp8_quantize(z(2, 2, 8), block_rows=128),
        lambda: tg.Fp8Layer(z(4, 144), z(1, 2)), lambda: tg.Fp8Layer(z(4, 144, dtype=e), z(4, 2)), lambda: tg.Fp8Layer(z(4, 144, dtype=e), z(1, 1)),
        lambda: tg.Fp8Layer(z(4, 144, dtype=e), z(1, 4)[:, ::2]),
        lambda: tg.Fp8Experts(z(2, 4, 288, dtype=e)[:, :, :144], z(2, 1, 2)), lambda: tg.Fp8Experts(z(2, 4, 144, dtype=e), z(2, 4, 2)),
        lambda: tg.Fp8Experts.from_dense(z(4, 144)),
        lambda: tg.fp8_gemm(Fake, xq.float(), xs), lambda: tg.fp8_gemm(Fake, z(2, 160, dtype=e), xs), lambda: tg.fp8_gemm(Fake, xq, z(2)),
        lambda: tg.fp8_gemm(Fake, xq, z(3, 2)), lambda: tg.fp8_gemm(Fake, xq, z(2, 2).t().double()), lambda: tg.fp8_gemm(Fake, xq, xs),
        lambda: tg.fp8_gemm(Fake, xq, z(2, 4)[:, ::2]),
        lambda: tg.fp8_gemm_grouped(Fake, xq, xs, z(3, dtype=i32), z(3, dtype=i32)),
        lambda: tg.fp8_gemm_grouped(Fake, xq, xs, z(2, dtype=i32), z(2, dtype=i32)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(str(i))


def test_sizes_beyond_32_bits():
    """The C entry points take sizes of 32 bits: larger ones are refused, not cut to their low half."""
    torch = pytest.importorskip("torch")
    e = torch.float8_e4m3fn
    meta = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="meta")
    big = 1 << 32

    class Layer:
        m, n, ldw, experts, device = 4, 16, 16, 2, "cpu"
        q, scales = meta(4, 16, dtype=e), meta(1, 1)

    class Wide(Layer):
        m = big + 4
    calls = [
        lambda: tg.rms_norm(meta(big + 1, 4), meta(4)), lambda: tg.rms_norm(meta(1, big + 4), meta(big + 4)),
        lambda: tg.fp8_quantize(meta(big + 1, 1)), lambda: tg.fp8_quantize(meta(1, big + 64)), lambda: tg.fp8_quantize(meta(1 << 16, 1 << 16, 3)),
        lambda: tg.fp8_gemm(Layer, meta(big + 2, 16, dtype=e), meta(big + 2, 1)), lambda: tg.fp8_gemm(Wide, meta(2, 16, dtype=e), meta(2, 1)),
        lambda: tg.fp8_workspace(Layer, big + 1), lambda: tg.fp8_workspace(Wide, 1),
        lambda: tg.fp8_gemm_grouped(Wide, meta(2, 16, dtype=e), meta(2, 1), meta(3, dtype=torch.int32), meta(2, dtype=torch.int32)),
        lambda: tg.fp8_gemm_grouped(Layer, meta(1 << 31, 16, dtype=e), meta(1 << 31, 1), meta(3, dtype=torch.int32), meta(big, dtype=torch.int32), 2),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(tg.TgError):
            call()
            pytest.fail(str(i))

"""More refusals of the routing and 8-bit entry points: every call here fails a host check, so nothing reaches a device."""
import pytest

from test_int8_route_abi import _gemm, _grouped
from trellis_coded_gemv_amd import binding as tg


@pytest.mark.parametrize("out", [tg.TG_ZERO_UNROUTED | 3, 0x200, tg.TG_ZERO_UNROUTED << 1 | 1, -1, tg.TG_ZERO_UNROUTED - 1])
def test_grouped_output_types(out):
    assert _grouped(out=out) == -8


def test_the_dense_product_has_no_unrouted_rows():
    assert _gemm(out=tg.TG_ZERO_UNROUTED) == -8
    assert _grouped(out=tg.TG_ZERO_UNROUTED, order=0) == -1          # past the check of the type


def test_sizes_beyond_32_bits():
    """The C entry points take sizes of 32 bits: larger ones are refused, not cut to their low half. Tensors without memory stand for
    the calls' own, whose shapes are looked at first."""
    torch = pytest.importorskip("torch")
    meta = lambda shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="meta")
    big = 1 << 32

    class Layer:
        m, n, ldw, experts, device = 4, 16, 16, 2, "cpu"
        q, scales = meta((4, 16), torch.int8), meta(4)

    class Wide(Layer):
        m = big + 4
    calls = [
        lambda: tg.moe_route(meta((big + 1, 4)), 2), lambda: tg.moe_route(meta((2, big + 4)), 2), lambda: tg.moe_route(meta((2, 4)), big + 2),
        lambda: tg.moe_route(meta((2, 4)), 2, n_group=big + 1), lambda: tg.moe_route(meta((2, 4)), 2, n_group=2, topk_group=big + 1),
        lambda: tg.moe_route(meta((2, 4)), 2, group_top=1 - big), lambda: tg.moe_route(meta((2, 4)), -1),
        lambda: tg.moe_group(meta(big + 5, torch.int32), 8), lambda: tg.moe_group(meta(4, torch.int32), big + 8),
        lambda: tg.moe_group(meta(4, torch.int32), -1),
        lambda: tg.int8_quantize(meta((big + 1, 1))), lambda: tg.int8_quantize(meta((1, big + 64))), lambda: tg.int8_quantize(meta((1 << 16, 1 << 16, 3))),
        lambda: tg.int8_gemm(Layer, meta((big + 2, 16), torch.int8), meta(big + 2)), lambda: tg.int8_gemm(Wide, meta((2, 16), torch.int8), meta(2)),
        lambda: tg.int8_workspace(Layer, big + 1), lambda: tg.int8_workspace(Wide, 1),
        lambda: tg.int8_gemm_grouped(Wide, meta((2, 16), torch.int8), meta(2), meta(3, torch.int32), meta(2, torch.int32)),
        lambda: tg.int8_gemm_grouped(Layer, meta((1 << 31, 16), torch.int8), meta(1 << 31), meta(3, torch.int32), meta(big, torch.int32), 2),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(tg.TgError):
            call()
            pytest.fail(str(i))


def test_stream_of_another_device():
    """A stream of another GPU than the tensors' is refused; it is not replaced by the tensors' own current stream."""
    torch = pytest.importorskip("torch")

    class Stream:
        cuda_stream = 0x5000

        def __init__(self, index):
            self.device = torch.device("cuda", index)
    with pytest.raises(ValueError, match="stream"):
        tg._Entered(0, Stream(1))
    tg._Entered(1, Stream(1))
    tg._Entered(0, None)


A = 0x100000            # a device address: never dereferenced


@pytest.mark.parametrize("sel,offsets,order", [(A, A + 0x10000, A), (A, A + 0x10000, A + 396), (A + 396, A + 0x10000, A), (A, A, A + 0x10000),
                                               (A, A + 396, A + 0x10000), (A + 32, A, A + 0x10000), (A + 0x10000, A, A), (A + 0x10000, A + 396, A),
                                               (A + 0x10000, A, A + 32)])
def test_group_in_place(sel, offsets, order):
    """The ids are read by every workgroup, twice where they are many, while others write: a place found from ids that have changed
    meanwhile can lie behind the list. 100 pairs of 8 experts: 400 bytes of ids and of order, 36 of offsets."""
    assert tg.lib().moe_group(100, 8, sel, offsets, order, None) == -8

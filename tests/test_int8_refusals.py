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

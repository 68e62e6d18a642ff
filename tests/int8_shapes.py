"""The kernel that a product of the 8-bit entry points takes."""
import ctypes

from trellis_coded_gemv_amd import binding as tg


def plan(M, m, n, experts=0):
    """(shape, parts, outputs of a tile, rows of a tile), as the library takes them."""
    out = (ctypes.c_int32 * 4)()
    assert tg.lib().tg_int8_plan(M, m, n, experts, out) == 0, (M, m, n, experts)
    return tuple(out)

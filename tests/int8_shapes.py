"""Products that between them take every kernel of the 8-bit entry points, for the tests that run them and the one that holds the
list against the library's own rule."""
import ctypes

from trellis_coded_gemv_amd import binding as tg

# M, m, n: each tile shape whole, and in every number of parts that the rule cuts its inner axis into; odd ends on all axes
DENSE = [
    (201, 33879, 528), (129, 29423, 10592), (1754, 2381, 7616), (140, 13519, 16576), (4114, 395, 21040), (5581, 139, 24944),   # shape 0
    (600, 8001, 4112), (1024, 8191, 8192), (700, 28675, 1040), (5464, 763, 2512), (4961, 397, 9584),                           # 1
    (129, 18481, 32), (515, 4099, 2064),                                                                                       # 2
    (6601, 279, 32), (5835, 130, 10192), (4135, 215, 6176), (2893, 133, 7952), (4281, 66, 13920), (2735, 67, 16528),           # 3
    (5817, 129, 32), (2985, 139, 8432), (4156, 65, 4704), (2957, 70, 11744), (2201, 69, 13968), (1470, 67, 19504),             # 4
    (4358, 33, 32), (3067, 35, 2816), (2223, 34, 2304), (808, 65, 14816), (1068, 34, 9360), (710, 35, 11248),                  # 5
    (2, 32, 32), (726, 34, 6208), (523, 33, 4352), (388, 35, 3952), (1, 35, 3104), (1, 33, 4160)]                              # 6

# pairs, m, n, experts, top_k: each tile shape that the rule takes for experts
GROUPED = [
    (6320, 1089, 528, 37, 4), (16384, 1025, 768, 64, 8), (2048, 2050, 4096, 16, 4), (7144, 519, 2592, 14, 2), (3000, 6001, 528, 3, 3),
    (4096, 1535, 768, 16, 4), (6608, 291, 1040, 5, 2), (7720, 70, 528, 34, 5), (4960, 405, 272, 51, 8), (4140, 33, 2064, 3, 2),
    (600, 1001, 1040, 40, 6), (8, 2050, 2064, 128, 8), (66, 35, 272, 2, 1)]


def plan(M, m, n, experts=0):
    """(shape, parts, outputs of a tile, rows of a tile), as the library takes them."""
    out = (ctypes.c_int32 * 4)()
    assert tg.lib().tg_int8_plan(M, m, n, experts, out) == 0, (M, m, n, experts)
    return tuple(out)

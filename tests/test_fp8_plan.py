"""The library's rule for e4m3 products: what it refuses, that a workspace holds its parts, and that the GPU tests run every kernel."""
import collections
import ctypes
import math
import random

from fp8_shapes import DENSE16, DENSE32, GROUPED16, GROUPED32, plan
from trellis_coded_gemv_amd import binding as tg

SIZES = [(256, 256), (256, 128), (128, 128), (128, 64), (64, 64), (64, 32), (64, 16), (32, 16)]


def _sweep(count, seed):
    rng = random.Random(seed)
    size = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    for _ in range(count):
        yield size(1, 8192), size(32, 40000), max(1, size(32, 40000) // 16) * 16, rng.choice([0, 0, size(2, 300)])


def test_plan_refusals():
    out = (ctypes.c_int32 * 4)()
    for args, status in (((0, 1, 16, 0, 0), -2), ((1, 1, 24, 0, 0), -2), ((1, 1, 16, -1, 0), -2), ((1, 1, 16, 1025, 0), -2), ((1, 1, 16, 0, 3), -8),
                         ((1, 1, 16, 0, -1), -8)):
        assert tg.lib().tg_fp8_plan(*args, out) == status
    assert tg.lib().tg_fp8_plan(1, 1, 16, 0, 0, None) == -1


def test_plans_are_what_the_kernels_take():
    for M, m, n, experts in _sweep(3000, 1):
        for out in (0, 1, 2):
            shape, parts, outputs, rows = plan(M, m, n, experts, out)
            assert (outputs, rows) == SIZES[shape]
            assert shape > 0 or out != 0                             # 32-bit outputs have no tile of 256 x 256
            assert 1 <= parts <= 8 and (parts == 1 or not experts)   # the experts' launch has no workspace
            assert parts * 512 <= n or parts == 1                    # every part has a step of every shape, 512 bytes at most
        assert plan(M, m, n, experts, 1) == plan(M, m, n, experts, 2)


def test_workspace_holds_the_parts():
    for M, m, n, _ in _sweep(3000, 2):
        for out in (0, 2):
            _, parts, outputs, rows = plan(M, m, n, 0, out)
            tiles = -(-m // outputs) * -(-M // rows)
            assert tg.lib().tg_fp8_workspace_size(M, m, n) >= 256 + 4096 + (0 if parts == 1 else tiles * parts * outputs * rows * 4)
            assert parts == 1 or tiles <= 1024                       # a counter for each tile


def test_the_lists_take_every_kernel():
    """What the rule takes in one of 5000 products or more, the GPU tests run."""
    for out, dense, grouped, shapes in ((2, DENSE16, GROUPED16, set(range(8))), (0, DENSE32, GROUPED32, set(range(1, 8)))):
        taken = collections.Counter(("experts" if c[3] else "dense",) + plan(*c, out)[:2] for c in _sweep(40000, 3))
        often = {k for k, v in taken.items() if v >= 8}
        run = {("dense",) + plan(*c, 0, out)[:2] for c in dense} | {("experts",) + plan(*c[:4], out)[:2] for c in grouped}
        assert often <= run, sorted(often - run)
        assert {k[1] for k in run if k[0] == "dense"} == {k[1] for k in run if k[0] == "experts"} == shapes

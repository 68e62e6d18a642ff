"""The library's own rule and tile numbering: the rule against its model in Python, the numbering compiled for the host, and the
products that the GPU tests run against what the rule takes."""
import collections
import ctypes
import math
import os
import random
import shutil
import subprocess

import pytest

from int8_shapes import DENSE, GROUPED, plan
from test_int8_plan_model import plan as model
from test_int8_plan_model import shapes
from trellis_coded_gemv_amd import binding as tg
from trellis_coded_gemv_amd.build import CSRC


def _sweep(count, seed):
    rng = random.Random(seed)
    size = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    for _ in range(count):
        yield size(1, 8192), size(32, 40000), max(1, size(32, 40000) // 16) * 16, rng.choice([0, 0, size(2, 300)])


def test_rule_is_the_model():
    """Equal estimates of two plans may differ in the last place between the compilers: none of this sweep's do."""
    rows = shapes()[0]
    for case in _sweep(1500, 1):
        shape, parts, outputs, tile_rows = plan(*case)
        assert (shape, parts) == model(*case), case
        assert (outputs, tile_rows) == rows[shape][:2]


def test_plan_refusals():
    out = (ctypes.c_int32 * 4)()
    for args, status in (((0, 1, 16, 0), -2), ((1, 1, 24, 0), -2), ((1, 1, 16, -1), -2), ((1, 1, 16, 1025), -2)):
        assert tg.lib().tg_int8_plan(*args, out) == status
    assert tg.lib().tg_int8_plan(1, 1, 16, 0, None) == -1


def test_workspace_holds_the_parts():
    for M, m, n, experts in _sweep(1500, 2):
        _, parts, outputs, rows = plan(M, m, n)
        need = 0 if parts == 1 else -(-m // outputs) * -(-M // rows) * parts * outputs * rows * 4
        assert tg.lib().tg_int8_workspace_size(M, m, n) >= 256 + 4096 + need
        if parts > 1:
            assert -(-m // outputs) * -(-M // rows) <= 1024          # a counter for each tile


def test_the_lists_take_every_kernel():
    """What the rule takes in one of 5000 products or more, the GPU tests run: tile shapes and parts of dense products, shapes of experts'."""
    taken = collections.Counter(("experts" if c[3] else "dense",) + plan(*c)[:2] for c in _sweep(40000, 3))
    often = {k for k, v in taken.items() if v >= 8}
    run = {("dense",) + plan(*c)[:2] for c in DENSE} | {("experts",) + plan(*c[:4])[:2] for c in GROUPED}
    assert often <= run, sorted(often - run)
    assert {k[1] for k in run if k[0] == "dense"} == {k[1] for k in run if k[0] == "experts"} == set(range(len(shapes()[0])))


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("tiles")
    (d / "tiles.cpp").write_text('''#include "int8_tiles.hpp"
extern "C" {
int number(int b, int all) { return tg::tile_number(b, all); }
void place(int id, int out_tiles, int row_tiles, int splits, int dense, int* p) {
  const tg::TilePlace t = tg::tile_place(id, out_tiles, row_tiles, splits, dense != 0);
  p[0] = t.ot; p[1] = t.rt; p[2] = t.sp;
}
int zeros(int b, int all) { return tg::zeros_number(b, all); }
int first_output(int tiles, int t, int g) { return tg::lane_output(tiles, t, g); }
int row_output(int tiles, int q) { return tg::lds_row_output(tiles, q); }
int grid_width() { return tg::kGridWidth; }
int grid_shift() { return tg::kGridShift; }
}
''')
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "tiles.cpp", "-o", "tiles.so"], cwd=d, check=True)
    return ctypes.CDLL(os.path.join(d, "tiles.so"))


@pytest.mark.parametrize("all_tiles,launched", [(1, 1), (7, 7), (8, 8), (1000, 1000), (1000, 1009), (0, 16), (12345, 12345)])
def test_every_number_is_taken_once(tiles, all_tiles, launched):
    got = [tiles.number(b, all_tiles) for b in range(launched)]
    assert sorted(g for g in got if g >= 0) == list(range(all_tiles))
    for x in range(8):                                               # an XCD's workgroups take neighbouring tiles
        mine = [g for g in got[x::8] if g >= 0]
        assert mine == list(range(mine[0], mine[0] + len(mine))) if mine else True


def test_numbers_over_two_dimensions(tiles):
    """Workgroup (x, y) is number y * width + x, whatever is launched over; the width keeps neighbours on their XCDs."""
    width = tiles.grid_width()
    assert width == 1 << tiles.grid_shift() and width % 8 == 0 and width * 512 < 1 << 32
    all_tiles = 2 * width + 12
    seen = bytearray(all_tiles)
    for y in range(3):
        for b in range(y * width, y * width + (width if y < 2 else 16)):
            i = tiles.number(b, all_tiles)
            if i >= 0:
                seen[i] += 1
    assert seen.count(1) == all_tiles


@pytest.mark.parametrize("out_tiles,row_tiles,splits", [(1, 1, 1), (112, 16, 1), (3, 19, 1), (7, 5, 3), (64, 1, 8), (1, 33, 2), (5, 8, 6)])
@pytest.mark.parametrize("dense", [0, 1])
def test_every_place_is_taken_once(tiles, out_tiles, row_tiles, splits, dense):
    p = (ctypes.c_int * 3)()
    got = []
    for i in range(out_tiles * row_tiles * splits):
        tiles.place(i, out_tiles, row_tiles, splits, dense, p)
        got.append(tuple(p))
    want = {(o, r, s) for o in range(out_tiles) for r in range(row_tiles) for s in range(splits)}
    assert len(got) == len(want) and set(got) == want
    for i in range(0, len(got), splits):                             # a tile's parts are neighbours
        assert {g[:2] for g in got[i:i + splits]} == {got[i][:2]}


def test_tiles_of_experts_and_of_zeros(tiles):
    """However the pairs fall, the launch (row tiles that they could need, and 8 workgroups) holds every expert's tiles once and those of
    the pairs without one once."""
    rng = random.Random(4)
    for _ in range(600):
        pairs, experts, rows, out_tiles = rng.randint(1, 400), rng.randint(1, 30), rng.choice([16, 32, 64, 128, 256]), rng.randint(1, 9)
        lists = [0] * (experts + 1)
        for _ in range(pairs):
            lists[rng.randint(0, experts) if rng.random() < 0.5 else rng.choice([0, experts])] += 1
        bound = pairs // rows + min(experts + 1, pairs)
        routed = out_tiles * sum(-(-c // rows) for c in lists[:experts])
        zeros = out_tiles * -(-lists[experts] // rows)
        products, cleared = [], []
        for b in range(out_tiles * bound + 8):
            if tiles.number(b, routed) >= 0:
                products.append(tiles.number(b, routed))
            elif 0 <= tiles.zeros(b, routed) < zeros:
                cleared.append(tiles.zeros(b, routed))
        assert sorted(products) == list(range(routed)) and sorted(cleared) == list(range(zeros))


@pytest.mark.parametrize("case", range(7))
def test_lds_rows_are_the_outputs(tiles, case):
    at, _, wo = shapes()[1][case][:3]
    outs = [tiles.row_output(at, q) for q in range(16 * at * wo)]
    assert sorted(outs) == list(range(16 * at * wo))
    for w in range(wo):                                              # where a lane stores is what its rows of LDS held
        for t in range(at):
            for g in range(4):
                first = 16 * at * w + tiles.first_output(at, t, g)
                assert [outs[16 * (at * w + t) + 4 * g + v] for v in range(4)] == list(range(first, first + 4))
            if t % 2 == 0 and at > 1:                                # two tiles: eight neighbours of a lane, 32 of a row's four
                assert all(tiles.first_output(at, t + 1, g) == tiles.first_output(at, t, g) + 4 for g in range(4))
                assert [tiles.first_output(at, t, g) - tiles.first_output(at, t, 0) for g in range(4)] == [0, 8, 16, 24]

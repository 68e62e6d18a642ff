"""Host-side models of the 8-bit products: which tile shape and split a product takes (the table read from the kernel's
source), that every tile of a launch is found exactly once, and that a tile's LDS rows cover its outputs."""
import os
import re

import numpy as np
import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "trellis_coded_gemv_amd", "csrc", "int8_gemm.hip")


def _source():
    with open(SRC) as f:
        return f.read()


def shapes():
    """[(out, rows, resident, alone, shared, tile)] of kTiles, and the template arguments of the launch's cases."""
    text = _source()
    table = text[text.index("constexpr TileCost kTiles[]"):]
    rows = re.findall(r"\{(\d+), (\d+), (\d+), ([\d.]+)f, ([\d.]+)f, ([\d.]+)f\}", table[:table.index("};")])
    cases = re.findall(r"case (\d+): return launch_shape<TileShape<([\d, ]+)>>", text)
    return [tuple(map(float, r)) for r in rows], [tuple(map(int, c[1].split(","))) for c in sorted(cases, key=lambda c: int(c[0]))]


def plan(M, m, n, experts=0):
    """(shape, splits), in binary32 as the library forms it."""
    f = np.float32
    reached = f(min(experts, M)) if experts else f(1)
    rows = f(M) / reached
    stream = (reached * f(m) * f(n) + f(M) * f(n) + f(2) * f(M) * f(m)) / f(5.3e6)
    steps, best, least = (n + 127) // 128, (0, 1), f(3.0e38)
    for i, (out, tx, resident, alone, shared, tile) in enumerate(shapes()[0]):
        if tx > 32 and f(tx) > f(2) * rows:
            continue
        rt = reached * max(f(1), rows / f(tx) + f(0.5)) if experts else f(-(-M // int(tx)))
        tiles = rt * f(-(-m // int(out)))
        for splits in (1, 2, 3, 4, 6, 8):
            if splits > 1 and (experts or tiles > 512 or splits * 512 > n):
                break
            groups, slots = tiles * f(splits), 256 * int(resident)
            rounds = f(int(groups / f(slots)))
            rest = groups - rounds * f(slots)
            length = f((steps + splits - 1) // splits)
            work = rounds * (f(shared) * length + f(tile))
            if rest > 0:
                work += (f(shared) if rest > 256 else f(alone)) * length + f(tile)
            us = max(work, stream) + f(0.2) * min(work, stream)
            if splits > 1:
                us += f(0.9) + f(2.1e-6) * f(splits) * f(M) * f(m)
            if us < least:
                least, best = us, (i, splits)
    return best


def test_table_matches_the_kernels():
    """Each row of the table is the tile of the kernel that its case launches; LDS and load counts fit."""
    rows, cases = shapes()
    assert len(rows) == len(cases) == 7
    for (out, tx, resident, *_), c in zip(rows, cases):
        at, rx, wo, wx, bk, st = c[:6]
        ew, occ = (c + (0, 2)[len(c) - 6:])[6:8] if len(c) < 8 else c[6:8]
        assert (16 * at * wo, 16 * rx * wx) == (out, tx)
        lds = (st + ew) * out * bk + st * tx * bk
        assert lds * resident <= 160 * 1024
        nw, rpi = wo * wx, 1024 // bk
        assert out % (rpi * nw) == 0 and tx % (rpi * nw) == 0
        assert st * bk % 64 == 0 and nw * resident * 1 <= 32


def test_every_shape_is_reached():
    seen = set()
    for M in (1, 8, 33, 64, 100, 200, 300, 700, 2048, 8192):
        for m, n in ((28672, 8192), (8192, 8192), (4096, 14336), (1024, 8192), (8192, 1024), (512, 512), (300, 20000), (9000, 272)):
            seen.add(plan(M, m, n)[0])
    assert seen == set(range(7))
    assert {plan(pairs, 1536, 2048, 128)[0] for pairs in (8, 512, 4096, 16384, 65536)} >= {0, 4, 5, 6}
    assert any(plan(M, 4096, 14336)[1] > 1 for M in (1, 61, 256))


def _find(b, out_tiles, row_tiles, splits, dense):
    """find_tile's numbering of workgroup b: (ot, rt, sp) or None."""
    total = out_tiles * row_tiles * splits
    per, rest, x, k = total >> 3, total & 7, b & 7, b >> 3
    if k >= per + (1 if x < rest else 0):
        return None
    i = x * per + min(x, rest) + k
    i, sp = divmod(i, splits)
    if not dense:
        return i % out_tiles, i // out_tiles, sp
    band, inside = divmod(i, 8 * out_tiles)
    high = min(8, row_tiles - band * 8)
    ot = inside // high
    return ot, band * 8 + inside - ot * high, sp


@pytest.mark.parametrize("out_tiles,row_tiles,splits", [(1, 1, 1), (112, 16, 1), (3, 19, 1), (7, 5, 3), (64, 1, 8), (1, 33, 2)])
def test_every_tile_is_found_once(out_tiles, row_tiles, splits):
    for dense in (True, False):
        for launched in (row_tiles, row_tiles + 9):          # an experts' launch may hold more than there are
            if dense and launched != row_tiles:
                continue
            found = [_find(b, out_tiles, row_tiles, splits, dense) for b in range(out_tiles * launched * splits)]
            found = [f for f in found if f is not None]
            want = {(o, r, s) for o in range(out_tiles) for r in range(row_tiles) for s in range(splits)}
            assert len(found) == len(want) and set(found) == want


@pytest.mark.parametrize("case", range(7))
def test_lds_rows_cover_the_outputs(case):
    at, _, wo = shapes()[1][case][:3]
    output = lambda t, g: 4 * g if at == 1 else 32 * (t // 2) + 8 * g + 4 * (t % 2)
    outs = [q // (16 * at) * (16 * at) + output((q >> 4) % at, (q >> 2) & 3) + (q & 3) for q in range(16 * at * wo)]
    assert sorted(outs) == list(range(16 * at * wo))
    for w in range(wo):                                      # a lane (group g) of a wave stores eight neighbours at once
        for g in range(4):
            for t in range(0, at - 1, 2):
                mine = [outs[16 * (at * w + u) + 4 * g + v] for u in (t, t + 1) for v in range(4)]
                assert mine == list(range(mine[0], mine[0] + 8)) and mine[0] % 8 == 0

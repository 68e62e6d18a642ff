// Numbering of the 8-bit products' tiles, on the host and in the kernel.
#pragma once

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define TG_BOTH __host__ __device__ __forceinline__
#else
#define TG_BOTH inline
#endif

namespace tg {

// A launch's workgroups are numbered over two dimensions, kGridWidth to a row: one holds fewer than 2^32 threads.
constexpr int kGridShift = 20, kGridWidth = 1 << kGridShift;

struct TilePlace {
  int ot, rt, sp;             // output tile, row tile, part of the inner axis
};

// Workgroup b -> its tile's number out of `all`, or -1. Workgroups b, b + 8, ... share an XCD and its L2: each XCD takes a
// run of neighbouring tiles, the same number for each.
TG_BOTH int tile_number(int b, int all) {
  const int per = all >> 3, rest = all & 7, x = b & 7, k = b >> 3;
  if (k >= per + (x < rest ? 1 : 0)) return -1;
  return x * per + (x < rest ? x : rest) + k;
}

// Workgroup b -> its number among the tiles of rows to set to zero, which are numbered behind `all` others from a multiple
// of 8 on and so spread over the XCDs; negative: none. At most 7 workgroups lie between.
TG_BOTH int zeros_number(int b, int all) { return b - ((all + 7) & ~7); }

// Dense: bands of 8 row tiles, rows first, then outputs. Else row tile by row tile, outputs first.
TG_BOTH TilePlace tile_place(int id, int out_tiles, int row_tiles, int splits, bool dense) {
  TilePlace t{0, 0, 0};
  if (splits > 1) {
    const int q = id / splits;
    t.sp = id - q * splits;
    id = q;
  }
  if (dense) {
    const int band = id / (8 * out_tiles), in = id - band * 8 * out_tiles;
    const int left = row_tiles - band * 8, high = left < 8 ? left : 8;
    t.ot = in / high;
    t.rt = band * 8 + in - t.ot * high;
  } else {
    t.rt = id / out_tiles;
    t.ot = id - t.rt * out_tiles;
  }
  return t;
}

// First of the four neighbouring outputs that lane group g (of 4) of a wave ends with for its tile t of 16, counted from
// the wave's first output: with two tiles or more, 8 neighbours of a row for a lane and 32 for the four lanes of the row.
TG_BOTH int lane_output(int tiles, int t, int g) { return tiles == 1 ? 4 * g : 32 * (t / 2) + 8 * g + 4 * (t % 2); }

// The output that row q of the layer's side in LDS holds, waves of `tiles` tiles: row 16 t + 4 g + v of a wave's is its
// output lane_output(tiles, t, g) + v.
TG_BOTH int lds_row_output(int tiles, int q) {
  const int wave = q / (16 * tiles) * (16 * tiles);
  return wave + lane_output(tiles, (q >> 4) % tiles, (q >> 2) & 3) + (q & 3);
}

}  // namespace tg

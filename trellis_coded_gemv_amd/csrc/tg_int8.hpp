// What the 8-bit product kernels share: the rows of a tile, the output types and the stores.
#pragma once

#include "tg_device.hpp"
#include "tg_internal.hpp"

namespace tg {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// Which output rows (pairs) a workgroup's row tile covers. Dense: [first, first + count). Experts: the tiles of
// `rows_per_tile` pairs are numbered expert by expert, `first` is a place in order, and every wave finds its tile's
// expert from the offsets (a lane holds up to 16 neighbouring experts).
struct RowTile {
  int expert, first, count;   // count 0: nothing to do
};

__device__ __forceinline__ RowTile find_tile(const Int8Args& a, int tile, int rows_per_tile) {
  if (!a.offsets) {
    const int first = tile * rows_per_tile;
    return {0, first, min(rows_per_tile, a.M - first)};
  }
  const int lane = threadIdx.x & 63;
  const int per = (a.experts + 63) >> 6;
  const int e0 = lane * per;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int e = e0 + i;
    if (e < a.experts) {
      const int b = min(max(a.offsets[e], 0), a.M), c = min(max(a.offsets[e + 1], 0), a.M);
      mine += c > b ? (c - b + rows_per_tile - 1) / rows_per_tile : 0;
    }
  }
  int upto = mine;
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d, 64);
    if (lane >= d) upto += v;
  }
  RowTile t{0, 0, 0};
  const uint64_t has = __ballot(upto > tile);
  if (has == 0) return t;
  const int owner = __builtin_ctzll(has);
  int left = tile - __shfl(upto - mine, owner, 64);
  for (int i = 0; i < per; ++i) {
    const int e = owner * per + i;
    if (e >= a.experts) break;
    const int b = min(max(a.offsets[e], 0), a.M), c = min(max(a.offsets[e + 1], 0), a.M);
    const int nt = c > b ? (c - b + rows_per_tile - 1) / rows_per_tile : 0;
    if (left < nt) {
      t.expert = e;
      t.first = b + left * rows_per_tile;
      t.count = min(rows_per_tile, c - t.first);
      return t;
    }
    left -= nt;
  }
  return t;
}

// Output row (pair) of row i of a tile, or -1; its activation row is pair / pairs_per_row.
__device__ __forceinline__ int pair_of(const Int8Args& a, const RowTile& t, int i) {
  if (i >= t.count) return -1;
  if (!a.offsets) return t.first + i;
  const int p = a.order[t.first + i];
  return p >= 0 && p < a.M ? p : -1;
}

template <int DT>
__device__ __forceinline__ uint32_t half_bits(float v) {
  if constexpr (DT == kF16) return __builtin_bit_cast(uint16_t, (_Float16)v);
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Four neighbouring outputs of a row, of which `valid` exist. wide: they may be stored at once.
template <int DT>
__device__ __forceinline__ void store4(void* y, int64_t at, const float (&v)[4], int valid, bool wide) {
  if constexpr (DT == kF32) {
    float* p = reinterpret_cast<float*>(y) + at;
    if (valid >= 4 && wide) *reinterpret_cast<float4_t*>(p) = float4_t{v[0], v[1], v[2], v[3]};
    else
      for (int i = 0; i < 4; ++i)
        if (i < valid) p[i] = v[i];
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(y) + at;
    if (valid >= 4 && wide)
      *reinterpret_cast<u32x2*>(p) = u32x2{half_bits<DT>(v[0]) | half_bits<DT>(v[1]) << 16,
                                           half_bits<DT>(v[2]) | half_bits<DT>(v[3]) << 16};
    else
      for (int i = 0; i < 4; ++i)
        if (i < valid) p[i] = (uint16_t)half_bits<DT>(v[i]);
  }
}

// Row tiles of a launch: exact for a dense product; for the experts' an upper bound that holds for every way the
// pairs can fall (each expert with pairs leaves at most one tile part-filled).
inline int row_tiles(const Int8Args& a, int rows_per_tile) {
  const int full = (a.M + rows_per_tile - 1) / rows_per_tile;
  if (!a.offsets) return full;
  return a.M / rows_per_tile + (a.experts < a.M ? a.experts : a.M);
}

hipError_t launch_int8_tile(const Int8Args& a, int shape, hipStream_t s);

}  // namespace tg

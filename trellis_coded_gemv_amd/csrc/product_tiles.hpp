// What the products of 8-bit rows share on the device (int8_gemm.hip, fp8_gemm.hip): which tile a workgroup has, the loads to
// LDS, the shape of a tile, the stores of its outputs.
#pragma once

#include "int8_tiles.hpp"
#include "tg_device.hpp"
#include "tg_internal.hpp"

namespace tg {

// A workgroup's tile. rows: dense, output rows first .. first + count - 1; experts, places first .. of order.
struct Tile {
  int ot, rt, sp;             // output tile, row tile, part of the inner axis
  int expert, first, count;   // expert -1: rows to set to zero; count 0: nothing to do
};

// Workgroup -> tile. Dense: 8 row tiles by all output tiles, rows first, so that an XCD's resident workgroups share a few
// row tiles and output tiles. Experts: the row tiles are numbered expert by expert (every wave finds them from the
// offsets, up to 16 neighbouring experts to a lane), outputs first, so that an expert's tiles stay together; the launch
// holds the most tiles that the pairs could need, and what is over ends at once. Pairs without an expert, where their rows
// are to be set to zero, are numbered apart and behind them, one by one over the XCDs: in one run with the experts' they
// fill whole XCDs, which leave the products to the others (8192 tokens over 128 experts, half of the pairs without one: 168
// us with their rows left, 241 in one run, 193 apart).
// Every value is wave-uniform.
__device__ __forceinline__ Tile find_tile(const Product8Args& a, int out_tiles, int row_tiles, int rows_per_tile) {
  constexpr int kHeld = 4;                      // experts of a lane whose places are kept
  Tile t{0, 0, 0, 0, 0, 0};
  const int lane = threadIdx.x & 63;
  const int per_lane = (a.experts + 63) >> 6;
  int at[kHeld + 1], mine = 0, scan = 0;        // where a lane's experts begin, and the one behind them
  // Past the last expert: where it ends, so none of its own. Places are cut to [0, M].
  auto place = [&](int e) { return min(max(a.offsets[min(e, a.experts)], 0), a.M); };
  auto tiles = [&](int from, int to) { return to > from ? (to - from + rows_per_tile - 1) / rows_per_tile : 0; };
  if (a.offsets) {
    if (per_lane <= kHeld) {
#pragma unroll
      for (int i = 0; i <= kHeld; ++i) at[i] = place(lane * per_lane + min(i, per_lane));
#pragma unroll
      for (int i = 0; i < kHeld; ++i) mine += tiles(at[i], at[i + 1]);
    } else {
      for (int i = 0; i < per_lane; ++i) mine += tiles(place(lane * per_lane + i), place(lane * per_lane + i + 1));
    }
    scan = wave_scan(mine);
    row_tiles = min(row_tiles, __builtin_amdgcn_readlane(scan, 63));
  }
  const int b = (int)(blockIdx.y << kGridShift | blockIdx.x), all = out_tiles * row_tiles * a.splits;
  const int id = tile_number(b, all);
  if (id < 0) {
    const int behind = zeros_number(b, all);
    if (!a.zero_rest || behind < 0) return t;
    const int nth = behind / out_tiles;
    t.ot = behind - nth * out_tiles;
    t.expert = -1;
    t.first = __builtin_amdgcn_readfirstlane(place(a.experts)) + nth * rows_per_tile;
    t.count = min(rows_per_tile, a.M - t.first);
    return t;
  }
  const TilePlace at_tile = tile_place(id, out_tiles, row_tiles, a.splits, !a.offsets);
  t.ot = at_tile.ot;
  t.rt = at_tile.rt;
  t.sp = at_tile.sp;
  if (!a.offsets) {
    t.first = t.rt * rows_per_tile;
    t.count = min(rows_per_tile, a.M - t.first);
    return t;
  }
  const int owner = __builtin_ctzll(__ballot(scan > t.rt));     // some lane is, as rt < the last lane's sum
  int left = t.rt - __builtin_amdgcn_readlane(scan - mine, owner);
  for (int i = 0; i < per_lane; ++i) {
    int from, to;
    if (per_lane <= kHeld) {
      int b = at[0], c = at[1];
#pragma unroll
      for (int h = 1; h < kHeld; ++h) {
        b = i == h ? at[h] : b;
        c = i == h ? at[h + 1] : c;
      }
      from = __builtin_amdgcn_readlane(b, owner);
      to = __builtin_amdgcn_readlane(c, owner);
    } else {
      from = __builtin_amdgcn_readfirstlane(place(owner * per_lane + i));
      to = __builtin_amdgcn_readfirstlane(place(owner * per_lane + i + 1));
    }
    const int n = tiles(from, to);
    if (left < n) {
      t.expert = owner * per_lane + i;
      t.first = from + left * rows_per_tile;
      t.count = min(rows_per_tile, to - t.first);
      return t;
    }
    left -= n;
  }
  return t;
}

// Output row (pair) of row i of a tile, or -1; its activation row is pair / pairs_per_row.
__device__ __forceinline__ int pair_of(const Product8Args& a, const Tile& t, int i) {
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

// N (4 or 8) neighbouring outputs of a row, of which `valid` exist, 16 bytes at once wherever the row begins (7890 x 28349
// x 144, rows of an odd number of fp16 outputs: 223 us, 471 with a store for each).
template <int DT, int N>
__device__ __forceinline__ void store_outputs(void* y, int64_t at, const float (&v)[N], int valid) {
  if constexpr (DT == kF32) {
    float* p = reinterpret_cast<float*>(y) + at;
    if (valid >= N) {
#pragma unroll
      for (int i = 0; i < N; i += 4) *reinterpret_cast<float4_any*>(p + i) = float4_any{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < valid) p[i] = v[i];
    }
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(y) + at;
    uint32_t h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) h[i] = half_bits<DT>(v[2 * i]) | half_bits<DT>(v[2 * i + 1]) << 16;
    if (valid >= N) {
      if constexpr (N == 8) *reinterpret_cast<u32x4_any*>(p) = u32x4_any{h[0], h[1], h[2], h[3]};
      else *reinterpret_cast<u32x2_any*>(p) = u32x2_any{h[0], h[1]};
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < valid) p[i] = (uint16_t)(h[i / 2] >> (16 * (i & 1)));
    }
  }
}

namespace {

// Row tiles of a launch: exact for a dense product; for the experts' an upper bound that holds for every way the
// pairs can fall (each expert with pairs leaves at most one tile part-filled, and so do the pairs without one).
int row_tiles(const Product8Args& a, int rows_per_tile) {
  const int full = (a.M + rows_per_tile - 1) / rows_per_tile;
  if (!a.offsets) return full;
  const int lists = a.experts + (a.zero_rest ? 1 : 0);
  return a.M / rows_per_tile + (lists < a.M ? lists : a.M);
}

// 16 bytes of global memory per lane to LDS at base + 16 * lane (base wave-uniform): from a lane's own address, or from
// a lane's offset to a wave-uniform address. The load reads m0 one wait state after a scalar write of it at the earliest,
// which the compiler does not see to inside inline assembly (its builtin would, but waits for the loads at every LDS read).
__device__ __forceinline__ void load_to_lds(const int8_t* p, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_base), "v"(p) : "m0", "memory");
}
__device__ __forceinline__ void load_to_lds(const int8_t* p, uint32_t offset, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds_base), "v"(offset), "s"(p) : "m0", "memory");
}

// Wait until at most N of this wave's loads are in flight and its LDS reads are done.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// AT x RX: 16x16 tiles of one wave (outputs x rows); WO x WX: waves of a workgroup; BK: bytes of the inner axis per
// step; ST: steps held in LDS, of the layer's side EW more.
template <int AT_, int RX_, int WO_, int WX_, int BK_, int ST_, int EW_ = 0, int OCC_ = 2>
struct TileShape {
  static constexpr int AT = AT_, RX = RX_, WO = WO_, WX = WX_, BK = BK_, ST = ST_, EW = EW_, OCC = OCC_;
  static constexpr bool AHEAD = OCC <= 2;                            // registers for two sets of operands
  static constexpr int NW = WO * WX, TO = 16 * AT * WO, TX = 16 * RX * WX;
  static constexpr int RPI = 1024 / BK;                             // LDS rows filled by one load instruction
  static constexpr int LW = TO / RPI / NW, LX = TX / RPI / NW;      // load instructions of a wave per step
  static constexpr int WBUF = TO * BK, XBUF = TX * BK;              // LDS bytes of a step
  static constexpr int XLDS = (ST + EW) * WBUF;                     // where the activations' steps begin
  static_assert(AHEAD || EW == 0, "");
  static_assert(LW * RPI * NW == TO && LX * RPI * NW == TX, "every wave loads whole instructions");
  // A row's 16-byte pieces are held in LDS in an order that depends on the row, so that the lanes which read the same
  // piece of neighbouring rows spread over the banks.
  static __device__ __forceinline__ int output(int t, int g) { return lane_output(AT, t, g); }
  static __device__ __forceinline__ int swizzle(int row) { return BK >= 128 ? row & 7 : (row >> 1) & 3; }
};

}  // namespace

}  // namespace tg

// Products of 8-bit rows: Y[r, o] = (sum_i xq[r, i] wq[o, i]) * xs[r] * ws[o], for a dense layer and for the experts of
// routed pairs, by tiles of TO outputs x TX rows.
//
// The sums are exact in int32 (|q| <= 128 and n < 2^17, so none leaves the type), whatever the order and the split of the
// work; an output is rounded three times in binary32 (the sum, and its product with either scale) and once more to a
// 16-bit output type.
//
// What bounds it (MI355X, 2.2 GHz under this load): 4096 x 28672 x 8192 runs at 2430-2540 TOP/s (758-793 us), 60-63% of
// what the matrix cores reach on such values from registers alone (4035 TOP/s; 4900 on zeros: the card's power). The
// loads to LDS alone take 508 of 789 us with these 256 x 256 tiles, and 722 of 899 with 256 x 128 (373 and 456 where every
// tile reads the same rows, out of L2); the reads from LDS alone 323. So the way into LDS comes next to the power, and the
// largest tiles ask least of it. The library's own 8-bit product takes 844 us there. 1 x 28672 x 8192 reads 235 MB in 42
// us (5.6 TB/s; a large copy moves 5.1). 8192 tokens over 128 experts, 1536 x 2048, top 8: 269-279 us; the loads to LDS
// alone 190, the stores 35-43, the first loads and lookups of short tiles some 40; 2048 x 768 with a row for each pair:
// 207-212 us, of which 268 MB of outputs are half the bytes. Workgroups that go on to a next tile and begin its loads
// before the stores of the last lose (312 -> 320 us with 256 x 128 tiles: loads wait for the stores before them).
//
// v_mfma_i32_16x16x64_i8 with the layer's rows as its A operand and the activation rows as its B operand: lane l
// supplies row l % 16 and the 16 bytes at 16 (l / 16) of 64 bytes of the inner axis on both sides, and ends with four
// neighbouring outputs of row l % 16. Both sides reach LDS by loads that do not pass through registers, a ring of ST
// steps of BK bytes, and the operands are read from there.
#include <type_traits>

#include "int8_tiles.hpp"
#include "tg_device.hpp"
#include "tg_internal.hpp"

namespace tg {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

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
__device__ __forceinline__ Tile find_tile(const Int8Args& a, int out_tiles, int row_tiles, int rows_per_tile) {
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
__device__ __forceinline__ int pair_of(const Int8Args& a, const Tile& t, int i) {
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
int row_tiles(const Int8Args& a, int rows_per_tile) {
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

__device__ __forceinline__ void put_partial(uint64_t* p, i32x4 v) {
  const u32x4 u = __builtin_bit_cast(u32x4, v);
  __hip_atomic_store(p, (uint64_t)u[1] << 32 | u[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(p + 1, (uint64_t)u[3] << 32 | u[2], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ i32x4 get_partial(uint64_t* p) {
  const uint64_t a = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint64_t b = __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return i32x4{(int)(uint32_t)a, (int)(a >> 32), (int)(uint32_t)b, (int)(b >> 32)};
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

template <class S, int DT>
__global__ __launch_bounds__(64 * S::NW, S::OCC) void int8_tile_kernel(const Int8Args a, int out_tiles, int row_tiles) {
  constexpr int AT = S::AT, RX = S::RX, BK = S::BK, ST = S::ST, TO = S::TO, TX = S::TX, NW = S::NW;
  __shared__ __attribute__((aligned(1024))) int8_t sh[S::XLDS + ST * S::XBUF];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int j = lane & 15, g = lane >> 4;
  const Tile tile = find_tile(a, out_tiles, row_tiles, TX);
  if (tile.count <= 0) return;
  const int ot = tile.ot, rt = tile.rt, sp = tile.sp;
  const int o0 = ot * TO;
  if (tile.expert < 0) {                         // eight neighbouring outputs to a thread
    const float zeros[8] = {};
    for (int i = threadIdx.x; i < tile.count * (TO / 8); i += 64 * NW) {
      const int pair = pair_of(a, tile, i / (TO / 8)), o = o0 + i % (TO / 8) * 8;
      if (pair >= 0 && o < a.m) store_outputs<DT, 8>(a.y, (int64_t)pair * a.ldy + o, zeros, a.m - o);
    }
    return;
  }
  const int wo = wave % S::WO, wx = wave / S::WO;

  // Loads: an instruction fills RPI rows of LDS; lane l the slot l % (BK / 16) of row l / (BK / 16), where the piece
  // slot ^ swizzle(row) of the row belongs.
  const int lrow = lane / (BK / 16);
  auto wrow = [&](int i) { return S::RPI * (S::LW * wave + i) + lrow; };   // LDS row of this lane in instruction i
  auto xrow = [&](int i) { return S::RPI * (S::LX * wave + i) + lrow; };
  auto piece = [&](int row) { return 16 * ((lane % (BK / 16)) ^ S::swizzle(row)); };
  // The layer's rows are addressed by 32-bit offsets to the tile's first row (the launch keeps their stride below 2^23).
  const int8_t* wbase = a.w + ((int64_t)tile.expert * a.m + o0) * a.ldw;
  uint32_t woff[S::LW];
  const int8_t* xp[S::LX];
#pragma unroll
  for (int i = 0; i < S::LW; ++i) {
    const int q = wrow(i);
    const int o = lds_row_output(AT, q);
    woff[i] = (uint32_t)min(o, a.m - 1 - o0) * (uint32_t)a.ldw;
  }
#pragma unroll
  for (int i = 0; i < S::LX; ++i) {
    xp[i] = a.x + (int64_t)(max(pair_of(a, tile, xrow(i)), 0) / a.pairs_per_row) * a.ldx;
  }
  const uint32_t sh0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t*)sh;
  const uint32_t wfill = __builtin_amdgcn_readfirstlane(sh0 + wave * S::LW * 1024);
  const uint32_t xfill = __builtin_amdgcn_readfirstlane(sh0 + S::XLDS + wave * S::LX * 1024);
  auto load_w = [&](int step, uint32_t buf) {
    const int k = step * BK, most = a.n - 16 - k;    // pieces past the end: any bytes of the row, not multiplied
#pragma unroll
    for (int i = 0; i < S::LW; ++i) load_to_lds(wbase, woff[i] + (uint32_t)(k + min(piece(wrow(i)), most)), wfill + buf + i * 1024);
  };
  auto load_x = [&](int step, uint32_t buf) {
    const int k = step * BK, most = a.n - 16 - k;
#pragma unroll
    for (int i = 0; i < S::LX; ++i) load_to_lds(xp[i] + (k + min(piece(xrow(i)), most)), xfill + buf + i * 1024);
  };

  i32x4 acc[AT][RX];
#pragma unroll
  for (int t = 0; t < AT; ++t)
#pragma unroll
    for (int r = 0; r < RX; ++r) acc[t][r] = i32x4{0, 0, 0, 0};
  const int slot = 16 * (g ^ S::swizzle(j));     // of the step's first 64 bytes; the h-th 64: slot ^ 64 h
  const int abase = (wo * 16 * AT + j) * BK + slot, bbase = S::XLDS + (wx * 16 + j) * BK + slot;
  // The operands of 64 bytes of the inner axis: read from LDS while the matrix cores work on those before.
  struct Frags {
    i32x4 a[AT], b[RX];
  };
  uint32_t wbuf = 0, xbuf = 0;                   // of step s
  auto read = [&](Frags& f, int h, auto rows) {
#pragma unroll
    for (int r = 0; r < decltype(rows)::value; ++r)
      f.b[r] = *reinterpret_cast<const i32x4*>(sh + xbuf + ((bbase ^ (64 * h)) + r * S::WX * 16 * BK));
#pragma unroll
    for (int t = 0; t < AT; ++t) f.a[t] = *reinterpret_cast<const i32x4*>(sh + wbuf + ((abase ^ (64 * h)) + t * 16 * BK));
  };
  auto cut = [&](Frags& f, int h, int left) {    // pieces past the end of the inner axis count as zero
    if (64 * h + 16 * g >= left) {
#pragma unroll
      for (int r = 0; r < RX; ++r) f.b[r] = i32x4{0, 0, 0, 0};
    }
  };
  auto multiply = [&](const Frags& f, auto rows) {
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int r = 0; r < decltype(rows)::value; ++r) acc[t][r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.a[t], f.b[r], acc[t][r], 0, 0, 0);
  };
  const int steps_all = (a.n + BK - 1) / BK;
  const int begin = (int)((int64_t)steps_all * sp / a.splits), end = (int)((int64_t)steps_all * (sp + 1) / a.splits);
  constexpr int U = BK / 64, EW = S::EW;
  Frags f[2];
  int s = begin;
  auto advance = [&]() {
    wbuf = wbuf == (uint32_t)(ST + EW - 1) * S::WBUF ? 0u : wbuf + S::WBUF;
    xbuf = xbuf == (uint32_t)(ST - 1) * S::XBUF ? 0u : xbuf + S::XBUF;
  };
  auto main_loop = [&](auto rows) {
    if constexpr (S::AHEAD) {
      // Loads in the order X(i), W(i + EW): what may still be in flight when X(i) and W(i) are needed.
      constexpr int kAhead = (EW > 0 ? S::LW : 0) + (ST - 1) * (S::LW + S::LX);
      if constexpr (EW > 0) load_w(begin, 0);
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        load_x(min(begin + i, end - 1), i * S::XBUF);
        load_w(min(begin + i + EW, end - 1), (i + EW) * S::WBUF);
      }
      wait_loads<kAhead>();
      __builtin_amdgcn_s_barrier();
      read(f[0], 0, rows);
      // A step: its 64-byte parts in turn, the next part read ahead. Before the next step's first part is read, its loads
      // have landed and every wave holds this step's last part, so this step's buffers are free for loads.
      auto step = [&](auto more) {
#pragma unroll
        for (int h = 0; h < U; ++h) {
          if (h == U - 1) {
            wait_loads<decltype(more)::value ? kAhead - (S::LW + S::LX) : 0>();
            __builtin_amdgcn_s_barrier();
            if constexpr (decltype(more)::value) {
              load_x(s + ST, xbuf);
              load_w(min(s + ST + EW, end - 1), wbuf);
            }
            advance();
            read(f[(h + 1) & 1], 0, rows);
          } else {
            read(f[(h + 1) & 1], h + 1, rows);
          }
          __builtin_amdgcn_sched_barrier(0);
          multiply(f[h & 1], rows);
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (U == 1) f[0] = f[1];
      };
      for (; s < end - ST; ++s) step(std::true_type{});
      for (; s < end - 1; ++s) step(std::false_type{});
      const int left = a.n - s * BK;
#pragma unroll
      for (int h = 0; h < U; ++h) {
        if (h < U - 1) read(f[(h + 1) & 1], h + 1, rows);
        cut(f[h & 1], h, left);
        multiply(f[h & 1], rows);
      }
    } else {
      // Several workgroups share a compute unit: each reads and multiplies in turn, and they fill each other's waits.
      constexpr int LPS = S::LW + S::LX;
#pragma unroll
      for (int i = 0; i < ST - 1; ++i) {
        load_x(min(begin + i, end - 1), i * S::XBUF);
        load_w(min(begin + i, end - 1), i * S::WBUF);
      }
      for (; s < end - (ST - 1); ++s) {
        wait_loads<(ST - 2) * LPS>();               // step s is in LDS, and this wave is done with step s - 1's buffers
        __builtin_amdgcn_s_barrier();
        load_x(s + ST - 1, xbuf == 0 ? (ST - 1) * S::XBUF : xbuf - S::XBUF);
        load_w(s + ST - 1, wbuf == 0 ? (ST - 1) * S::WBUF : wbuf - S::WBUF);
#pragma unroll
        for (int h = 0; h < U; ++h) {
          read(f[0], h, rows);
          multiply(f[0], rows);
        }
        advance();
      }
      wait_loads<0>();
      __builtin_amdgcn_s_barrier();
      for (; s < end; ++s) {
#pragma unroll
        for (int h = 0; h < U; ++h) {
          read(f[0], h, rows);
          if (s == end - 1) cut(f[0], h, a.n - s * BK);
          multiply(f[0], rows);
        }
        advance();
      }
    }
  };
  // The rows' tiles of 16 go round the waves, and a wave multiplies all of its own, half or a quarter, as the tile has rows:
  // the last of an expert's tiles is part empty (8192 tokens over 128 experts 293 -> 278 us with tiles of 256 x 256, 301 ->
  // 295 and 297 -> 292 with the two of 256 x 128).
  const int there = ((tile.count + 15) / 16 - wx + S::WX - 1) / S::WX;
  if constexpr (RX >= 4) {
    if (there > RX / 2) main_loop(std::integral_constant<int, RX>{});
    else if (there > RX / 4) main_loop(std::integral_constant<int, RX / 2>{});
    else main_loop(std::integral_constant<int, RX / 4>{});
  } else {
    main_loop(std::integral_constant<int, RX>{});
  }
  wait_loads<0>();

  // Split inner axis: every workgroup of the tile leaves its sums, the last to arrive adds the others' (whole
  // numbers: the order does not matter) and goes on.
  if (a.splits > 1) {
    constexpr int T = 64 * NW;
    uint64_t* mine = a.partials + ((size_t)(rt * out_tiles + ot) * a.splits + sp) * (2 * T * AT * RX) + 2 * threadIdx.x;
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int r = 0; r < RX; ++r) put_partial(mine + 2 * T * (t * RX + r), acc[t][r]);
    __syncthreads();                              // the operands' LDS is done with: its first word is the flag
    if (!arrive_is_last(a.counters + rt * out_tiles + ot, a.splits, reinterpret_cast<uint32_t*>(sh))) return;
    for (int o = 0; o < a.splits; ++o) {
      if (o == sp) continue;
      uint64_t* theirs = mine + ((ptrdiff_t)o - sp) * (2 * T * AT * RX);
#pragma unroll
      for (int t = 0; t < AT; ++t)
#pragma unroll
        for (int r = 0; r < RX; ++r) acc[t][r] += get_partial(theirs + 2 * T * (t * RX + r));
    }
    if (threadIdx.x == 0) reset_counter(a.counters + rt * out_tiles + ot);
  }

  // The scales and places of the lane's outputs first: a store could not be passed by a load.
  const int ob = o0 + 16 * AT * wo;
  const float* ws = a.ws + (int64_t)tile.expert * a.m;
  float wsv[AT][4], xs[RX];
  int pair[RX];
#pragma unroll
  for (int t = 0; t < AT; ++t) {
    const int o = ob + S::output(t, g);
    if (o0 + TO <= a.m) {
      const float4_any f = *reinterpret_cast<const float4_any*>(ws + o);
#pragma unroll
      for (int c = 0; c < 4; ++c) wsv[t][c] = f[c];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) wsv[t][c] = ws[min(o + c, a.m - 1)];
    }
  }
#pragma unroll
  for (int r = 0; r < RX; ++r) {
    pair[r] = pair_of(a, tile, 16 * (S::WX * r + wx) + j);
    xs[r] = a.xs[max(pair[r], 0) / a.pairs_per_row];
  }
  constexpr int N = AT == 1 ? 4 : 8;
#pragma unroll
  for (int r = 0; r < RX; ++r) {
    if (pair[r] < 0) continue;
#pragma unroll
    for (int t = 0; t < AT; t += N / 4) {
      const int o = ob + S::output(t, g);
      if (o >= a.m) continue;
      float v[N];
#pragma unroll
      for (int c = 0; c < N; ++c) v[c] = (float)acc[t + c / 4][r][c % 4] * xs[r] * wsv[t + c / 4][c % 4];
      store_outputs<DT, N>(a.y, (int64_t)pair[r] * a.ldy + o, v, a.m - o);
    }
  }
}

template <class S, int DT>
static hipError_t launch_shape_t(const Int8Args& a, hipStream_t s) {
  const int ot = (a.m + S::TO - 1) / S::TO, rt = row_tiles(a, S::TX);
  const int64_t groups = (int64_t)ot * rt * a.splits + (a.zero_rest ? 8 : 0);   // 8: as zeros_number asks
  if (groups >= (int64_t)1 << 31) return hipErrorInvalidConfiguration;   // no accepted shape has as many
  const dim3 grid((unsigned)(groups < kGridWidth ? groups : kGridWidth), (unsigned)((groups + kGridWidth - 1) / kGridWidth));
  hipLaunchKernelGGL((int8_tile_kernel<S, DT>), grid, dim3(64 * S::NW), 0, s, a, ot, rt);
  return hipGetLastError();
}

template <class S>
static hipError_t launch_shape(const Int8Args& a, hipStream_t s) {
  if (a.out == kF32) return launch_shape_t<S, kF32>(a, s);
  if (a.out == kF16) return launch_shape_t<S, kF16>(a, s);
  return launch_shape_t<S, kBf16>(a, s);
}

// The tile shapes. What one costs, measured over 13 layers (300 to 28672 outputs, 768 to 20000 inputs) at 1 to 8192 rows
// and fitted: microseconds per 128 bytes of the inner axis for a compute unit that holds one workgroup, and for one that
// holds two; microseconds per tile beside that (its first loads, its stores).
struct TileCost {
  int out, rows, resident;
  float alone, shared, tile;
};
constexpr TileCost kTiles[] = {
    {256, 256, 1, 1.484f, 1.484f, 5.05f}, // TileShape<4, 8, 4, 2, 128, 2, 1>
    {256, 128, 1, 0.974f, 0.974f, 4.26f}, // TileShape<4, 4, 4, 2, 128, 3>
    {256, 128, 2, 1.10f, 2.15f, 1.8f},    // TileShape<4, 4, 4, 2, 64, 3, 0, 4>: two workgroups fill each other's waits
    {128, 128, 1, 0.533f, 0.533f, 2.24f}, // TileShape<2, 4, 4, 2, 128, 3>
    {128, 64, 2, 0.321f, 0.677f, 2.28f},  // TileShape<2, 4, 4, 1, 128, 3>
    {64, 32, 2, 0.124f, 0.222f, 1.13f},   // TileShape<1, 2, 4, 1, 256, 3>
    {32, 16, 2, 0.047f, 0.14f, 0.85f},    // TileShape<1, 1, 2, 1, 512, 3>
};
constexpr float kStreamRate = 5.3e6f;   // bytes per microsecond of a product that waits for memory alone

// The cheapest shape and split of the inner axis: rounds of workgroups over the compute units, and the time that the
// bytes take, of which a part is not hidden behind the other. Over the sweep this loses 0.5% against trying everything
// (17% at worst, 1.9 us of a 9.4 us product), and 1.1% over 7 sets of experts at 1 to 16384 tokens (22% at worst); the best
// single shape loses 19% on average and a factor of 2.1 at worst, the largest tile a factor of 1.9 and 6.2. A split inner
// axis costs the parts' sums, so only products with few tiles take one (64 x 4096 x 14336: 20.2 us whole, 15.6 us in two
// parts; 256 x 28672 x 8192: 70 us whole, 96 us in two). Experts: row tiles as an even routing fills them, one half-filled
// for each expert.
Int8Plan int8_plan(int M, int m, int n, int experts) {
  const float reached = experts > 0 ? (float)(experts < M ? experts : M) : 1.f;
  const float rows = (float)M / reached;
  const float stream = (reached * m * (float)n + (float)M * n + 2.f * M * m) / kStreamRate;
  const int steps = (n + 127) / 128;
  Int8Plan best{0, 1};
  float least = 3.0e38f;
  for (int shape = 0; shape < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++shape) {
    const TileCost& t = kTiles[shape];
    if (t.rows > 32 && t.rows > 2.f * rows) continue;          // more than half of it empty
    const float rt = experts > 0 ? reached * (rows / t.rows + 0.5f > 1.f ? rows / t.rows + 0.5f : 1.f)
                                 : (float)((M + t.rows - 1) / t.rows);
    const float tiles = rt * (float)((m + t.out - 1) / t.out);
    const int slots = kComputeUnits * t.resident;
    for (int splits : {1, 2, 3, 4, 6, 8}) {
      if (splits > 1 && (experts > 0 || tiles > kInt8Counters / 2 || splits * 512 > n)) break;
      const float groups = tiles * splits;
      const float rounds = (float)(int64_t)(groups / slots), rest = groups - rounds * slots;
      const float len = (float)((steps + splits - 1) / splits);
      float work = rounds * (t.shared * len + t.tile);
      if (rest > 0.f) work += (rest > kComputeUnits ? t.shared : t.alone) * len + t.tile;
      float us = (work > stream ? work : stream) + 0.2f * (work > stream ? stream : work);
      if (splits > 1) us += 0.9f + 2.1e-6f * splits * M * m;
      if (us < least) {
        least = us;
        best = {shape, splits};
      }
    }
  }
  return best;
}

void int8_plan_tile(const Int8Plan& p, int* outputs, int* rows) {
  *outputs = kTiles[p.shape].out;
  *rows = kTiles[p.shape].rows;
}

size_t int8_partial_bytes(int M, int m, int n) {
  const Int8Plan p = int8_plan(M, m, n, 0);
  if (p.splits <= 1) return 0;
  const TileCost& t = kTiles[p.shape];
  return (size_t)((m + t.out - 1) / t.out) * ((M + t.rows - 1) / t.rows) * p.splits * t.out * t.rows * 4;
}

hipError_t launch_int8_gemm(const Int8Args& args, hipStream_t s) {
  Int8Args a = args;
  const Int8Plan p = int8_plan(a.M, a.m, a.n, a.offsets ? a.experts : 0);
  a.splits = p.splits;
  switch (p.shape) {
    case 0: return launch_shape<TileShape<4, 8, 4, 2, 128, 2, 1>>(a, s);
    case 1: return launch_shape<TileShape<4, 4, 4, 2, 128, 3>>(a, s);
    case 2: return launch_shape<TileShape<4, 4, 4, 2, 64, 3, 0, 4>>(a, s);
    case 3: return launch_shape<TileShape<2, 4, 4, 2, 128, 3>>(a, s);
    case 4: return launch_shape<TileShape<2, 4, 4, 1, 128, 3>>(a, s);
    case 5: return launch_shape<TileShape<1, 2, 4, 1, 256, 3>>(a, s);
    case 6: return launch_shape<TileShape<1, 1, 2, 1, 512, 3>>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tg

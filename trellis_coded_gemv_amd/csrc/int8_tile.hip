// 8-bit products of more than a few rows: tiles of TO outputs x TX activation rows, both operands through LDS.
#include <type_traits>

#include "tg_int8.hpp"

namespace tg {

namespace {

// 16 bytes of global memory per lane to LDS at base + 16 * lane (base wave-uniform): from a lane's own address, or from
// a lane's offset to a wave-uniform address.
__device__ __forceinline__ void load_to_lds(const int8_t* p, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_base), "v"(p) : "memory");
}
__device__ __forceinline__ void load_to_lds(const int8_t* p, uint32_t offset, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds_base), "v"(offset), "s"(p) : "memory");
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
// step; ST: steps held in LDS.
template <int AT_, int RX_, int WO_, int WX_, int BK_, int ST_, int OCC_ = 2>
struct TileShape {
  static constexpr int AT = AT_, RX = RX_, WO = WO_, WX = WX_, BK = BK_, ST = ST_, OCC = OCC_;
  static constexpr int NW = WO * WX, TO = 16 * AT * WO, TX = 16 * RX * WX;
  static constexpr int RPI = 1024 / BK;                             // LDS rows filled by one load instruction
  static constexpr int LW = TO / RPI / NW, LX = TX / RPI / NW;      // load instructions of a wave per step
  static constexpr int BUF = (TO + TX) * BK;
  static_assert(LW * RPI * NW == TO && LX * RPI * NW == TX, "every wave loads whole instructions");
  static_assert(BK < 256 || (LW % 2 == 0 && LX % 2 == 0), "a wave's rows start at a multiple of the swizzle's period");
  // A row's 16-byte pieces are held in LDS in an order that depends on the row, so that the lanes which read the same
  // piece of neighbouring rows spread over the banks.
  static __device__ __forceinline__ int swizzle(int row) { return BK >= 128 ? row & 7 : (row >> 1) & 3; }
};

}  // namespace

template <class S, int DT>
__global__ __launch_bounds__(64 * S::NW, S::OCC) void int8_tile_kernel(const Int8Args a, int out_tiles, int row_tiles) {
  constexpr int AT = S::AT, RX = S::RX, BK = S::BK, ST = S::ST, TO = S::TO, TX = S::TX, NW = S::NW;
  __shared__ __attribute__((aligned(1024))) int8_t sh[ST * S::BUF];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int j = lane & 15, g = lane >> 4;
  // Workgroup -> tile and split. Workgroups b, b + 8, ... share an XCD and its L2: each XCD takes a run of neighbouring
  // tiles. Dense: 8 row tiles by all output tiles, rows first, so that an XCD's resident workgroups share a few row
  // tiles and output tiles. Experts: outputs first, so that an expert's tiles stay together.
  const int total = out_tiles * row_tiles;
  int id, sp = 0;
  {
    const int all = total * a.splits;
    const int per = all >> 3, rest = all & 7, x = blockIdx.x & 7;
    id = x * per + min(x, rest) + (blockIdx.x >> 3);
  }
  if (a.splits > 1) {
    const int t = id / a.splits;
    sp = id - t * a.splits;
    id = t;
  }
  int ot, rt;
  if (a.offsets) {
    rt = id / out_tiles;
    ot = id - rt * out_tiles;
  } else {
    const int band = id / (8 * out_tiles), in = id - band * 8 * out_tiles;
    const int high = min(8, row_tiles - band * 8);
    ot = in / high;
    rt = band * 8 + in - ot * high;
  }
  RowTile tile = find_tile(a, rt, TX);
  tile.expert = __builtin_amdgcn_readfirstlane(tile.expert);
  tile.first = __builtin_amdgcn_readfirstlane(tile.first);
  tile.count = __builtin_amdgcn_readfirstlane(tile.count);
  if (tile.count <= 0) return;
  const int o0 = ot * TO;
  const int wo = wave % S::WO, wx = wave / S::WO;

  // Loads: an instruction fills RPI rows of LDS; lane l the slot l % (BK / 16) of row l / (BK / 16), where the piece
  // slot ^ swizzle(row) of the row belongs. LDS row 16 (AT wo + t) + 4 g + v of the layer's side holds output
  // 16 AT wo + 4 AT g + 4 t + v, so that a lane ends with 4 AT neighbouring outputs of a row.
  const int lrow = lane / (BK / 16);
  auto piece = [&](int i) { return 16 * ((lane % (BK / 16)) ^ S::swizzle(S::RPI * i + lrow)); };   // of instruction i
  // The layer's rows are addressed by 32-bit offsets to the tile's first row (the launch keeps their stride below 2^23).
  const int8_t* wbase = a.w + ((int64_t)tile.expert * a.m + o0) * a.ldw;
  uint32_t woff[S::LW];
  const int8_t* xp[S::LX];
#pragma unroll
  for (int i = 0; i < S::LW; ++i) {
    const int q = S::RPI * (S::LW * wave + i) + lrow;
    const int o = q / (16 * AT) * (16 * AT) + 4 * AT * ((q >> 2) & 3) + 4 * ((q >> 4) % AT) + (q & 3);
    woff[i] = (uint32_t)min(o, a.m - 1 - o0) * (uint32_t)a.ldw;
  }
#pragma unroll
  for (int i = 0; i < S::LX; ++i) {
    const int q = S::RPI * (S::LX * wave + i) + lrow;
    xp[i] = a.x + (int64_t)(max(pair_of(a, tile, q), 0) / a.pairs_per_row) * a.ldx;
  }
  const uint32_t sh0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t*)sh;
  const uint32_t wfill = __builtin_amdgcn_readfirstlane(sh0 + wave * S::LW * 1024);
  const uint32_t xfill = __builtin_amdgcn_readfirstlane(sh0 + TO * BK + wave * S::LX * 1024);
  auto load = [&](int step, uint32_t buf) {
    const int k = step * BK, most = a.n - 16 - k;    // pieces past the end: any bytes of the row, not multiplied
#pragma unroll
    for (int i = 0; i < S::LW; ++i) load_to_lds(wbase, woff[i] + (uint32_t)(k + min(piece(i), most)), wfill + buf + i * 1024);
#pragma unroll
    for (int i = 0; i < S::LX; ++i) load_to_lds(xp[i] + (k + min(piece(i), most)), xfill + buf + i * 1024);
  };

  i32x4 acc[AT][RX];
#pragma unroll
  for (int t = 0; t < AT; ++t)
#pragma unroll
    for (int r = 0; r < RX; ++r) acc[t][r] = i32x4{0, 0, 0, 0};
  const int slot = 16 * (g ^ S::swizzle(j));     // of the step's first 64 bytes; the h-th 64: slot ^ 64 h
  const int abase = (wo * 16 * AT + j) * BK + slot, bbase = TO * BK + (wx * 16 * RX + j) * BK + slot;
  // The operands of 64 bytes of the inner axis: read from LDS while the matrix cores work on those before.
  struct Frags {
    i32x4 a[AT], b[RX];
  };
  auto read = [&](Frags& f, uint32_t buf, int h) {
    const int8_t* at = sh + buf;
#pragma unroll
    for (int r = 0; r < RX; ++r) f.b[r] = *reinterpret_cast<const i32x4*>(at + ((bbase ^ (64 * h)) + r * 16 * BK));
#pragma unroll
    for (int t = 0; t < AT; ++t) f.a[t] = *reinterpret_cast<const i32x4*>(at + ((abase ^ (64 * h)) + t * 16 * BK));
  };
  auto cut = [&](Frags& f, int h, int left) {    // pieces past the end of the inner axis count as zero
    if (64 * h + 16 * g >= left) {
#pragma unroll
      for (int r = 0; r < RX; ++r) f.b[r] = i32x4{0, 0, 0, 0};
    }
  };
  auto multiply = [&](const Frags& f) {
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int r = 0; r < RX; ++r) acc[t][r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.a[t], f.b[r], acc[t][r], 0, 0, 0);
  };
  const int steps_all = (a.n + BK - 1) / BK;
  const int begin = (int)((int64_t)steps_all * sp / a.splits), end = (int)((int64_t)steps_all * (sp + 1) / a.splits);
  constexpr int U = BK / 64, LPS = S::LW + S::LX;
  uint32_t buf = 0;                               // of step s
  auto next = [](uint32_t b) { return b == (uint32_t)(ST - 1) * S::BUF ? 0u : b + S::BUF; };
#pragma unroll
  for (int i = 0; i < ST; ++i) load(min(begin + i, end - 1), i * S::BUF);
  wait_loads<(ST - 1) * LPS>();
  __builtin_amdgcn_s_barrier();
  Frags f[2];
  read(f[0], 0, 0);
  int s = begin;
  // A step: its 64-byte parts in turn, the next part read ahead. Before the next step's first part is read, its loads
  // have landed and every wave holds this step's last part, so this step's buffer is free for the loads of step s + ST.
  auto step = [&](auto more) {
#pragma unroll
    for (int h = 0; h < U; ++h) {
      if (h == U - 1) {
        wait_loads<decltype(more)::value ? (ST - 2) * LPS : 0>();
        __builtin_amdgcn_s_barrier();
        if constexpr (decltype(more)::value) load(s + ST, buf);
        buf = next(buf);
        read(f[(h + 1) & 1], buf, 0);
      } else {
        read(f[(h + 1) & 1], buf, h + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      multiply(f[h & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (U == 1) f[0] = f[1];
  };
  for (; s < end - ST; ++s) step(std::true_type{});
  for (; s < end - 1; ++s) step(std::false_type{});
  const int left = a.n - s * BK;
#pragma unroll
  for (int h = 0; h < U; ++h) {
    if (h < U - 1) read(f[(h + 1) & 1], buf, h + 1);
    cut(f[h & 1], h, left);
    multiply(f[h & 1]);
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
    __shared__ uint32_t flag;
    if (!arrive_is_last(a.counters + rt * out_tiles + ot, a.splits, &flag)) return;
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

  // Lane: outputs o0 + 16 AT wo + 4 AT g + 4 t + v of row 16 RX wx + 16 r + j.
  const int ob = o0 + 16 * AT * wo + 4 * AT * g;
#pragma unroll
  for (int r = 0; r < RX; ++r) {
    const int p = pair_of(a, tile, 16 * (RX * wx + r) + j);
    if (p < 0) continue;
    const float xs = a.xs[p / a.pairs_per_row];
#pragma unroll
    for (int t = 0; t < AT; ++t) {
      const int o = ob + 4 * t;
      if (o >= a.m) continue;
      float v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = (float)acc[t][r][c] * xs * a.ws[(int64_t)tile.expert * a.m + min(o + c, a.m - 1)];
      store4<DT>(a.y, (int64_t)p * a.ldy + o, v, a.m - o, a.wide_y);
    }
  }
}

template <class S, int DT>
static hipError_t launch_shape_t(const Int8Args& a, hipStream_t s) {
  const int ot = (a.m + S::TO - 1) / S::TO, rt = row_tiles(a, S::TX);
  hipLaunchKernelGGL((int8_tile_kernel<S, DT>), dim3((unsigned)ot * (unsigned)rt * (unsigned)a.splits), dim3(64 * S::NW), 0,
                     s, a, ot, rt);
  return hipGetLastError();
}

template <class S>
static hipError_t launch_shape(const Int8Args& a, hipStream_t s) {
  if (a.out == kF32) return launch_shape_t<S, kF32>(a, s);
  if (a.out == kF16) return launch_shape_t<S, kF16>(a, s);
  return launch_shape_t<S, kBf16>(a, s);
}

hipError_t launch_int8_tile(const Int8Args& a, int shape, hipStream_t s) {
  switch (shape) {
    case 0: return launch_shape<TileShape<8, 4, 2, 4, 128, 2>>(a, s);   // 256 x 256
    case 1: return launch_shape<TileShape<4, 4, 2, 2, 128, 2>>(a, s);   // 128 x 128
    case 2: return launch_shape<TileShape<2, 4, 4, 1, 128, 3>>(a, s);   // 128 x 64
    case 3: return launch_shape<TileShape<2, 2, 4, 1, 128, 3>>(a, s);   // 128 x 32
    case 4: return launch_shape<TileShape<8, 4, 2, 4, 64, 4>>(a, s);    // 256 x 256
    case 5: return launch_shape<TileShape<8, 4, 2, 2, 64, 3>>(a, s);    // 256 x 128
    case 6: return launch_shape<TileShape<4, 4, 2, 2, 128, 4>>(a, s);   // 128 x 128
    case 7: return launch_shape<TileShape<8, 4, 2, 2, 128, 2>>(a, s);   // 256 x 128
    case 8: return launch_shape<TileShape<4, 4, 2, 2, 64, 4>>(a, s);   // 128 x 128
    case 9: return launch_shape<TileShape<4, 4, 4, 2, 128, 3>>(a, s);   // 256 x 128 8 waves
    case 10: return launch_shape<TileShape<4, 8, 2, 2, 64, 3>>(a, s);   // 128 x 256
    case 11: return launch_shape<TileShape<2, 4, 2, 1, 128, 4>>(a, s);   // 64 x 64
    case 12: return launch_shape<TileShape<4, 4, 4, 2, 64, 3, 4>>(a, s);   // 256x128
    case 13: return launch_shape<TileShape<4, 4, 2, 2, 64, 2, 4>>(a, s);   // 128x128
    case 14: return launch_shape<TileShape<4, 4, 2, 2, 64, 3, 3>>(a, s);   // 128x128
    case 15: return launch_shape<TileShape<2, 4, 4, 2, 128, 3>>(a, s);   // 128x128 8 waves
    case 16: return launch_shape<TileShape<4, 4, 4, 2, 64, 2, 4>>(a, s);   // 256x128
    case 17: return launch_shape<TileShape<8, 2, 2, 4, 64, 3, 4>>(a, s);   // 256x128
    case 18: return launch_shape<TileShape<2, 4, 4, 1, 256, 2>>(a, s);   // 128x64
    case 19: return launch_shape<TileShape<2, 2, 4, 1, 256, 2>>(a, s);   // 128x32
    case 20: return launch_shape<TileShape<1, 4, 4, 1, 256, 2>>(a, s);   // 64x64
    case 21: return launch_shape<TileShape<1, 2, 4, 1, 256, 3>>(a, s);   // 64x32
    case 22: return launch_shape<TileShape<2, 2, 4, 1, 128, 5>>(a, s);   // 128x32 deep
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tg

// 8-bit products of many rows: tiles of 256 outputs x 256 activation rows, fed through LDS.
#include "tg_int8.hpp"

namespace tg {

namespace {

constexpr int kTO = 256;            // outputs per tile
constexpr int kTX = 256;            // activation rows per tile
constexpr int kTK = 128;            // bytes of the inner axis per step
constexpr int kSide = kTO * kTK;    // LDS bytes of one operand of one step
constexpr int kBuf = 2 * kSide;

// 16 bytes of global memory per lane to LDS at base + 16 * lane (base wave-uniform).
__device__ __forceinline__ void load_to_lds(const int8_t* p, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_base), "v"(p) : "memory", "m0");
}

}  // namespace

template <int DT>
__global__ __launch_bounds__(512, 2) void int8_tile_kernel(const Int8Args a, int out_tiles, int row_tiles) {
  __shared__ __attribute__((aligned(1024))) int8_t sh[2 * kBuf];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int j = lane & 15, g = lane >> 4;
  // Workgroup -> tile. Workgroups b, b + 8, ... share an XCD and its L2: each XCD takes a run of neighbouring tiles.
  // Dense: 8 row tiles by all output tiles, rows first, so that an XCD's 32 resident workgroups share 8 row tiles and 4
  // output tiles. Experts: outputs first, so that an expert's tiles stay together.
  const int total = out_tiles * row_tiles;
  int id = blockIdx.x;
  {
    const int per = total >> 3, rest = total & 7, x = id & 7;
    id = x * per + min(x, rest) + (id >> 3);
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
  const RowTile tile = find_tile(a, rt, kTX);
  if (tile.count <= 0) return;
  const int o0 = ot * kTO;
  const int wo = wave & 1, wx = wave >> 1;

  // Loads: instruction i of wave w fills LDS rows 8 (4w + i) .. + 7 of either operand; lane l the 16-byte slot l % 8 of
  // row l / 8, where the row's piece (l % 8) ^ (row % 8) belongs.
  const int piece = 16 * ((lane & 7) ^ (lane >> 3));
  const int8_t* wp[4];
  const int8_t* xp[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = 8 * (4 * wave + i) + (lane >> 3);
    const int o = o0 + (q & 128) + 32 * ((q >> 2) & 3) + 4 * ((q >> 4) & 7) + (q & 3);
    wp[i] = a.w + ((int64_t)tile.expert * a.m + min(o, a.m - 1)) * a.ldw;
    xp[i] = a.x + (int64_t)(max(pair_of(a, tile, q), 0) / a.pairs_per_row) * a.ldx;
  }
  const uint32_t sh0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t*)sh;
  const uint32_t fill = __builtin_amdgcn_readfirstlane(sh0 + wave * 4096);
  auto load = [&](int step, int buf) {
    const int k = min(step * kTK + piece, a.n - 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      load_to_lds(wp[i] + k, fill + buf * kBuf + i * 1024);
      load_to_lds(xp[i] + k, fill + buf * kBuf + kSide + i * 1024);
    }
  };

  i32x4 acc[8][4];
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[t][r] = i32x4{0, 0, 0, 0};
  const int slot = 16 * (g ^ (lane & 7));       // the second half of a step: slot ^ 64
  const int abase = (wo * 128 + j) * kTK + slot, bbase = kSide + (wx * 64 + j) * kTK + slot;
  auto multiply = [&](int buf, int left) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x4 av[8], bv[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) bv[r] = *reinterpret_cast<const i32x4*>(sh + buf * kBuf + ((bbase ^ (64 * h)) + r * 16 * kTK));
#pragma unroll
      for (int t = 0; t < 8; ++t) av[t] = *reinterpret_cast<const i32x4*>(sh + buf * kBuf + ((abase ^ (64 * h)) + t * 16 * kTK));
      if (64 * h + 16 * g >= left) {
#pragma unroll
        for (int r = 0; r < 4; ++r) bv[r] = i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[t], bv[r], acc[t][r], 0, 0, 0);
    }
  };
  const int steps = (a.n + kTK - 1) / kTK;
  load(0, 0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  for (int s = 0; s < steps - 1; ++s) {
    load(s + 1, (s + 1) & 1);
    multiply(s & 1, kTK);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
  }
  multiply((steps - 1) & 1, a.n - (steps - 1) * kTK);

  // Lane: outputs o0 + 128 wo + 32 g + 4 t + v of row 64 wx + 16 r + j.
  const int ob = o0 + 128 * wo + 32 * g;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int p = pair_of(a, tile, 64 * wx + 16 * r + j);
    if (p < 0) continue;
    const float xs = a.xs[p / a.pairs_per_row];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int o = ob + 4 * t;
      if (o >= a.m) continue;
      float v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = (float)acc[t][r][c] * xs * a.ws[(int64_t)tile.expert * a.m + min(o + c, a.m - 1)];
      store4<DT>(a.y, (int64_t)p * a.ldy + o, v, a.m - o, a.wide_y);
    }
  }
}

hipError_t launch_int8_tile(const Int8Args& a, hipStream_t s) {
  const int ot = (a.m + kTO - 1) / kTO, rt = row_tiles(a, kTX);
  const dim3 grid((unsigned)ot * (unsigned)rt), block(512);
  if (a.out == kF32) hipLaunchKernelGGL(int8_tile_kernel<kF32>, grid, block, 0, s, a, ot, rt);
  else if (a.out == kF16) hipLaunchKernelGGL(int8_tile_kernel<kF16>, grid, block, 0, s, a, ot, rt);
  else hipLaunchKernelGGL(int8_tile_kernel<kBf16>, grid, block, 0, s, a, ot, rt);
  return hipGetLastError();
}

}  // namespace tg

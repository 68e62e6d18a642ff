// Products of e4m3 rows with a scale for each block of 128: Y[r, o] = sum_b xs[r, b] ws[o / 128, b] sum_{i in b} xq[r, i] wq[o, i],
// for a dense layer and for the experts of routed pairs, by tiles of TO outputs x TX rows.
//
// A block's sum leaves the matrix cores and is added to the output's by one fused multiply-add in binary32 with the product
// of its two scales, in rising order of the blocks; parts of a split inner axis are added in rising order too. So the
// same call gives the same bits. Which instruction forms a block's sum goes by the output's type:
//   16 bits  v_mfma_f32_16x16x128_f8f6f4, which aligns eight products at a time to the largest exponent among them (measured by
//            single products; a subnormal factor counts with the smallest normal one's) and drops what lies below 2^-13 of it.
//            So eight are off by 2^-10 of the largest at most, or by 2^-7 where that has a subnormal factor; on normally
//            distributed values 2^-16 of the result (2^-16.01 to 2^-16.07 over six shapes), where the type keeps 2^-11 or 2^-8;
//   32 bits  v_mfma_f32_16x16x32_f16 on the values widened to binary16, which hold them exactly: sums of binary32 (a block's is off by
//            2^-26 of itself on normal values, an output with its blocks' additions by 2^-23), at half of the rate of the matrix
//            cores. Products of few rows wait for the layer's bytes in either form.
//
// What bounds it (MI355X): 4096 x 28672 x 8192 bf16 runs at 2220-2350 TFLOP/s (820-867 us); the library's product with one scale for
// each side takes 705 us. Of an 885 us form, what is left without its loads was 663 us, without its scaling 797, without both
// 564; from registers alone, with the scaling, the matrix cores reach 3830-3900 TFLOP/s (500 us; 4550 without), the card's power.
// With every tile reading the same rows, out of L2, 756. So loads into LDS and scaling share the time beside the matrix cores.
// Larger instructions (32x32x64) with the scaling reach 3430 from registers. 32-bit outputs there: 1600 us, 1200 TFLOP/s.
// 1 x 28672 x 8192 reads 235 MB in 42.6 us (5.5 TB/s). 61 x 4096 x 14336 20 us for 61 MB: first loads, join of four parts and the
// widening. 8192 tokens over 128 experts, 1536 x 2048, top 8: 270-281 us; 2000 tokens, 2048 x 768, a row for each pair: 73-85 us, of
// which 42 us are the same with one step of the inner axis (first loads, lookups and stores of short tiles).
//
// The layer's rows are the A operand and the activation rows the B operand: lane l supplies row l % 16 and, of 128 bytes of
// the inner axis, the 16 at 16 (l / 16) and the 16 at 64 + 16 (l / 16) on both sides, and ends with four neighbouring outputs of row
// l % 16. Both sides and the scales reach LDS by loads that do not pass through registers, a ring of ST steps of BK bytes.
#include <type_traits>

#include "product_tiles.hpp"

namespace tg {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

namespace {

__device__ __forceinline__ void put_partial(uint64_t* p, f32x4 v) {
  const u32x4 u = __builtin_bit_cast(u32x4, v);
  __hip_atomic_store(p, (uint64_t)u[1] << 32 | u[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(p + 1, (uint64_t)u[3] << 32 | u[2], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ f32x4 get_partial(uint64_t* p) {
  const uint64_t a = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint64_t b = __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return __builtin_bit_cast(f32x4, u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)});
}

// 4 bytes of global memory per lane to LDS at base + 4 * lane, as load_to_lds.
__device__ __forceinline__ void load4_to_lds(const float* p, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds_base), "v"(p) : "m0", "memory");
}

// Eight e4m3 values as binary16, which holds every one of them.
__device__ __forceinline__ f16x8 widen(int lo, int hi) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A step's scales in LDS: every wave brings a slot of 64 floats. Its first PER hold its part of the rows' scales, numbered
// ((u WX + wx) 16 + j) RX + r for block u of the step and row 16 (WX r + wx) + j of the tile, so that a lane finds its rows' as
// neighbours; behind them the layer's scales of the wave's own outputs, one for each block of the step.
template <class S>
struct ScaleSlots {
  static constexpr int U = S::BK / 128;
  static constexpr int PER = S::TX * U / S::NW;
  static constexpr int BUF = S::NW * 256;        // LDS bytes of a step
  static_assert(S::BK % 128 == 0 && PER * S::NW == S::TX * U && PER % S::RX == 0 && PER + U <= 64, "");
  static __device__ __forceinline__ int slot(int value) { return value / PER * 64 + value % PER; }
};

}  // namespace

template <class S, int DT>
__global__ __launch_bounds__(64 * S::NW, S::OCC) void fp8_tile_kernel(const Product8Args a, int out_tiles, int row_tiles) {
  constexpr int AT = S::AT, RX = S::RX, BK = S::BK, ST = S::ST, TO = S::TO, TX = S::TX, NW = S::NW;
  using Slots = ScaleSlots<S>;
  constexpr int U = Slots::U, SLDS = S::XLDS + ST * S::XBUF;
  constexpr bool WIDE = DT == kF32;
  constexpr bool LARGE = AT * RX >= 16;          // registers for one set of operands beside the sums
  constexpr int LIST = SLDS + ST * Slots::BUF;   // the tile's entries of order
  __shared__ __attribute__((aligned(1024))) int8_t sh[LIST + (TX < 64 ? 64 : TX) * 4];
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
  auto xrow = [&](int i) { return S::RPI * (NW * i + wave) + lrow; };
  auto piece = [&](int row) { return 16 * ((lane % (BK / 16)) ^ S::swizzle(row)); };
  // The layer's rows are addressed by 32-bit offsets to the tile's first row (the launch keeps their stride below 2^23).
  const int8_t* wbase = a.w + ((int64_t)tile.expert * a.m + o0) * a.ldw;
  uint32_t woff[S::LW];
#pragma unroll
  for (int i = 0; i < S::LW; ++i) woff[i] = (uint32_t)min(lds_row_output(AT, wrow(i)), a.m - 1 - o0) * (uint32_t)a.ldw;
  const uint32_t sh0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t*)sh;
  const uint32_t wfill = __builtin_amdgcn_readfirstlane(sh0 + wave * S::LW * 1024);
  const uint32_t xfill = __builtin_amdgcn_readfirstlane(sh0 + S::XLDS + wave * 1024);
  const uint32_t sfill = __builtin_amdgcn_readfirstlane(sh0 + SLDS + wave * 256);
  auto load_w = [&](int step, uint32_t buf, int from, int to) {
    const int k = step * BK, most = a.n - 16 - k;    // pieces past the end: any bytes of the row, not multiplied
#pragma unroll
    for (int i = from; i < to; ++i)
      load_to_lds(wbase, woff[i] + (uint32_t)(k + min(piece(wrow(i)), most)), wfill + buf * S::WBUF + i * 1024);
  };
  const int steps_all = (a.n + BK - 1) / BK;
  const int begin = (int)((int64_t)steps_all * sp / a.splits), end = (int)((int64_t)steps_all * (sp + 1) / a.splits);
  int s = begin;

  // The layer's first rows are asked for while the experts' list of the tile's rows is on its way, which the rest of the loads wait
  // for, and which is kept for the stores (8192 tokens over 128 experts: 278 -> 270 us, 2000 tokens' down products 89 -> 85).
  const int* list = reinterpret_cast<const int*>(sh + LIST);
  if (a.offsets) {
    constexpr int WAVES = (TX + 63) / 64;        // whose lanes hold the list; the others ask for the same again
    const int part = wave % WAVES;
    load4_to_lds(reinterpret_cast<const float*>(a.order + tile.first + min(64 * part + lane, tile.count - 1)), sh0 + LIST + 256 * part);
  }
  load_w(begin, 0, 0, S::LW);
  if (a.offsets) {
    wait_loads<S::LW>();
    __builtin_amdgcn_s_barrier();
  }
  // Output row (pair) of the tile's row i, or -1, and its activation row.
  auto pair_at = [&](int i) {
    if (i >= tile.count) return -1;
    if (!a.offsets) return tile.first + i;
    const int p = list[i];
    return p >= 0 && p < a.M ? p : -1;
  };
  auto source = [&](int i) { return (int64_t)(max(pair_at(i), 0) / a.pairs_per_row); };
  const int8_t* xp[S::LX];
#pragma unroll
  for (int i = 0; i < S::LX; ++i) xp[i] = a.x + source(xrow(i)) * a.ldx;
  const int blocks = (a.n + 127) >> 7;           // of the inner axis
  const float* sp0;                              // where the lane's scale of block 0 of a step lies for step 0
  int su;                                        // which block of a step it is
  {
    const int v = wave * Slots::PER + min(lane, Slots::PER - 1), r = v % RX, vj = v / RX % 16, uw = v / (16 * RX);
    const int ob = min((o0 + 16 * AT * wo) >> 7, (a.m - 1) >> 7);
    const bool own = lane >= Slots::PER;
    su = own ? min(lane - Slots::PER, U - 1) : uw / S::WX;
    sp0 = own ? a.ws + ((int64_t)tile.expert * ((a.m + 127) >> 7) + ob) * blocks
              : a.xs + source(16 * (S::WX * r + uw % S::WX) + vj) * a.ldxs;
  }
  auto load_x = [&](int step, uint32_t buf, int from, int to) {
    const int k = step * BK, most = a.n - 16 - k;
#pragma unroll
    for (int i = from; i < to; ++i) load_to_lds(xp[i] + (k + min(piece(xrow(i)), most)), xfill + buf * S::XBUF + i * (NW * 1024));
  };
  auto load_s = [&](int step, uint32_t buf) { load4_to_lds(sp0 + min(step * U + su, blocks - 1), sfill + buf * Slots::BUF); };

  f32x4 acc[AT][RX];
#pragma unroll
  for (int t = 0; t < AT; ++t)
#pragma unroll
    for (int r = 0; r < RX; ++r) acc[t][r] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int slot = 16 * (g ^ S::swizzle(j));     // of the step's first 64 bytes; the h-th 64: slot ^ 64 h
  const int abase = (wo * 16 * AT + j) * BK + slot, bbase = S::XLDS + (wx * 16 + j) * BK + slot;
  uint32_t buf = 0;                              // of step s
  // Reads of block u of step s.
  auto both = [&](int at, int u) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(sh + (at ^ (128 * u))), hi = *reinterpret_cast<const i32x4*>(sh + (at ^ (128 * u + 64)));
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  auto read_w = [&](int t, int u) { return both(buf * S::WBUF + abase + t * 16 * BK, u); };
  auto read_x = [&](int r, int u) { return both(buf * S::XBUF + bbase + r * S::WX * 16 * BK, u); };
  auto scales = [&]() { return reinterpret_cast<const float*>(sh + SLDS + buf * Slots::BUF); };
  auto read_xs = [&](int r, int u) { return scales()[Slots::slot(((u * S::WX + wx) * 16 + j) * RX) + r]; };
  auto read_ws = [&](int u) { return scales()[wave * 64 + Slots::PER + u]; };
  auto cut = [&](i32x8& b, int left) {           // pieces past the end of the inner axis count as zero
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (64 * h + 16 * g >= left) {
#pragma unroll
        for (int d = 0; d < 4; ++d) b[4 * h + d] = 0;
      }
  };
  struct Wide {                                  // an operand widened
    f16x8 q[4];
  };
  auto widen_all = [&](const i32x8& v) {
    Wide w;
#pragma unroll
    for (int q = 0; q < 4; ++q) w.q[q] = widen(v[2 * q], v[2 * q + 1]);
    return w;
  };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  auto product = [&](const i32x8& w, const i32x8& x) { return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, 0, 0, 0, 0, 0, 0); };
  auto add = [&](f32x4& sum, const f32x4& p, float scale) {
#pragma unroll
    for (int c = 0; c < 4; ++c) sum[c] = fmaf(p[c], scale, sum[c]);
  };

  // A step's loads: W, X, scales; the first W is under way. kAhead may still be in flight when the first step's are needed.
  constexpr int kStep = S::LW + S::LX + 1, kAhead = (ST - 1) * kStep;
  auto first_loads = [&]() {
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      const int step = min(begin + i, end - 1);
      if (i > 0) load_w(step, i, 0, S::LW);
      load_x(step, i, 0, S::LX);
      load_s(step, i);
    }
    wait_loads<kAhead>();
    __builtin_amdgcn_s_barrier();
  };
  // On to the next step: its loads have landed and every wave holds the rest of this one in registers, so this step's buffers
  // are free for loads, of which `early` are under way.
  constexpr bool STREAM = LARGE && !WIDE;
  constexpr int kEarly = STREAM ? S::LW + S::LX / 2 : 0;
  auto next_step = [&](auto more) {
    wait_loads<decltype(more)::value ? kAhead - kStep + kEarly : 0>();
    __builtin_amdgcn_s_barrier();
    if constexpr (decltype(more)::value) {
      if constexpr (!STREAM) load_w(s + ST, buf, 0, S::LW);
      load_x(s + ST, buf, STREAM ? S::LX / 2 : 0, S::LX);
      load_s(s + ST, buf);
    }
    buf = buf == (uint32_t)(ST - 1) ? 0u : buf + 1u;
    ++s;
  };
  auto load_early = [&](int i) {
    if (i < S::LW) load_w(s + ST, buf, i, i + 1);
    else load_x(s + ST, buf, i - S::LW, i - S::LW + 1);
  };
  auto wait_lds = [&]() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };
  using More = std::true_type;
  using Rest = std::false_type;

  // Large tiles: the layer's operands of a block stay in registers, those of the rows come one tile of 16 ahead, and the sums of a
  // tile of 16 rows are added up while the matrix cores work on the next. Once every wave holds the layer's operands and the first
  // half of the rows', their buffers are filled again, a few loads with each of the row tiles that are left (4096 x 28672 x 8192: 851
  // us; all of them at once 875, at the end of a step 890; operands in groups of four tiles with one barrier a step 893; one product
  // between a sum and its addition 1008).
  auto stream_loop = [&](auto rows) __attribute__((always_inline)) {
    constexpr int R = decltype(rows)::value;
    static_assert(U == 1 && R % 2 == 0 && S::LX % 2 == 0, "");
    constexpr int kMiddle = R == RX ? R / 2 - 1 : R - 1;   // row tiles of fewer lie in the first half all
    i32x8 w[AT], x[2];
    f32x4 p[2][AT];
    float xs[2], ws, before = 0.f;               // before: the scale of the sums in hand
#pragma unroll
    for (int t = 0; t < AT; ++t) p[1][t] = zero;
    first_loads();
    auto read_first = [&](auto last) {
      if constexpr (!decltype(last)::value) {
        xs[0] = read_xs(0, 0);
        ws = read_ws(0);
        x[0] = read_x(0, 0);
      }
    };
    read_first(std::false_type{});
#pragma unroll
    for (int t = 0; t < AT; ++t) w[t] = read_w(t, 0);
    auto step = [&](auto last, auto more) __attribute__((always_inline)) {
      constexpr bool LAST = decltype(last)::value;
      const int left = LAST ? a.n - s * BK : BK;
      if constexpr (LAST) cut(x[0], left);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int cur = r & 1;
        const float scale = xs[cur] * ws;
        if (r < R - 1) {
          xs[cur ^ 1] = read_xs(r + 1, 0);
          x[cur ^ 1] = read_x(r + 1, 0);
          if constexpr (LAST) cut(x[cur ^ 1], left);
        }
        if (decltype(more)::value && r == kMiddle) {
          wait_lds();
          __builtin_amdgcn_s_barrier();
        }
        if (decltype(more)::value && r >= kMiddle) {
          constexpr int PER = (kEarly + R - kMiddle - 1) / (R - kMiddle);
#pragma unroll
          for (int e = (r - kMiddle) * PER; e < min(kEarly, (r - kMiddle + 1) * PER); ++e) load_early(e);
        }
        if (!LAST && r == R - 1) {
          next_step(more);
          read_first(last);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < AT; ++t) {
          p[cur][t] = product(w[t], x[cur]);
          if (!LAST && r == R - 1) w[t] = read_w(t, 0);
          add(acc[t][(r + R - 1) % R], p[cur ^ 1][t], before);
          __builtin_amdgcn_sched_barrier(0);
        }
        before = scale;
      }
    };
    while (s < end - ST) step(std::false_type{}, More{});
    while (s < end - 1) step(std::false_type{}, Rest{});
    step(std::true_type{}, Rest{});
#pragma unroll
    for (int t = 0; t < AT; ++t) add(acc[t][R - 1], p[1][t], before);
  };

  // Tiles of 32-bit outputs: the rows' operands of a block are widened at once and the layer's one by one, which leaves their places to
  // the next block's (4096 x 28672 x 8192: 1600 us; the layer's at once, with 256 x 256 tiles that do not fit the registers, 2150).
  auto wide_loop = [&](auto rows) __attribute__((always_inline)) {
    constexpr int R = decltype(rows)::value;
    static_assert(U == 1 && R % 2 == 0, "");
    i32x8 w[AT], x[R];
    float xs[R], ws;
    auto read_rows = [&]() __attribute__((always_inline)) {
      ws = read_ws(0);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        xs[r] = read_xs(r, 0);
        x[r] = read_x(r, 0);
      }
    };
    first_loads();
    read_rows();
#pragma unroll
    for (int t = 0; t < AT; ++t) w[t] = read_w(t, 0);
    auto step = [&](auto last, auto more) __attribute__((always_inline)) {
      constexpr bool LAST = decltype(last)::value;
      const int left = LAST ? a.n - s * BK : BK;
      Wide xw[R];
      float scale[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if constexpr (LAST) cut(x[r], left);
        scale[r] = xs[r] * ws;
        xw[r] = widen_all(x[r]);
      }
#pragma unroll
      for (int t = 0; t < AT; ++t) {
        const Wide ww = widen_all(w[t]);
        if constexpr (!LAST) {
          if (t == 0) next_step(more);
          w[t] = read_w(t, 0);
          if (t == AT - 1) read_rows();
        }
#pragma unroll
        for (int r = 0; r < R; r += 2) {
          f32x4 p[2];
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i) p[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ww.q[q], xw[r + i].q[q], q == 0 ? zero : p[i], 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 2; ++i) add(acc[t][r + i], p[i], scale[r + i]);
        }
      }
    };
    while (s < end - ST) step(std::false_type{}, More{});
    while (s < end - 1) step(std::false_type{}, Rest{});
    step(std::true_type{}, Rest{});
  };

  // Small tiles: the operands and scales of a block are read, and the sums of the block before are added up, while the matrix cores
  // work on a block (61 x 4096 x 14336 with 64 x 32 tiles: 16.1 us in 16 bits and 19.8 in 32; sums added at once 16.8 and 21.2).
  struct Frags {
    i32x8 w[AT], x[RX];
    float xs[RX], ws;
  };
  struct Sums {
    f32x4 p[AT][RX];
    float scale[RX];
  };
  auto ahead_loop = [&](auto rows) __attribute__((always_inline)) {
    constexpr int R = decltype(rows)::value;
    Frags f[2];
    Sums z[2];
    auto read = [&](Frags& f, int u) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        f.x[r] = read_x(r, u);
        f.xs[r] = read_xs(r, u);
      }
      f.ws = read_ws(u);
#pragma unroll
      for (int t = 0; t < AT; ++t) f.w[t] = read_w(t, u);
    };
    auto multiply = [&](const Frags& f, Sums& z) {
#pragma unroll
      for (int r = 0; r < R; ++r) z.scale[r] = f.xs[r] * f.ws;
      if constexpr (WIDE) {
        constexpr int PAIR = R > 1 ? 2 : 1;      // row tiles whose chains of four products take turns
        Wide w[AT];
#pragma unroll
        for (int t = 0; t < AT; ++t) w[t] = widen_all(f.w[t]);
#pragma unroll
        for (int r = 0; r < R; r += PAIR) {
          Wide x[PAIR];
#pragma unroll
          for (int i = 0; i < PAIR; ++i) x[i] = widen_all(f.x[r + i]);
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int t = 0; t < AT; ++t)
#pragma unroll
              for (int i = 0; i < PAIR; ++i)
                z.p[t][r + i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[t].q[q], x[i].q[q], q == 0 ? zero : z.p[t][r + i], 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t = 0; t < AT; ++t) z.p[t][r] = product(f.w[t], f.x[r]);
      }
    };
    auto add_up = [&](const Sums& z) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < AT; ++t) add(acc[t][r], z.p[t][r], z.scale[r]);
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
      z[1].scale[r] = 0.f;
#pragma unroll
      for (int t = 0; t < AT; ++t) z[1].p[t][r] = zero;
    }
    first_loads();
    read(f[0], 0);
    auto step = [&](auto more, auto first) __attribute__((always_inline)) {   // from set `first` on
      constexpr int F = decltype(first)::value;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u == U - 1) next_step(more);
        read(f[(F + u + 1) & 1], (u + 1) % U);
        __builtin_amdgcn_sched_barrier(0);
        multiply(f[(F + u) & 1], z[(F + u) & 1]);
        add_up(z[(F + u + 1) & 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto back = [&]() {                          // an odd number of blocks: what is in hand goes to where an even one leaves it
      f[0] = f[1];
      z[1] = z[0];
    };
    using Even = std::integral_constant<int, 0>;
    using Odd = std::integral_constant<int, 1>;
    if constexpr (U % 2 == 0) {
      while (s < end - ST) step(More{}, Even{});
    } else {
      while (s < end - ST - 1) {
        step(More{}, Even{});
        step(More{}, Odd{});
      }
      if (s < end - ST) {
        step(More{}, Even{});
        back();
      }
    }
    while (s < end - 1) {
      step(Rest{}, Even{});
      if constexpr (U % 2 == 1) back();
    }
    add_up(z[1]);
    const int left = a.n - s * BK;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (128 * u >= left) break;
      if (u < U - 1) read(f[(u + 1) & 1], u + 1);
#pragma unroll
      for (int r = 0; r < R; ++r) cut(f[u & 1].x[r], left - 128 * u);
      multiply(f[u & 1], z[0]);
      add_up(z[0]);
    }
  };
  auto main_loop = [&](auto rows) __attribute__((always_inline)) {
    if constexpr (LARGE && WIDE) wide_loop(rows);
    else if constexpr (LARGE) stream_loop(rows);
    else ahead_loop(rows);
  };
  // The rows' tiles of 16 go round the waves, and a wave multiplies all of its own, half or a quarter, as the tile has rows.
  const int there = ((tile.count + 15) / 16 - wx + S::WX - 1) / S::WX;
  constexpr int kLeast = LARGE ? 2 : 1;          // an even number of products, and of rows' tiles widened together
  if constexpr (RX / 2 >= kLeast) {
    if (there > RX / 2) {
      main_loop(std::integral_constant<int, RX>{});
    } else {
      if constexpr (RX / 4 >= kLeast) {
        if (there > RX / 4) main_loop(std::integral_constant<int, RX / 2>{});
        else main_loop(std::integral_constant<int, RX / 4>{});
      } else {
        main_loop(std::integral_constant<int, RX / 2>{});
      }
    }
  } else {
    main_loop(std::integral_constant<int, RX>{});
  }
  wait_loads<0>();

  // Split inner axis: every workgroup of the tile leaves its sums, the last to arrive adds all of them, the first part's first,
  // and goes on.
  if (a.splits > 1) {
    constexpr int T = 64 * NW;
    uint64_t* first = a.partials + (size_t)(rt * out_tiles + ot) * a.splits * (2 * T * AT * RX) + 2 * threadIdx.x;
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int r = 0; r < RX; ++r) put_partial(first + (size_t)sp * (2 * T * AT * RX) + 2 * T * (t * RX + r), acc[t][r]);
    __syncthreads();                              // the operands' LDS is done with: its first word is the flag
    if (!arrive_is_last(a.counters + rt * out_tiles + ot, a.splits, reinterpret_cast<uint32_t*>(sh))) return;
    for (int o = 0; o < a.splits; ++o) {
      uint64_t* part = first + (size_t)o * (2 * T * AT * RX);
#pragma unroll
      for (int t = 0; t < AT; ++t)
#pragma unroll
        for (int r = 0; r < RX; ++r) {
          const f32x4 v = get_partial(part + 2 * T * (t * RX + r));
          acc[t][r] = o == 0 ? v : acc[t][r] + v;
        }
    }
    if (threadIdx.x == 0) reset_counter(a.counters + rt * out_tiles + ot);
  }

  const int ob = o0 + 16 * AT * wo;
  int pair[RX];
#pragma unroll
  for (int r = 0; r < RX; ++r) pair[r] = pair_at(16 * (S::WX * r + wx) + j);
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
      for (int c = 0; c < N; ++c) v[c] = acc[t + c / 4][r][c % 4];
      store_outputs<DT, N>(a.y, (int64_t)pair[r] * a.ldy + o, v, a.m - o);
    }
  }
}

template <class S, int DT>
static hipError_t launch_shape_t(const Product8Args& a, hipStream_t s) {
  const int ot = (a.m + S::TO - 1) / S::TO, rt = row_tiles(a, S::TX);
  const int64_t groups = (int64_t)ot * rt * a.splits + (a.zero_rest ? 8 : 0);   // 8: as zeros_number asks
  if (groups >= (int64_t)1 << 31) return hipErrorInvalidConfiguration;   // no accepted shape has as many
  const dim3 grid((unsigned)(groups < kGridWidth ? groups : kGridWidth), (unsigned)((groups + kGridWidth - 1) / kGridWidth));
  hipLaunchKernelGGL((fp8_tile_kernel<S, DT>), grid, dim3(64 * S::NW), 0, s, a, ot, rt);
  return hipGetLastError();
}

template <class S>
static hipError_t launch_shape(const Product8Args& a, hipStream_t s) {
  if constexpr (S::AT * S::RX < 32) {
    if (a.out == kF32) return launch_shape_t<S, kF32>(a, s);
  }
  if (a.out == kF16) return launch_shape_t<S, kF16>(a, s);
  return launch_shape_t<S, kBf16>(a, s);
}

// The tile shapes: outputs, rows, workgroups on a compute unit.
struct TileSize {
  int out, rows, resident;
};
constexpr TileSize kTiles[] = {
    {256, 256, 1},  // TileShape<4, 8, 4, 2, 128, 2>, not for 32-bit outputs: its registers do not hold widened operands
    {256, 128, 1},  // TileShape<4, 4, 4, 2, 128, 3>
    {128, 128, 2},  // TileShape<4, 4, 2, 2, 128, 2>
    {128, 64, 2},   // TileShape<2, 4, 4, 1, 128, 3>
    {64, 64, 2},    // TileShape<2, 2, 2, 2, 128, 4>
    {64, 32, 2},    // TileShape<1, 2, 4, 1, 256, 3>
    {64, 16, 2},    // TileShape<1, 1, 4, 1, 256, 3>
    {32, 16, 2},    // TileShape<1, 1, 2, 1, 512, 3>
};
constexpr int kShapes = sizeof(kTiles) / sizeof(kTiles[0]);

// What they cost with 16-bit and with 32-bit outputs, fitted to 14 layers (130 to 28672 outputs, 768 to 20000 inputs) at 1 to 4096
// rows and 15 sets of experts: microseconds per 128 of the inner axis for a compute unit that holds one workgroup, and for one that
// holds two; microseconds per tile beside that (its first loads, its stores). Of the product: bytes per microsecond where it
// waits for memory alone, and the part of the shorter of the two times that the longer does not hide; of a split inner axis:
// microseconds at all, for each part, and for each value of a part's sums.
struct TileCost {
  float alone, shared, tile;
};
struct Costs {
  TileCost tiles[kShapes];
  float stream, unhidden, join, part, value;
};
constexpr Costs kCosts[2] = {
    {{{1.580f, 1.580f, 4.85f}, {0.959f, 0.959f, 3.62f}, {0.642f, 1.057f, 2.94f}, {0.467f, 0.758f, 2.39f},
      {0.313f, 0.483f, 2.05f}, {0.177f, 0.331f, 1.72f}, {0.151f, 0.263f, 1.14f}, {0.090f, 0.144f, 2.22f}},
     7.36e6f, 0.578f, 0.37f, 0.459f, 2.83e-6f},
    {{{0.f, 0.f, 0.f}, {1.555f, 1.555f, 7.85f}, {0.958f, 1.700f, 5.45f}, {0.601f, 1.079f, 3.59f},
      {0.394f, 0.668f, 2.59f}, {0.252f, 0.437f, 1.84f}, {0.198f, 0.325f, 1.45f}, {0.142f, 0.192f, 2.23f}},
     6.33e6f, 0.311f, 0.17f, 0.395f, 2.12e-6f}};

// The cheapest shape and split of the inner axis: rounds of workgroups over the compute units, and the time that the bytes
// take. Over the sweep this loses 1.6% against trying everything (38% at worst, 9 of 34 us). Experts: row tiles as an even routing
// fills them, one half-filled for each expert; their inner axis stays whole, as their launch has no workspace.
Int8Plan fp8_plan(int M, int m, int n, int experts, bool wide) {
  const Costs& c = kCosts[wide ? 1 : 0];
  const float reached = experts > 0 ? (float)(experts < M ? experts : M) : 1.f;
  const float rows = (float)M / reached;
  const float stream = (reached * m * (float)n + (float)M * n + 2.f * M * m) / c.stream;
  const int steps = (n + 127) / 128;
  Int8Plan best{0, 1};
  float least = 3.0e38f;
  for (int shape = wide ? 1 : 0; shape < kShapes; ++shape) {
    const TileSize& t = kTiles[shape];
    const TileCost& cost = c.tiles[shape];
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
      float work = rounds * (cost.shared * len + cost.tile);
      if (rest > 0.f) work += (rest > kComputeUnits ? cost.shared : cost.alone) * len + cost.tile;
      float us = (work > stream ? work : stream) + c.unhidden * (work > stream ? stream : work);
      if (splits > 1) us += c.join + c.part * splits + c.value * splits * M * m;
      if (us < least) {
        least = us;
        best = {shape, splits};
      }
    }
  }
  return best;
}

void fp8_plan_tile(const Int8Plan& p, int* outputs, int* rows) {
  *outputs = kTiles[p.shape].out;
  *rows = kTiles[p.shape].rows;
}

// For outputs of every type.
size_t fp8_partial_bytes(int M, int m, int n) {
  size_t most = 0;
  for (bool wide : {false, true}) {
    const Int8Plan p = fp8_plan(M, m, n, 0, wide);
    const TileSize& t = kTiles[p.shape];
    const size_t bytes = (size_t)((m + t.out - 1) / t.out) * ((M + t.rows - 1) / t.rows) * p.splits * t.out * t.rows * 4;
    if (p.splits > 1 && bytes > most) most = bytes;
  }
  return most;
}

hipError_t launch_fp8_gemm(const Product8Args& args, hipStream_t s) {
  Product8Args a = args;
  const Int8Plan p = fp8_plan(a.M, a.m, a.n, a.offsets ? a.experts : 0, a.out == kF32);
  a.splits = p.splits;
  switch (p.shape) {
    case 0: return launch_shape<TileShape<4, 8, 4, 2, 128, 2>>(a, s);
    case 1: return launch_shape<TileShape<4, 4, 4, 2, 128, 3>>(a, s);
    case 2: return launch_shape<TileShape<4, 4, 2, 2, 128, 2>>(a, s);
    case 3: return launch_shape<TileShape<2, 4, 4, 1, 128, 3>>(a, s);
    case 4: return launch_shape<TileShape<2, 2, 2, 2, 128, 4>>(a, s);
    case 5: return launch_shape<TileShape<1, 2, 4, 1, 256, 3>>(a, s);
    case 6: return launch_shape<TileShape<1, 1, 4, 1, 256, 3>>(a, s);
    case 7: return launch_shape<TileShape<1, 1, 2, 1, 512, 3>>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tg

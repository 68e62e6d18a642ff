// 8-bit integer rows and products: a quantiser with a scale for each row, and
// Y[r, o] = (sum_i xq[r, i] wq[o, i]) * xs[r] * ws[o] for a dense layer and for the experts of routed pairs.
//
// The sums are exact in int32 (|q| <= 128 and n < 2^17, so no sum leaves the type), whatever the order and the
// split of the work; one output is rounded three times in binary32 (the sum, and its product with either scale),
// and once more to a 16-bit output type.
#include "tg_int8.hpp"

namespace tg {

// ---------------------------------------------------------------------------
// Quantiser: amax = max |x_i| of the row, scale = amax / 127, q_i = the whole number nearest to x_i * 127 / amax,
// an exact half to the even one. Which step a value goes to is decided exactly: 127 x / amax is formed in binary64
// (off by at most 2^-45), where the true quotient of two binary32 values is either a half or at least 2^-33 away
// from one, and then rounded to a multiple of 2^-40, which puts every half back on the half.
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (DT == kF32) return reinterpret_cast<const float*>(p)[i];
  const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
  if constexpr (DT == kF16) return half_bits_to_float(b);
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}

__device__ __forceinline__ int quantize_step(float x, double inv) {
  const double t = (double)x * inv;
  const double snap = 1.5 * 4096.0;                        // ulp 2^-40: the grid that holds every half
  const double whole = 1.5 * 4503599627370496.0;           // ulp 1: rounds to the nearest whole number, halves to even
  const double s = (t + snap) - snap;
  return (int)__builtin_bit_cast(uint64_t, s + whole);     // the low word of the sum is the whole number
}

// max |x| of a row over its workgroup, as the bits of a binary32 (NaN and infinity come out on top of every number).
template <int THREADS>
__device__ __forceinline__ uint32_t row_max(uint32_t top, uint32_t* sh) {
  for (int m = 32; m; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m, 64));
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) top = max(top, sh[w]);
  return top;
}

// The row's scale, and 127 / amax for its steps. Not finite: scale NaN, and `finite` false.
struct RowScale {
  double inv;
  bool finite;
};

__device__ __forceinline__ RowScale row_scale(uint32_t top, float* scale) {
  const float amax = __builtin_bit_cast(float, top);
  RowScale r;
  r.finite = top < 0x7F800000u;
  r.inv = r.finite && top != 0 ? 127.0 / (double)amax : 0.0;
  if (threadIdx.x == 0) *scale = r.finite ? amax / 127.0f : __builtin_nanf("");
  return r;
}

// Rows whose 16-byte pieces are aligned: the row stays in registers between the two passes, PER pieces to a thread,
// and is read once.
template <int DT, int THREADS, int PER>
__global__ __launch_bounds__(THREADS) void quantize_rows_kernel(const void* __restrict__ x, int64_t ldx,
                                                                int8_t* __restrict__ q, int64_t ldq,
                                                                float* __restrict__ scales, int n) {
  constexpr int VEC = DT == kF32 ? 4 : 8;
  __shared__ uint32_t wmax[THREADS / 64];
  const int row = blockIdx.x;
  const int64_t base = (int64_t)row * ldx;
  const int pieces = n / VEC, rest = n - pieces * VEC;
  u32x4 v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = threadIdx.x + THREADS * i;
    v[i] = u32x4{0, 0, 0, 0};
    if (c < pieces) {
      if constexpr (DT == kF32) v[i] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const float*>(x) + base + c * VEC);
      else v[i] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(x) + base + c * VEC);
    }
  }
  float last = 0.f;                                        // the row's end, short of a piece: one value to a thread
  if ((int)threadIdx.x < rest) last = load_elem<DT>(x, base + pieces * VEC + threadIdx.x);
  uint32_t top = 0;
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int d = 0; d < 4; ++d) top = max(top, v[i][d] & 0x7FFFFFFFu);
  } else {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 t2 = {0, 0};
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int d = 0; d < 4; ++d)
        t2 = __builtin_elementwise_max(t2, __builtin_bit_cast(u16x2, v[i][d] & 0x7FFF7FFFu));
    const uint16_t t1 = max(t2[0], t2[1]);
    top = DT == kBf16 ? (uint32_t)t1 << 16 : __builtin_bit_cast(uint32_t, half_bits_to_float(t1));
  }
  top = max(top, __builtin_bit_cast(uint32_t, last) & 0x7FFFFFFFu);
  const RowScale r = row_scale(row_max<THREADS>(top, wmax), scales + row);
  int8_t* qr = q + (int64_t)row * ldq;
  const uint32_t keep = r.finite ? ~0u : 0u;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = threadIdx.x + THREADS * i;
    if (c >= pieces) break;
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h) {
      int b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t word = DT == kF32 ? v[i][e] : v[i][2 * h + e / 2];
        float f;
        if constexpr (DT == kF32) f = __builtin_bit_cast(float, word);
        else if constexpr (DT == kF16) f = half_bits_to_float((uint16_t)(word >> (16 * (e & 1))));
        else f = __builtin_bit_cast(float, e & 1 ? word & 0xFFFF0000u : word << 16);
        b[e] = quantize_step(f, r.inv);
      }
      w[h] = (((uint32_t)b[0] & 255u) | ((uint32_t)b[1] & 255u) << 8 | ((uint32_t)b[2] & 255u) << 16 | (uint32_t)b[3] << 24) & keep;
    }
    if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(qr + c * VEC) = w[0];
    else *reinterpret_cast<u32x2*>(qr + c * VEC) = u32x2{w[0], w[1]};
  }
  if ((int)threadIdx.x < rest) qr[pieces * VEC + threadIdx.x] = r.finite ? (int8_t)quantize_step(last, r.inv) : (int8_t)0;
}

// Rows of any alignment and length, read twice.
template <int DT, int THREADS>
__global__ __launch_bounds__(THREADS) void quantize_any_kernel(const void* __restrict__ x, int64_t ldx,
                                                               int8_t* __restrict__ q, int64_t ldq,
                                                               float* __restrict__ scales, int n) {
  __shared__ uint32_t wmax[THREADS / 64];
  const int row = blockIdx.x;
  const int64_t base = (int64_t)row * ldx;
  uint32_t top = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += THREADS)
    top = max(top, __builtin_bit_cast(uint32_t, load_elem<DT>(x, base + i)) & 0x7FFFFFFFu);
  const RowScale r = row_scale(row_max<THREADS>(top, wmax), scales + row);
  int8_t* qr = q + (int64_t)row * ldq;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += THREADS)
    qr[i] = r.finite ? (int8_t)quantize_step(load_elem<DT>(x, base + i), r.inv) : (int8_t)0;
}

template <int DT, int THREADS>
static void launch_quantize_rows(int rows, int n, const void* x, int64_t ldx, int8_t* q, int64_t ldq, float* scales,
                                 hipStream_t s) {
  constexpr int VEC = DT == kF32 ? 4 : 8;
  const int per = (n / VEC + THREADS - 1) / THREADS;
  const dim3 grid((unsigned)rows), block(THREADS);
  if (per <= 1) hipLaunchKernelGGL((quantize_rows_kernel<DT, THREADS, 1>), grid, block, 0, s, x, ldx, q, ldq, scales, n);
  else if (per <= 2) hipLaunchKernelGGL((quantize_rows_kernel<DT, THREADS, 2>), grid, block, 0, s, x, ldx, q, ldq, scales, n);
  else if (per <= 4) hipLaunchKernelGGL((quantize_rows_kernel<DT, THREADS, 4>), grid, block, 0, s, x, ldx, q, ldq, scales, n);
  else hipLaunchKernelGGL((quantize_rows_kernel<DT, THREADS, 8>), grid, block, 0, s, x, ldx, q, ldq, scales, n);
}

template <int DT>
static hipError_t launch_quantize_t(int rows, int n, const void* x, int64_t ldx, int8_t* q, int64_t ldq, float* scales,
                                    hipStream_t s) {
  constexpr int VEC = DT == kF32 ? 4 : 8;
  const bool aligned = (uintptr_t)x % 16 == 0 && (uintptr_t)q % VEC == 0 &&
                       (rows == 1 || (ldx % VEC == 0 && ldq % VEC == 0));
  const int pieces = n / VEC;
  if (aligned && pieces <= 256 && pieces >= 1) launch_quantize_rows<DT, 256>(rows, n, x, ldx, q, ldq, scales, s);
  else if (aligned && pieces <= 8 * 256 && rows > 512) launch_quantize_rows<DT, 256>(rows, n, x, ldx, q, ldq, scales, s);
  else if (aligned && pieces <= 8 * 1024 && pieces >= 1) launch_quantize_rows<DT, 1024>(rows, n, x, ldx, q, ldq, scales, s);
  else if (n <= 1024) hipLaunchKernelGGL((quantize_any_kernel<DT, 256>), dim3((unsigned)rows), dim3(256), 0, s, x, ldx, q, ldq, scales, n);
  else hipLaunchKernelGGL((quantize_any_kernel<DT, 1024>), dim3((unsigned)rows), dim3(1024), 0, s, x, ldx, q, ldq, scales, n);
  return hipGetLastError();
}

hipError_t launch_int8_quantize(int rows, int n, const void* x, int dtype, int64_t ldx, int8_t* q, int64_t ldq,
                                float* scales, hipStream_t s) {
  if (dtype == kF32) return launch_quantize_t<kF32>(rows, n, x, ldx, q, ldq, scales, s);
  if (dtype == kF16) return launch_quantize_t<kF16>(rows, n, x, ldx, q, ldq, scales, s);
  return launch_quantize_t<kBf16>(rows, n, x, ldx, q, ldq, scales, s);
}

// ---------------------------------------------------------------------------
// Products. The layer's rows are the A operand of v_mfma_i32_16x16x64_i8 and the activation rows the B operand, so a
// lane ends with four neighbouring outputs of one activation row. Lane l supplies row l % 16 and the 16 bytes at
// 16 * (l / 16) of a 64-byte step on both sides.
// ---------------------------------------------------------------------------

// A workgroup of 8 waves owns 16*OT outputs and 16*RT activation rows; its waves share out the inner axis in blocks
// of 256 bytes and are summed through LDS at the end.
template <int RT, int OT, int DT>
__global__ __launch_bounds__(512) void int8_rows_kernel(const Int8Args a) {
  __shared__ i32x4 red[8][OT * RT][64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int j = lane & 15, g = lane >> 4;
  const int o0 = blockIdx.x * 16 * OT;
  const RowTile tile = find_tile(a, blockIdx.y, 16 * RT);
  if (tile.count <= 0) return;
  const int8_t* wp[OT];
  const int8_t* xp[RT];
#pragma unroll
  for (int t = 0; t < OT; ++t) wp[t] = a.w + ((int64_t)tile.expert * a.m + min(o0 + 16 * t + j, a.m - 1)) * a.ldw + 16 * g;
#pragma unroll
  for (int r = 0; r < RT; ++r) xp[r] = a.x + (int64_t)(max(pair_of(a, tile, 16 * r + j), 0) / a.pairs_per_row) * a.ldx + 16 * g;
  i32x4 acc[OT][RT];
#pragma unroll
  for (int t = 0; t < OT; ++t)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[t][r] = i32x4{0, 0, 0, 0};
  const int nb = a.n >> 8;
  for (int b = wave; b < nb; b += 8) {
    i32x4 wv[4][OT], xv[4][RT];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int t = 0; t < OT; ++t) wv[u][t] = *reinterpret_cast<const i32x4*>(wp[t] + b * 256 + u * 64);
#pragma unroll
      for (int r = 0; r < RT; ++r) xv[u][r] = *reinterpret_cast<const i32x4*>(xp[r] + b * 256 + u * 64);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int t = 0; t < OT; ++t)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[t][r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[u][t], xv[u][r], acc[t][r], 0, 0, 0);
  }
  if (wave == (nb & 7)) {   // the rest of the inner axis, below 256 bytes: 16-byte pieces past its end count as zero
    for (int k = nb * 256; k < a.n; k += 64) {
      const bool in = k + 16 * g < a.n;
      i32x4 wv[OT], xv[RT];
#pragma unroll
      for (int t = 0; t < OT; ++t) wv[t] = in ? *reinterpret_cast<const i32x4*>(wp[t] + k) : i32x4{0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < RT; ++r) xv[r] = in ? *reinterpret_cast<const i32x4*>(xp[r] + k) : i32x4{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < OT; ++t)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[t][r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[t], xv[r], acc[t][r], 0, 0, 0);
    }
  }
#pragma unroll
  for (int t = 0; t < OT; ++t)
#pragma unroll
    for (int r = 0; r < RT; ++r) red[wave][t * RT + r][lane] = acc[t][r];
  __syncthreads();
  for (int i = threadIdx.x; i < OT * RT * 64; i += 512) {
    const int tr = i >> 6, l = i & 63;
    i32x4 sum = red[0][tr][l];
#pragma unroll
    for (int w = 1; w < 8; ++w) sum += red[w][tr][l];
    const int t = tr / RT, r = tr % RT;
    const int p = pair_of(a, tile, 16 * r + (l & 15));
    const int o = o0 + 16 * t + 4 * (l >> 4);
    if (p < 0 || o >= a.m) continue;
    const float xs = a.xs[p / a.pairs_per_row];
    float v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = (float)sum[c] * xs * a.ws[(int64_t)tile.expert * a.m + min(o + c, a.m - 1)];
    store4<DT>(a.y, (int64_t)p * a.ldy + o, v, a.m - o, a.wide_y);
  }
}

template <int RT, int OT>
static hipError_t launch_rows(const Int8Args& a, int tiles, hipStream_t s) {
  const dim3 grid((unsigned)((a.m + 16 * OT - 1) / (16 * OT)), (unsigned)tiles), block(512);
  if (a.out == kF32) hipLaunchKernelGGL((int8_rows_kernel<RT, OT, kF32>), grid, block, 0, s, a);
  else if (a.out == kF16) hipLaunchKernelGGL((int8_rows_kernel<RT, OT, kF16>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((int8_rows_kernel<RT, OT, kBf16>), grid, block, 0, s, a);
  return hipGetLastError();
}

// Outputs and rows of the tile shapes of int8_tile.hip.
struct TileSize {
  int out, rows;
};
constexpr TileSize kTiles[] = {{256, 256}, {128, 128}, {128, 64}, {128, 32}, {256, 256}, {256, 128}, {128, 128}, {256, 128}, {128, 128}, {256, 128}, {128, 256}, {64, 64}, {256,128},{128,128},{128,128},{128,128},{256,128},{256,128},{128,64},{128,32},{64,64},{64,32},{128,32}};

Int8Plan int8_plan(int M, int m, int n, int experts) {
  const int avg = experts > 0 ? (M + experts - 1) / experts : M;
  if (avg <= 16) return {-1, 1};
  if (avg <= 32) return {3, 1};
  if (avg <= 64) return {2, 1};
  if (avg <= 128) return {1, 1};
  return {0, 1};
}

size_t int8_partial_bytes(int M, int m, int n) {
  const Int8Plan p = int8_plan(M, m, n, 0);
  if (p.splits <= 1) return 0;
  const TileSize t = kTiles[p.shape];
  return (size_t)((m + t.out - 1) / t.out) * ((M + t.rows - 1) / t.rows) * p.splits * t.out * t.rows * 4;
}

hipError_t launch_int8_gemm(const Int8Args& args, hipStream_t s) {
  Int8Args a = args;
  const Int8Plan p = int8_plan(a.M, a.m, a.n, a.offsets ? a.experts : 0);
  a.splits = p.splits;
  if (p.shape >= 0) return launch_int8_tile(a, p.shape, s);
  return launch_rows<1, 1>(a, row_tiles(a, 16), s);
}

}  // namespace tg

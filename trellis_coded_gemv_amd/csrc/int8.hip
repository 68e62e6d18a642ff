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

template <int DT>
__global__ __launch_bounds__(256) void quantize_kernel(const void* __restrict__ x, int64_t ldx, int8_t* __restrict__ q,
                                                       int64_t ldq, float* __restrict__ scales, int n) {
  __shared__ uint32_t wmax[4];
  const int row = blockIdx.x;
  const int64_t base = (int64_t)row * ldx;
  uint32_t top = 0;                                        // max of |x| as bits: NaN and infinity come out on top
  for (int i = threadIdx.x; i < n; i += 256)
    top = max(top, __builtin_bit_cast(uint32_t, load_elem<DT>(x, base + i)) & 0x7FFFFFFFu);
  for (int m = 32; m; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m, 64));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = top;
  __syncthreads();
  top = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  const float amax = __builtin_bit_cast(float, top);
  const bool finite = top < 0x7F800000u;
  if (threadIdx.x == 0) scales[row] = finite ? amax / 127.0f : __builtin_nanf("");
  const double inv = finite && top != 0 ? 127.0 / (double)amax : 0.0;
  int8_t* qr = q + (int64_t)row * ldq;
  for (int i = threadIdx.x; i < n; i += 256)
    qr[i] = finite ? (int8_t)quantize_step(load_elem<DT>(x, base + i), inv) : (int8_t)0;
}

hipError_t launch_int8_quantize(int rows, int n, const void* x, int dtype, int64_t ldx, int8_t* q, int64_t ldq,
                                float* scales, hipStream_t s) {
  const dim3 grid((unsigned)rows), block(256);
  if (dtype == kF32) hipLaunchKernelGGL(quantize_kernel<kF32>, grid, block, 0, s, x, ldx, q, ldq, scales, n);
  else if (dtype == kF16) hipLaunchKernelGGL(quantize_kernel<kF16>, grid, block, 0, s, x, ldx, q, ldq, scales, n);
  else hipLaunchKernelGGL(quantize_kernel<kBf16>, grid, block, 0, s, x, ldx, q, ldq, scales, n);
  return hipGetLastError();
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

hipError_t launch_int8_gemm(const Int8Args& a, hipStream_t s) {
  const int avg = a.offsets ? (a.M + a.experts - 1) / a.experts : a.M;
  if (avg <= 16) return launch_rows<1, 1>(a, row_tiles(a, 16), s);
  if (avg <= 32) return launch_rows<2, 2>(a, row_tiles(a, 32), s);
  if (avg > 128) return launch_int8_tile(a, s);
  return launch_rows<4, 2>(a, row_tiles(a, 64), s);
}

}  // namespace tg

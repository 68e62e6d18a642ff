// e4m3 rows with a scale for each 128 values, and e4m3 layers with a scale for each block of 128 x 128:
//     amax = max |x_i| of the block, scale = amax / 448, q_i = the e4m3 value nearest to 448 x_i / amax.
#include "product_tiles.hpp"
#include "rows8.hpp"

namespace tg {

namespace {

// What a block's lanes share after its largest magnitude is known, as the bits of a binary32.
struct BlockScale {
  double inv, amax;
  bool finite;
};

__device__ __forceinline__ BlockScale block_scale(uint32_t top) {
  BlockScale s;
  s.finite = top < 0x7F800000u;
  s.amax = (double)__builtin_bit_cast(float, top);
  s.inv = s.finite && top != 0 ? (double)kE4m3Max / s.amax : 0.0;
  return s;
}

// Rounded once; not finite: NaN.
__device__ __forceinline__ float scale_of(const BlockScale& s) {
  return s.finite ? (float)(s.amax / (double)kE4m3Max) : __builtin_nanf("");
}

__device__ __forceinline__ uint32_t top8(const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
  return top;
}

// A lane's eight steps. Blocks that are not finite hold zeros.
__device__ __forceinline__ void store_steps(uint8_t* q, const float (&v)[8], const BlockScale& s, int valid) {
  const double p[2][4] = {{v[0], v[1], v[2], v[3]}, {v[4], v[5], v[6], v[7]}};
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) w[h] = s.finite ? e4m3_steps(p[h], s.inv, s.amax) : 0u;
  if (valid >= 8) {
    *reinterpret_cast<u32x2_any*>(q) = u32x2_any{w[0], w[1]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) q[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

}  // namespace

// Blocks of 128 values of a row, numbered row by row: 16 lanes to a block, PER blocks to a lane whose loads are all under
// way before the first is looked at.
template <int DT, int PER>
__global__ __launch_bounds__(256) void fp8_rows_kernel(const void* __restrict__ x, int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                                                       float* __restrict__ scales, int64_t lds, int n, uint32_t per_row, uint32_t blocks) {
  const int l = threadIdx.x & 15;
  const uint64_t first = ((uint64_t)blockIdx.y << kGridShift | blockIdx.x) * (16 * PER) + (threadIdx.x >> 4);
  Raw8 raw[PER];
  uint32_t row[PER];
  int at[PER], valid[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint64_t block = first + 16 * i;
    row[i] = (uint32_t)block / per_row;
    at[i] = ((uint32_t)block - row[i] * per_row) * 128 + 8 * l;
    valid[i] = block < blocks ? n - at[i] : 0;
    load8<DT>(raw[i], x, block < blocks ? (int64_t)row[i] * ldx + at[i] : 0, valid[i]);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    float v[8];
    widen8<DT>(raw[i], v);
    const BlockScale s = block_scale(row16_max(top8(v)));
    if (first + 16 * i >= blocks) break;
    if (l == 0) scales[(int64_t)row[i] * lds + (at[i] >> 7)] = scale_of(s);
    if (valid[i] > 0) store_steps(q + (int64_t)row[i] * ldq + at[i], v, s, valid[i]);
  }
}

// A workgroup for each block of 128 x 128: 16 lanes to a row, 8 rows to a lane.
template <int DT>
__global__ __launch_bounds__(256) void fp8_layer_kernel(const void* __restrict__ x, int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                                                        float* __restrict__ scales, int64_t lds, int rows, int n, uint32_t per_row, uint32_t blocks) {
  __shared__ uint32_t sh[4];
  const uint64_t block = (uint64_t)blockIdx.y << kGridShift | blockIdx.x;
  if (block >= blocks) return;
  const uint32_t br = (uint32_t)block / per_row, bc = (uint32_t)block - br * per_row;
  const int row0 = (int)br * 128 + (threadIdx.x >> 4), at = (int)bc * 128 + 8 * (threadIdx.x & 15);
  Raw8 raw[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) load8<DT>(raw[i], x, (int64_t)min(row0 + 16 * i, rows - 1) * ldx + min(at, n - 1), row0 + 16 * i < rows ? n - at : 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    widen8<DT>(raw[i], v);
    top = max(top, top8(v));
  }
  for (int m = 32; m; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m, 64));
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = top;
  __syncthreads();
  const BlockScale s = block_scale(max(max(sh[0], sh[1]), max(sh[2], sh[3])));
  if (threadIdx.x == 0) scales[(int64_t)br * lds + bc] = scale_of(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    widen8<DT>(raw[i], v);
    if (row0 + 16 * i < rows && at < n) store_steps(q + (int64_t)(row0 + 16 * i) * ldq + at, v, s, n - at);
  }
}

// Workgroups over two dimensions of a launch: one holds fewer than 2^32 threads.
static dim3 grid_of(uint64_t groups) {
  return dim3((unsigned)(groups < kGridWidth ? groups : kGridWidth), (unsigned)((groups + kGridWidth - 1) / kGridWidth));
}

template <int DT>
static hipError_t launch_fp8_t(int rows, int n, const void* x, int64_t ldx, bool layer, uint8_t* q, int64_t ldq, float* scales,
                               int64_t lds, hipStream_t s) {
  const uint32_t per_row = ((uint32_t)n + 127) / 128;
  const uint64_t blocks = (uint64_t)(layer ? ((uint32_t)rows + 127) / 128 : (uint32_t)rows) * per_row;   // below 2^32: fp8_quantize's sizes
  if (layer) hipLaunchKernelGGL(fp8_layer_kernel<DT>, grid_of(blocks), dim3(256), 0, s, x, ldx, q, ldq, scales, lds, rows, n, per_row, (uint32_t)blocks);
  else if (blocks <= 16 * 1024) hipLaunchKernelGGL((fp8_rows_kernel<DT, 1>), grid_of((blocks + 15) / 16), dim3(256), 0, s, x, ldx, q, ldq, scales, lds, n, per_row, (uint32_t)blocks);
  else hipLaunchKernelGGL((fp8_rows_kernel<DT, 4>), grid_of((blocks + 63) / 64), dim3(256), 0, s, x, ldx, q, ldq, scales, lds, n, per_row, (uint32_t)blocks);
  return hipGetLastError();
}

hipError_t launch_fp8_quantize(int rows, int n, const void* x, int dtype, int64_t ldx, bool layer, uint8_t* q, int64_t ldq,
                               float* scales, int64_t lds, hipStream_t s) {
  if (dtype == kF32) return launch_fp8_t<kF32>(rows, n, x, ldx, layer, q, ldq, scales, lds, s);
  if (dtype == kF16) return launch_fp8_t<kF16>(rows, n, x, ldx, layer, q, ldq, scales, lds, s);
  return launch_fp8_t<kBf16>(rows, n, x, ldx, layer, q, ldq, scales, lds, s);
}

}  // namespace tg

// e4m3 rows with a scale for each 128 values, and e4m3 layers with a scale for each block of 128 x 128:
//     amax = max |x_i| of the block, scale = amax / 448, q_i = the e4m3 value nearest to 448 x_i / amax.
// Bound by memory: 8192 x 8192 fp16 (203 MB) 38.6 us, 5.2 TB/s, where a large copy moves 4.9 to 5.1; 4096 x 14336 bf16 (178 MB) 37.7
// us, binary32 53 us (5.5 TB/s; the same rows again and again 32, 35 and 44 us); a layer of 28672 x 8192 bf16 (705 MB) 127 to 139 us. One row of 8192 takes 2.3 us. Quotients and scales
// by binary64 divisions and one block to a lane took 41.2 us for 4096 x 14336, four blocks to a lane 39.3.
#include "product_tiles.hpp"
#include "rows8.hpp"

namespace tg {

namespace {

// A block's scale, rounded once; top: the bits of its largest magnitude. Not finite: NaN. The quotient is corrected by its exact
// remainder, which leaves it rounded once where neither is near the ends of binary32.
__device__ __forceinline__ float scale_of(uint32_t top, bool plain) {
  const float amax = __builtin_bit_cast(float, top);
  if (!plain) return top < 0x7F800000u ? amax / kE4m3Max : __builtin_nanf("");
  constexpr float inv = 1.f / kE4m3Max;
  const float q = amax * inv;
  return fmaf(fmaf(-kE4m3Max, q, amax), inv, q);
}

// Bits of the largest magnitude of eight values, as a binary32.
template <int DT>
__device__ __forceinline__ uint32_t top8(const Raw8& r) {
  if constexpr (DT == kF32) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(r.a[i] & 0x7FFFFFFFu, r.b[i] & 0x7FFFFFFFu));
    return top;
  } else {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 t = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, r.a[i] & 0x7FFF7FFFu));
    const uint16_t top = max(t[0], t[1]);
    return DT == kBf16 ? (uint32_t)top << 16 : __builtin_bit_cast(uint32_t, half_bits_to_float(top));
  }
}

// A lane's eight steps. Blocks that are not finite hold zeros.
template <bool TAIL>
__device__ __forceinline__ void store_steps(uint8_t* q, const float (&v)[8], const BlockFactors& f, uint32_t top, int valid) {
  const float amax = __builtin_bit_cast(float, top);
  uint32_t w[2] = {0, 0};
  if (top < 0x7F800000u) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x[4] = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
      const double p[4] = {x[0], x[1], x[2], x[3]};
      w[h] = e4m3_steps(x, p, f, (double)amax);
    }
  }
  store_bytes<TAIL>(q, w, valid);
}

}  // namespace

// Blocks of 128 values of a row, numbered row by row: 16 lanes to a block, PER blocks to a lane whose loads are all under
// way before the first is looked at.
template <int DT, int PER, bool TAIL>
__global__ __launch_bounds__(256) void fp8_rows_kernel(const void* __restrict__ x, int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                                                       float* __restrict__ scales, int64_t lds, int n, uint32_t per_row, uint32_t blocks) {
  const int l = threadIdx.x & 15;
  const uint64_t first = ((uint64_t)blockIdx.y << kGridShift | blockIdx.x) * (16 * PER) + (threadIdx.x >> 4);
  Raw8 raw[PER];
  uint32_t row[PER], col[PER];
  int valid[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t block = (uint32_t)first + 16 * i;
    if (i == 0 || per_row < 16) {
      row[i] = block / per_row;
      col[i] = block - row[i] * per_row;
    } else {                                     // 16 blocks on: in this row or the next
      col[i] = col[i - 1] + 16;
      row[i] = row[i - 1] + (col[i] >= per_row ? 1 : 0);
      col[i] -= col[i] >= per_row ? per_row : 0;
    }
    valid[i] = first + 16 * i < blocks ? n - (int)(128 * col[i]) - 8 * l : 0;
    load8<DT, TAIL>(raw[i], x, (int64_t)row[i] * ldx + (128 * col[i] + 8 * l), valid[i]);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    float v[8];
    widen8<DT>(raw[i], v);
    const uint32_t top = row16_max(top8<DT>(raw[i]));
    const BlockFactors f = block_factors(__builtin_bit_cast(float, top));
    if (first + 16 * i >= blocks) break;
    if (l == 0) scales[(int64_t)row[i] * lds + col[i]] = scale_of(top, f.plain);
    if (valid[i] > 0) store_steps<TAIL>(q + (int64_t)row[i] * ldq + (128 * col[i] + 8 * l), v, f, top, valid[i]);
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
  for (int i = 0; i < 8; ++i) load8<DT, true>(raw[i], x, (int64_t)min(row0 + 16 * i, rows - 1) * ldx + min(at, n - 1), row0 + 16 * i < rows ? n - at : 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, top8<DT>(raw[i]));
  for (int m = 32; m; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m, 64));
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = top;
  __syncthreads();
  top = max(max(sh[0], sh[1]), max(sh[2], sh[3]));
  const BlockFactors f = block_factors(__builtin_bit_cast(float, top));
  if (threadIdx.x == 0) scales[(int64_t)br * lds + bc] = scale_of(top, f.plain);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    widen8<DT>(raw[i], v);
    if (row0 + 16 * i < rows && at < n) store_steps<true>(q + (int64_t)(row0 + 16 * i) * ldq + at, v, f, top, n - at);
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
  const uint32_t b32 = (uint32_t)blocks;
  if (layer) {
    hipLaunchKernelGGL(fp8_layer_kernel<DT>, grid_of(blocks), dim3(256), 0, s, x, ldx, q, ldq, scales, lds, rows, n, per_row, b32);
  } else if (n % 8 != 0) {
    hipLaunchKernelGGL((fp8_rows_kernel<DT, 2, true>), grid_of((blocks + 31) / 32), dim3(256), 0, s, x, ldx, q, ldq, scales, lds, n, per_row, b32);
  } else if (blocks <= 16 * 1024) {
    hipLaunchKernelGGL((fp8_rows_kernel<DT, 1, false>), grid_of((blocks + 15) / 16), dim3(256), 0, s, x, ldx, q, ldq, scales, lds, n, per_row, b32);
  } else {
    hipLaunchKernelGGL((fp8_rows_kernel<DT, 2, false>), grid_of((blocks + 31) / 32), dim3(256), 0, s, x, ldx, q, ldq, scales, lds, n, per_row, b32);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_quantize(int rows, int n, const void* x, int dtype, int64_t ldx, bool layer, uint8_t* q, int64_t ldq,
                               float* scales, int64_t lds, hipStream_t s) {
  if (dtype == kF32) return launch_fp8_t<kF32>(rows, n, x, ldx, layer, q, ldq, scales, lds, s);
  if (dtype == kF16) return launch_fp8_t<kF16>(rows, n, x, ldx, layer, q, ldq, scales, lds, s);
  return launch_fp8_t<kBf16>(rows, n, x, ldx, layer, q, ldq, scales, lds, s);
}

}  // namespace tg

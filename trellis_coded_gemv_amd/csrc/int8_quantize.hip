// 8-bit rows with a scale for each row. Bound by memory: 4096 rows of 14336 bf16 values (117 MB in, 59 MB out) take 30
// us, 5.9 TB/s, where a large copy moves 5.1; reading a row twice took 105 us. Rows of 14335, none of them aligned: 40 us (72
// read value by value). One row of 8192 takes 2.7 us.
#include "tg_device.hpp"
#include "tg_internal.hpp"

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

// Rows of up to PER * THREADS 16-byte pieces, at any address: the row stays in registers between the two passes, PER
// pieces to a thread, and is read once.
template <int DT, int THREADS, int PER>
__global__ __launch_bounds__(THREADS) void quantize_rows_kernel(const void* __restrict__ x, int64_t ldx,
                                                                int8_t* __restrict__ q, int64_t ldq,
                                                                float* __restrict__ scales, int n, int rows) {
  constexpr int VEC = DT == kF32 ? 4 : 8;
  __shared__ uint32_t wmax[THREADS / 64];
  const int row = blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= rows) return;
  const int64_t base = (int64_t)row * ldx;
  const int pieces = n / VEC, rest = n - pieces * VEC;
  u32x4 v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = threadIdx.x + THREADS * i;
    v[i] = u32x4{0, 0, 0, 0};
    if (c < pieces) {
      if constexpr (DT == kF32) v[i] = *reinterpret_cast<const u32x4_any*>(reinterpret_cast<const float*>(x) + base + c * VEC);
      else v[i] = *reinterpret_cast<const u32x4_any*>(reinterpret_cast<const uint16_t*>(x) + base + c * VEC);
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
    if constexpr (VEC == 4) *reinterpret_cast<u32_any*>(qr + c * VEC) = w[0];
    else *reinterpret_cast<u32x2_any*>(qr + c * VEC) = u32x2_any{w[0], w[1]};
  }
  if ((int)threadIdx.x < rest) qr[pieces * VEC + threadIdx.x] = r.finite ? (int8_t)quantize_step(last, r.inv) : (int8_t)0;
}

// Longer rows, read twice and value by value: 4096 rows of 40960 binary32 values 246 us (3.4 TB/s; 32768 of them 126 us, 5.3
// TB/s, by the kernel above), 1024 of 131072 bf16 163 us, one row of 131072 28 us.
template <int DT>
__global__ __launch_bounds__(1024) void quantize_long_kernel(const void* __restrict__ x, int64_t ldx, int8_t* __restrict__ q,
                                                             int64_t ldq, float* __restrict__ scales, int n, int rows) {
  constexpr int THREADS = 1024;
  __shared__ uint32_t wmax[THREADS / 64];
  const int row = blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= rows) return;
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

// A workgroup for each row; one dimension of a launch holds fewer than 2^32 threads.
static dim3 row_grid(int rows) {
  const unsigned x = rows < 65536 ? (unsigned)rows : 65536u;
  return dim3(x, ((unsigned)rows + x - 1) / x);
}

// A row is a workgroup's, of 256 threads where a thread then holds one 16-byte piece (4096 rows of 1024 fp16 values: 5.6
// us, with 1024 threads 14.2), or up to four of many rows (2048 x 8192: 11.6 and 13.1), else of 1024 (1 x 8192: 2.7 and
// 3.1; 4096 x 14336: 30 and 48).
template <int DT, int THREADS>
static void launch_quantize_rows(int rows, int n, const void* x, int64_t ldx, int8_t* q, int64_t ldq, float* scales,
                                 hipStream_t s) {
  constexpr int VEC = DT == kF32 ? 4 : 8;
  const int per = (n / VEC + THREADS - 1) / THREADS;
  const dim3 grid = row_grid(rows), block(THREADS);
  if (per <= 1) hipLaunchKernelGGL((quantize_rows_kernel<DT, THREADS, 1>), grid, block, 0, s, x, ldx, q, ldq, scales, n, rows);
  else if (per <= 2) hipLaunchKernelGGL((quantize_rows_kernel<DT, THREADS, 2>), grid, block, 0, s, x, ldx, q, ldq, scales, n, rows);
  else if (per <= 4) hipLaunchKernelGGL((quantize_rows_kernel<DT, THREADS, 4>), grid, block, 0, s, x, ldx, q, ldq, scales, n, rows);
  else hipLaunchKernelGGL((quantize_rows_kernel<DT, THREADS, 8>), grid, block, 0, s, x, ldx, q, ldq, scales, n, rows);
}

template <int DT>
static hipError_t launch_quantize_t(int rows, int n, const void* x, int64_t ldx, int8_t* q, int64_t ldq, float* scales,
                                    hipStream_t s) {
  constexpr int VEC = DT == kF32 ? 4 : 8;
  const int pieces = n / VEC;
  if (pieces <= 256 || (pieces <= 4 * 256 && rows >= 512)) launch_quantize_rows<DT, 256>(rows, n, x, ldx, q, ldq, scales, s);
  else if (pieces <= 8 * 1024) launch_quantize_rows<DT, 1024>(rows, n, x, ldx, q, ldq, scales, s);
  else hipLaunchKernelGGL(quantize_long_kernel<DT>, row_grid(rows), dim3(1024), 0, s, x, ldx, q, ldq, scales, n, rows);
  return hipGetLastError();
}

hipError_t launch_int8_quantize(int rows, int n, const void* x, int dtype, int64_t ldx, int8_t* q, int64_t ldq,
                                float* scales, hipStream_t s) {
  if (dtype == kF32) return launch_quantize_t<kF32>(rows, n, x, ldx, q, ldq, scales, s);
  if (dtype == kF16) return launch_quantize_t<kF16>(rows, n, x, ldx, q, ldq, scales, s);
  return launch_quantize_t<kBf16>(rows, n, x, ldx, q, ldq, scales, s);
}

}  // namespace tg

// Root-mean-square norm of rows, with the residual's addition before it and rows of 16 or 32 bits, or of 8 with scales, behind it:
//     h = round(x + residual), r = 1 / sqrt(mean(h^2) + eps), p = h w;
//     y = p r,   or   q = the step nearest to T p / amax, scale = amax r / T
// with T = 127 and amax the row's largest |p| (int8), or T = 448 and that of each 128 values (e4m3). The norm scales a row as a
// whole, so the steps do not depend on it: they are decided on the exact products p, which binary64 holds.
#include <type_traits>

#include "product_tiles.hpp"
#include "rows8.hpp"

namespace tg {

namespace {

// The int8 step nearest to 127 p / amax, halves to the even one; inv = 127 / amax. t is off by at most 2^-44: unless it lies
// that near to a half, its nearest whole number is the step. Else 254 |p| is compared with (2 k + 1) amax, of products in two
// parts, as they have up to 56 bits.
__device__ __forceinline__ int int8_step(double p, double inv, double amax) {
  const double t = p * inv, k = rint(t);
  if (fabs(fabs(t - k) - 0.5) > 0x1p-30) return (int)k;
  const double low = floor(fabs(t)), odd = 2.0 * low + 1.0;
  const double a = 254.0 * fabs(p), b = odd * amax;
  const double rest = (a - b) + (fma(254.0, fabs(p), -a) - fma(odd, amax, -b));
  const int m = (int)low + (rest > 0.0 || (rest == 0.0 && ((int)low & 1)) ? 1 : 0);
  return p < 0.0 ? -m : m;
}

template <class F>
__device__ __forceinline__ void with_type(int type, F f) {
  if (type == kF32) f(std::integral_constant<int, kF32>{});
  else if (type == kF16) f(std::integral_constant<int, kF16>{});
  else f(std::integral_constant<int, kBf16>{});
}

__device__ __forceinline__ double wave_sum(double v) {
  v += dpp64<0x128>(v);                          // row_ror 8, 4, 2, 1: the sum of a row's 16 lanes, in each of them
  v += dpp64<0x124>(v);
  v += dpp64<0x122>(v);
  v += dpp64<0x121>(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

__device__ __forceinline__ double wave_max(double v) {
  v = row16_max(v);
  v = fmax(v, __shfl_xor(v, 16, 64));
  return fmax(v, __shfl_xor(v, 32, 64));
}

// Eight values rounded to a 16-bit type.
template <int DT>
__device__ __forceinline__ void round8(float (&v)[8]) {
  Raw8 r{};
#pragma unroll
  for (int i = 0; i < 4; ++i) r.a[i] = half_bits<DT>(v[2 * i]) | half_bits<DT>(v[2 * i + 1]) << 16;
  widen8<DT>(r, v);
}

}  // namespace

// A row is a workgroup's, in registers from its one read to its one write: piece c of eight values to thread c % THREADS, PER
// pieces to a thread, so that 16 neighbouring lanes hold 128 neighbouring values.
template <int THREADS, int PER>
__global__ __launch_bounds__(THREADS) void rms_norm_kernel(const NormArgs a) {
  __shared__ double sums[THREADS / 64], tops[THREADS / 64];
  const int row = blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.rows) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto at = [&](int i) { return 8 * ((int)threadIdx.x + THREADS * i); };   // first value of the thread's piece i
  Raw8 xr[PER], rr[PER], wr[PER];
  with_type(a.x_type, [&](auto t) {
#pragma unroll
    for (int i = 0; i < PER; ++i) load8<decltype(t)::value>(xr[i], a.x, (int64_t)row * a.ldx + min(at(i), a.n - 1), a.n - at(i));
  });
  if (a.residual) {
    with_type(a.r_type, [&](auto t) {
#pragma unroll
      for (int i = 0; i < PER; ++i) load8<decltype(t)::value>(rr[i], a.residual, (int64_t)row * a.ldr + min(at(i), a.n - 1), a.n - at(i));
    });
  }
  with_type(a.w_type, [&](auto t) {
#pragma unroll
    for (int i = 0; i < PER; ++i) load8<decltype(t)::value>(wr[i], a.w, min(at(i), a.n - 1), a.n - at(i));
  });

  float h[PER][8];
  with_type(a.x_type, [&](auto t) {
#pragma unroll
    for (int i = 0; i < PER; ++i) widen8<decltype(t)::value>(xr[i], h[i]);
  });
  if (a.residual) {
    with_type(a.r_type, [&](auto t) {
      constexpr int DT = decltype(t)::value;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        float r[8];
        widen8<DT>(rr[i], r);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] += r[e];
        if constexpr (DT != kF32) round8<DT>(h[i]);
        if (at(i) < a.n) store_outputs<DT, 8>(a.total, (int64_t)row * a.ldt + at(i), h[i], a.n - at(i));
      }
    });
  }

  double sum = 0.0, top = 0.0;
  uint32_t word = 0;
  float w[PER][8];
  with_type(a.w_type, [&](auto t) {
#pragma unroll
    for (int i = 0; i < PER; ++i) widen8<decltype(t)::value>(wr[i], w[i]);
  });
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fma((double)h[i][e], (double)h[i][e], sum);
  if (a.out == kInt8) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double p = (double)h[i][e] * (double)w[i][e];
        top = fmax(top, fabs(p));
        word = max(word, magnitude_word(p));
      }
    if (word >= kNotFinite) top = __builtin_inf();
    top = wave_max(top);
  }
  sum = wave_sum(sum);
  if constexpr (THREADS > 64) {
    if (lane == 0) {
      sums[wave] = sum;
      tops[wave] = top;
    }
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int v = 0; v < THREADS / 64; ++v) {
      sum += sums[v];
      top = fmax(top, tops[v]);
    }
  }
  const bool finite = sum < __builtin_inf();     // a square of finite binary32 values is far from the end of binary64
  const double mean = sum / (double)a.n + (double)a.eps;
  const double r = !finite ? __builtin_nan("") : mean > 0.0 ? 1.0 / sqrt(mean) : 0.0;

  if (a.out == kInt8) {
    const bool good = finite && top < __builtin_inf();
    const double inv = good && top > 0.0 ? 127.0 / top : 0.0;
    if (threadIdx.x == 0) a.scales[(int64_t)row * a.lds] = good ? (float)(top * r / 127.0) : __builtin_nanf("");
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int valid = a.n - at(i);
      if (valid <= 0) break;
      uint32_t b[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        b[e >> 2] |= ((uint32_t)(good ? int8_step((double)h[i][e] * (double)w[i][e], inv, top) : 0) & 255u) << (8 * (e & 3));
      uint8_t* q = reinterpret_cast<uint8_t*>(a.y) + (int64_t)row * a.ldy + at(i);
      if (valid >= 8) {
        *reinterpret_cast<u32x2_any*>(q) = u32x2_any{b[0], b[1]};
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < valid) q[e] = (uint8_t)(b[e >> 2] >> (8 * (e & 3)));
      }
    }
  } else if (a.out == kE4m3) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      double p[2][4], most = 0.0;
      uint32_t hi = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e >> 2][e & 3] = (double)h[i][e] * (double)w[i][e];
        most = fmax(most, fabs(p[e >> 2][e & 3]));
        hi = max(hi, magnitude_word(p[e >> 2][e & 3]));
      }
      most = row16_max(most);
      const bool good = finite && row16_max(hi) < kNotFinite;
      const int valid = a.n - at(i);
      if (valid <= 0) break;
      if ((lane & 15) == 0) a.scales[(int64_t)row * a.lds + (at(i) >> 7)] = good ? (float)(most * r / (double)kE4m3Max) : __builtin_nanf("");
      const double inv = good && most > 0.0 ? (double)kE4m3Max / most : 0.0;
      uint32_t b[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) b[k] = good ? e4m3_steps(p[k], inv, most) : 0u;
      uint8_t* q = reinterpret_cast<uint8_t*>(a.y) + (int64_t)row * a.ldy + at(i);
      if (valid >= 8) {
        *reinterpret_cast<u32x2_any*>(q) = u32x2_any{b[0], b[1]};
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < valid) q[e] = (uint8_t)(b[e >> 2] >> (8 * (e & 3)));
      }
    }
  } else {
    with_type(a.out, [&](auto t) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = (float)((double)h[i][e] * (double)w[i][e] * r);
        if (at(i) < a.n) store_outputs<decltype(t)::value, 8>(a.y, (int64_t)row * a.ldy + at(i), y, a.n - at(i));
      }
    });
  }
}

// A row is a wave's up to 1024 values, and of 256 threads where a thread then holds one piece, or up to four of many rows, else
// of 1024.
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  const int pieces = (a.n + 7) / 8;
  const unsigned x = a.rows < 65536 ? (unsigned)a.rows : 65536u;
  const dim3 grid(x, ((unsigned)a.rows + x - 1) / x);
  if (pieces <= 64) hipLaunchKernelGGL((rms_norm_kernel<64, 1>), grid, dim3(64), 0, s, a);
  else if (pieces <= 128) hipLaunchKernelGGL((rms_norm_kernel<64, 2>), grid, dim3(64), 0, s, a);
  else if (pieces <= 256) hipLaunchKernelGGL((rms_norm_kernel<256, 1>), grid, dim3(256), 0, s, a);
  else if (pieces <= 512 && a.rows >= 512) hipLaunchKernelGGL((rms_norm_kernel<256, 2>), grid, dim3(256), 0, s, a);
  else if (pieces <= 1024 && a.rows >= 512) hipLaunchKernelGGL((rms_norm_kernel<256, 4>), grid, dim3(256), 0, s, a);
  else if (pieces <= 1024) hipLaunchKernelGGL((rms_norm_kernel<1024, 1>), grid, dim3(1024), 0, s, a);
  else if (pieces <= 2048) hipLaunchKernelGGL((rms_norm_kernel<1024, 2>), grid, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((rms_norm_kernel<1024, 4>), grid, dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace tg

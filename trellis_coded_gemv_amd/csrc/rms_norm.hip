// Root-mean-square norm of rows, with the residual's addition before it and rows of 16 or 32 bits, or of 8 with scales, behind it:
//     h = round(x + residual), r = 1 / sqrt(mean(h^2) + eps), p = h w;
//     y = p r,   or   q = the step nearest to T p / amax, scale = amax r / T
// with T = 127 and amax the row's largest |p| (int8), or T = 448 and that of each 128 values (e4m3). The norm scales a row as a
// whole, so the steps do not depend on it: they are decided on the exact products p, which binary64 holds.
//
// Bound by memory: 8192 x 8192 bf16 with a residual into e4m3 (472 MB) 93 to 98 us, 5.0 TB/s, where a large copy moves 4.9 to 5.1; into
// bf16 (537 MB) 102 to 105 us; into int8 with binary32 weights 113 us, where the instructions show. A row of which no thread sees an
// end inside eight values has code without it: with that code 125, 124 and 121 us. One row of 8192 takes 4.1 us.
#include <type_traits>

#include "product_tiles.hpp"
#include "rows8.hpp"

namespace tg {

namespace {

// The int8 step nearest to 127 p / amax, halves to the even one; inv = 127 / amax. t is off by at most 2^-44: unless it lies
// that near to a half, its nearest whole number is the step. Else 254 |p| is compared with (2 k + 1) amax, of products in two
// parts, as they have up to 56 bits: a and b are rounded, and what they lack is added behind their difference. So a - b has to take a as it
// was rounded: fused into fma(254, |p|, -b) it would hold what a lacks already, and decide ties by it.
__device__ __forceinline__ int int8_step(double p, double inv, double amax) {
#pragma clang fp contract(off)
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

// Eight values as bits of a type; those of 16-bit types are rounded.
__device__ __forceinline__ void widen(const Raw8& r, int type, float (&v)[8]) {
  with_type(type, [&](auto t) { widen8<decltype(t)::value>(r, v); });
}

template <bool NARROW>
__device__ __forceinline__ void narrow(const float (&v)[8], int type, Raw8& r) {
  if (!NARROW && type == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.a[i] = __builtin_bit_cast(uint32_t, v[i]);
      r.b[i] = __builtin_bit_cast(uint32_t, v[i + 4]);
    }
  } else if (type == kF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.a[i] = half_bits<kF16>(v[2 * i]) | half_bits<kF16>(v[2 * i + 1]) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.a[i] = half_bits<kBf16>(v[2 * i]) | half_bits<kBf16>(v[2 * i + 1]) << 16;
  }
}

// The first `valid` of eight values to a row.
template <bool NARROW, bool TAIL>
__device__ __forceinline__ void store8(const Raw8& r, int type, void* p, int64_t at, int valid) {
  if (!NARROW && type == kF32) {
    float* f = reinterpret_cast<float*>(p) + at;
    if (!TAIL || valid >= 8) {
      *reinterpret_cast<u32x4_any*>(f) = r.a;
      *reinterpret_cast<u32x4_any*>(f + 4) = r.b;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < valid) f[i] = __builtin_bit_cast(float, (uint32_t)r.a[i]);
        if (i + 4 < valid) f[i + 4] = __builtin_bit_cast(float, (uint32_t)r.b[i]);
      }
    }
  } else {
    uint16_t* h = reinterpret_cast<uint16_t*>(p) + at;
    if (!TAIL || valid >= 8) {
      *reinterpret_cast<u32x4_any*>(h) = r.a;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid) h[i] = (uint16_t)(r.a[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// The pieces of a thread: `type` asks for the loads of all of them before any is looked at.
template <int PER, bool NARROW, bool TAIL, class At>
__device__ __forceinline__ void load_pieces(Raw8 (&raw)[PER], const void* p, int64_t row, int type, int n, At at) {
  auto all = [&](auto t) {
#pragma unroll
    for (int i = 0; i < PER; ++i) load8<decltype(t)::value, TAIL>(raw[i], p, row + min(at(i), n - 1), n - at(i));
  };
  if (!NARROW && type == kF32) all(std::integral_constant<int, kF32>{});
  else all(std::integral_constant<int, kF16>{});           // 16-bit types load alike
}

}  // namespace

// A row is a workgroup's, in registers from its one read to its one write, as bits of the type that it is stored in: piece c of eight
// values to thread c % THREADS, PER pieces to a thread, so that 16 neighbouring lanes hold 128 neighbouring values. NARROW: x, residual
// and weight are of 16 bits. TAIL: rows end inside a piece.
template <int THREADS, int PER, bool NARROW, bool TAIL>
__global__ __launch_bounds__(THREADS) void rms_norm_kernel(const NormArgs a) {
  __shared__ double sums[THREADS / 64];
  __shared__ uint32_t words[THREADS / 64];
  const int row = blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.rows) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto at = [&](int i) { return 8 * ((int)threadIdx.x + THREADS * i); };   // first value of the thread's piece i
  Raw8 hr[PER], rr[PER], wr[PER];
  load_pieces<PER, NARROW, TAIL>(hr, a.x, (int64_t)row * a.ldx, a.x_type, a.n, at);
  if (a.residual) load_pieces<PER, NARROW, TAIL>(rr, a.residual, (int64_t)row * a.ldr, a.r_type, a.n, at);
  load_pieces<PER, NARROW, TAIL>(wr, a.w, 0, a.w_type, a.n, at);

  // Eight squares are summed in binary32, which eight roundings leave off by 8 * 2^-24 of their sum at most, and those sums in binary64;
  // where squares may leave binary32's range, all in binary64.
  const int h_type = a.residual ? a.r_type : a.x_type;
  double sum = 0.0;
  uint32_t top = 0;                              // int8: bits of the largest product, rounded to binary32
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    float h[8];
    widen(hr[i], a.x_type, h);
    if (a.residual) {
      float r[8];
      widen(rr[i], a.r_type, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] += r[e];
      narrow<NARROW>(h, a.r_type, hr[i]);
      if (at(i) < a.n) store8<NARROW, TAIL>(hr[i], a.r_type, a.total, (int64_t)row * a.ldt + at(i), a.n - at(i));
      widen(hr[i], a.r_type, h);
    }
    float part = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) part = fmaf(h[e], h[e], part);
    if (part >= 0x1p-90f && part <= 0x1p100f) {
      sum += (double)part;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fma((double)h[e], (double)h[e], sum);
    }
    if (a.out == kInt8) {
      float w[8];
      widen(wr[i], a.w_type, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __builtin_bit_cast(uint32_t, h[e] * w[e]) & 0x7FFFFFFFu);
    }
  }
  if (a.out == kInt8) {
    top = row16_max(top);
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
  }
  sum = wave_sum(sum);
  if constexpr (THREADS > 64) {
    if (lane == 0) {
      sums[wave] = sum;
      words[wave] = top;
    }
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int v = 0; v < THREADS / 64; ++v) {
      sum += sums[v];
      top = max(top, words[v]);
    }
  }
  const bool finite = sum < __builtin_inf();     // a square of finite binary32 values is far from the end of binary64
  const double mean = sum / (double)a.n + (double)a.eps;
  const double root = sqrt(mean);
  const double r = !finite ? __builtin_nan("") : mean > 0.0 ? 1.0 / root : 0.0;

  // int8: the row's largest product. It is what binary32 says of products of 16-bit values in its range; of wider ones, it is the
  // largest of those that are rounded to what binary32 says; out of its range, the largest of all in binary64 (every thread alike).
  double most = 0.0, inv = 0.0;
  bool good = finite, plain = false;
  if (a.out == kInt8) {
    plain = top >= 0x0D800000u && top <= 0x71800000u;   // 2^-100 to 2^100
    most = (double)__builtin_bit_cast(float, top);
    if (!NARROW || !plain) {
      most = 0.0;
      uint32_t word = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        float h[8], w[8];
        widen(hr[i], h_type, h);
        widen(wr[i], a.w_type, w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!plain || (__builtin_bit_cast(uint32_t, h[e] * w[e]) & 0x7FFFFFFFu) == top) {
            const double p = (double)h[e] * (double)w[e];
            most = fmax(most, fabs(p));
            word = max(word, magnitude_word(p));
          }
      }
      if (word >= kNotFinite) most = __builtin_inf();
      most = wave_max(most);
      if constexpr (THREADS > 64) {
        __syncthreads();                         // every thread has read the sums
        if (lane == 0) sums[wave] = most;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < THREADS / 64; ++v) most = fmax(most, sums[v]);
      }
    }
    good = finite && most < __builtin_inf();
    inv = good && most > 0.0 ? 127.0 / most : 0.0;
    if (threadIdx.x == 0) a.scales[(int64_t)row * a.lds] = good ? (float)(most * r / 127.0) : __builtin_nanf("");
  }
  const float inv32 = (float)inv;
  const double step = r / (double)kE4m3Max;
  const float r32 = (float)r;
  // Where every h r32 is zero or a normal number, y is formed in binary32; else in binary64, as a large weight may bring back what a
  // subnormal one loses. `least`: bits of the smallest such |h|, less one.
  const bool in_range = r >= 0x1p-120 && r <= 0x1p120;
  const uint32_t least = max(__builtin_bit_cast(uint32_t, (float)(0x1p-125 * root)), 1u) - 1u;

#pragma unroll
  for (int i = 0; i < PER; ++i) {
    float h[8], w[8];
    widen(hr[i], h_type, h);
    widen(wr[i], a.w_type, w);
    const int valid = a.n - at(i);
    const int64_t to = (int64_t)row * a.ldy + at(i);
    if (a.out == kE4m3) {
      float v[2][4];
      uint32_t bits = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e >> 2][e & 3] = h[e] * w[e];
        bits = max(bits, __builtin_bit_cast(uint32_t, v[e >> 2][e & 3]) & 0x7FFFFFFFu);
      }
      bits = row16_max(bits);
      const BlockFactors f = block_factors(__builtin_bit_cast(float, bits));
      double largest = (double)__builtin_bit_cast(float, bits);
      bool fine = finite && bits < 0x7F800000u;
      if (!NARROW || !f.plain) {                 // as for int8, in the 16 lanes of the block
        double top64 = 0.0;
        uint32_t word = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!f.plain || (__builtin_bit_cast(uint32_t, v[e >> 2][e & 3]) & 0x7FFFFFFFu) == bits) {
            const double p = (double)h[e] * (double)w[e];
            top64 = fmax(top64, fabs(p));
            word = max(word, magnitude_word(p));
          }
        largest = row16_max(top64);
        fine = finite && row16_max(word) < kNotFinite;
      }
      if (valid <= 0) break;
      if ((lane & 15) == 0) a.scales[(int64_t)row * a.lds + (at(i) >> 7)] = fine ? (float)(largest * step) : __builtin_nanf("");
      uint32_t b[2] = {0, 0};
      if (fine) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          double p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = (double)h[4 * k + e] * (double)w[4 * k + e];
          b[k] = e4m3_steps(v[k], p, f, largest);
        }
      }
      store_bytes<TAIL>(reinterpret_cast<uint8_t*>(a.y) + to, b, valid);
    } else if (a.out == kInt8) {
      if (valid <= 0) break;
      uint32_t b[2] = {0, 0};
      if (good) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float t = h[e] * w[e] * inv32, k = rintf(t);
          // t is off by 3 * 2^-24 of itself at most, less than 2^-15
          int q = (int)k;
          if (!plain || fabsf(fabsf(t - k) - 0.5f) <= 0x1p-14f) q = int8_step((double)h[e] * (double)w[e], inv, most);
          b[e >> 2] |= ((uint32_t)q & 255u) << (8 * (e & 3));
        }
      }
      store_bytes<TAIL>(reinterpret_cast<uint8_t*>(a.y) + to, b, valid);
    } else {
      if (valid <= 0) break;
      float y[8];
      uint32_t low = 0xFFFFFFFFu;                // zeros count as large
#pragma unroll
      for (int e = 0; e < 8; ++e) low = min(low, (__builtin_bit_cast(uint32_t, h[e]) & 0x7FFFFFFFu) - 1u);
      if (in_range && low >= least) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[e] * r32 * w[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = (float)((double)h[e] * (double)w[e] * r);
      }
      Raw8 bits;
      narrow<false>(y, a.out, bits);
      store8<false, TAIL>(bits, a.out, a.y, to, valid);
    }
  }
}

template <bool NARROW, bool TAIL>
static void launch_norm(const NormArgs& a, hipStream_t s) {
  const int pieces = (a.n + 7) / 8;
  const unsigned x = a.rows < 65536 ? (unsigned)a.rows : 65536u;
  const dim3 grid(x, ((unsigned)a.rows + x - 1) / x);
  // A row is a wave's up to 1024 values. Longer ones: of many rows, the fewest threads that hold it (4096 x 10240 bf16 with a residual,
  // into e4m3: 256 threads 69.7 us, 512 72.3, 1024 93.8; 2000 x 15000 fp32 with a bf16 residual, into int8: 115, 78 and 98); of few, as
  // many as there are pieces (1 x 16384: 11.1, 7.5 and 6.5).
  const bool many = a.rows >= 512;
  if (pieces <= 64) hipLaunchKernelGGL((rms_norm_kernel<64, 1, NARROW, TAIL>), grid, dim3(64), 0, s, a);
  else if (pieces <= 128) hipLaunchKernelGGL((rms_norm_kernel<64, 2, NARROW, TAIL>), grid, dim3(64), 0, s, a);
  else if (pieces <= 256) hipLaunchKernelGGL((rms_norm_kernel<256, 1, NARROW, TAIL>), grid, dim3(256), 0, s, a);
  else if (pieces <= 512 && many) hipLaunchKernelGGL((rms_norm_kernel<256, 2, NARROW, TAIL>), grid, dim3(256), 0, s, a);
  else if (pieces <= 768 && many) hipLaunchKernelGGL((rms_norm_kernel<256, 3, NARROW, TAIL>), grid, dim3(256), 0, s, a);
  else if (pieces <= 1024 && many) hipLaunchKernelGGL((rms_norm_kernel<256, 4, NARROW, TAIL>), grid, dim3(256), 0, s, a);
  else if (pieces <= 1024) hipLaunchKernelGGL((rms_norm_kernel<1024, 1, NARROW, TAIL>), grid, dim3(1024), 0, s, a);
  else if (pieces <= 1280 && many) hipLaunchKernelGGL((rms_norm_kernel<256, 5, NARROW, TAIL>), grid, dim3(256), 0, s, a);
  else if (pieces <= 1536 && many) hipLaunchKernelGGL((rms_norm_kernel<512, 3, NARROW, TAIL>), grid, dim3(512), 0, s, a);
  else if (pieces <= 2048 && many) hipLaunchKernelGGL((rms_norm_kernel<512, 4, NARROW, TAIL>), grid, dim3(512), 0, s, a);
  else if (pieces <= 2048) hipLaunchKernelGGL((rms_norm_kernel<1024, 2, NARROW, TAIL>), grid, dim3(1024), 0, s, a);
  else if (pieces <= 3 * 1024) hipLaunchKernelGGL((rms_norm_kernel<1024, 3, NARROW, TAIL>), grid, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((rms_norm_kernel<1024, 4, NARROW, TAIL>), grid, dim3(1024), 0, s, a);
}

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  const bool narrow = a.x_type != kF32 && a.w_type != kF32 && (!a.residual || a.r_type != kF32), tail = a.n % 8 != 0;
  if (narrow) tail ? launch_norm<true, true>(a, s) : launch_norm<true, false>(a, s);
  else tail ? launch_norm<false, true>(a, s) : launch_norm<false, false>(a, s);
  return hipGetLastError();
}

}  // namespace tg

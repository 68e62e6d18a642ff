// Steps of 8-bit rows from values held in binary64, each the nearest one to the true quotient (fp8_quantize.hip, rms_norm.hip).
#pragma once

#include "tg_device.hpp"
#include "tg_internal.hpp"

namespace tg {

// Eight neighbouring values of a row as they lie in memory: 16-bit types fill `a`.
struct Raw8 {
  u32x4 a, b;
};

// The first `valid` of eight values from element `at` on (at any address of the type), zeros behind them. TAIL: a row may end inside
// eight; else `valid` is 8 or more, or none, and the code for its end is not there (which costs 40 instructions a piece).
template <int DT, bool TAIL>
__device__ __forceinline__ void load8(Raw8& r, const void* p, int64_t at, int valid) {
  r.a = r.b = u32x4{0, 0, 0, 0};
  if constexpr (DT == kF32) {
    const float* f = reinterpret_cast<const float*>(p) + at;
    if (TAIL ? valid >= 8 : valid > 0) {
      r.a = *reinterpret_cast<const u32x4_any*>(f);
      r.b = *reinterpret_cast<const u32x4_any*>(f + 4);
    } else if constexpr (TAIL) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < valid) r.a[i] = __builtin_bit_cast(uint32_t, f[i]);
        if (i + 4 < valid) r.b[i] = __builtin_bit_cast(uint32_t, f[i + 4]);
      }
    }
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p) + at;
    if (TAIL ? valid >= 8 : valid > 0) {
      r.a = *reinterpret_cast<const u32x4_any*>(h);
    } else if constexpr (TAIL) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid) r.a[i >> 1] |= (uint32_t)h[i] << (16 * (i & 1));
    }
  }
}

// The first `valid` (more than none) of eight bytes.
template <bool TAIL>
__device__ __forceinline__ void store_bytes(uint8_t* q, const uint32_t (&w)[2], int valid) {
  if (!TAIL || valid >= 8) {
    *reinterpret_cast<u32x2_any*>(q) = u32x2_any{w[0], w[1]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) q[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

template <int DT>
__device__ __forceinline__ void widen8(const Raw8& r, float (&v)[8]) {
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __builtin_bit_cast(float, (uint32_t)r.a[i]);
      v[i + 4] = __builtin_bit_cast(float, (uint32_t)r.b[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = r.a[i >> 1];
      if constexpr (DT == kF16) v[i] = half_bits_to_float((uint16_t)(w >> (16 * (i & 1))));
      else v[i] = __builtin_bit_cast(float, i & 1 ? w & 0xFFFF0000u : w << 16);
    }
  }
}

// Largest value over the 16 lanes of a row of the wave, in every one of them.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));   // row_ror 8, 4, 2, 1
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false));
}

template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double row16_max(double v) {
  v = fmax(v, dpp64<0x128>(v));
  v = fmax(v, dpp64<0x124>(v));
  v = fmax(v, dpp64<0x122>(v));
  return fmax(v, dpp64<0x121>(v));
}

// The high word of |v|: 0x7FF00000 and above for an infinity or a NaN, which a maximum of values would lose.
__device__ __forceinline__ uint32_t magnitude_word(double v) {
  return (uint32_t)(__builtin_bit_cast(uint64_t, v) >> 32) & 0x7FFFFFFFu;
}
constexpr uint32_t kNotFinite = 0x7FF00000u;

constexpr float kE4m3Max = 448.f;

// The e4m3 code of p where it lies next to the border of the magnitudes `low` and `low + 1`: 448 |p| / amax against the
// border, multiplied out. Both sides are exact: p and amax have 48 significant bits at most (products of two binary32), 896
// has three and twice the border five.
__device__ __forceinline__ uint32_t e4m3_at_border(uint32_t low, uint32_t sign, double p, double amax) {
  const double twice = (double)__builtin_amdgcn_cvt_f32_fp8((int)low, 0) + (double)__builtin_amdgcn_cvt_f32_fp8((int)low + 1, 0);
  const double a = 2.0 * kE4m3Max * fabs(p), b = twice * amax;
  return sign | (a > b || (a == b && (low & 1)) ? low + 1 : low);
}

// Four e4m3 steps from quotients below and above the true ones: where both round to one step, that is the step; else it is
// decided exactly (about one value in 30000 of random ones). at(i): the value and its amax.
template <class At>
__device__ __forceinline__ uint32_t e4m3_between(const float (&below)[4], const float (&above)[4], At at) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(below[0], below[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(below[2], below[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(above[0], above[1], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(above[2], above[3], hi, true);
  uint32_t q = (uint32_t)hi;
  if (lo != hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t l = (uint32_t)lo >> (8 * i) & 255u, h = (uint32_t)hi >> (8 * i) & 255u;
      if (l != h) q = (q & ~(255u << (8 * i))) | at(i, l & 127u, h & 128u) << (8 * i);
    }
  }
  return q;
}

// The factors that bring a block's values to e4m3 quotients a little below and above the true ones, from its largest magnitude as a
// binary32 (rounded once). v_rcp_f32 is off by 2^-23 of itself at most; the value, the magnitude, 448 times the reciprocal, the
// factor and the quotient are rounded by 2^-24 each: 7 * 2^-24 together, less than half of kNear.
constexpr float kNear = 0x1p-20f;
struct BlockFactors {
  float below, above;
  bool plain;                                    // amax is far from the ends of binary32; else the quotients are formed in binary64
};
__device__ __forceinline__ BlockFactors block_factors(float amax) {
  BlockFactors f;
  f.plain = amax >= 0x1p-100f && amax <= 0x1p100f;
  const float inv = kE4m3Max * __builtin_amdgcn_rcpf(amax);
  f.below = inv * (1.f - kNear);
  f.above = inv * (1.f + kNear);
  return f;
}

// Four steps of values p (or of p rounded once, v) in a block of largest magnitude amax.
__device__ __forceinline__ uint32_t e4m3_steps(const float (&v)[4], const double (&p)[4], const BlockFactors& f, double amax) {
  float below[4], above[4];
  if (f.plain) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      below[i] = v[i] * f.below;
      above[i] = v[i] * f.above;
    }
  } else {
    const double inv = amax > 0.0 ? (double)kE4m3Max / amax : 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float t = (float)(p[i] * inv);
      below[i] = t * (1.f - kNear);
      above[i] = t * (1.f + kNear);
    }
  }
  return e4m3_between(below, above, [&](int i, uint32_t low, uint32_t sign) { return e4m3_at_border(low, sign, p[i], amax); });
}

}  // namespace tg

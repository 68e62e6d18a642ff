// Routing of tokens to experts: scores, groups, the top_k ids with their weights (moe_route), and the routed pairs in
// expert order (moe_group).
//
// An id is decided by comparing scores, so scores, keys and group values are formed in binary64 and equal ones go to
// the lowest index; a weight is rounded to binary32 once.
#include "tg_device.hpp"
#include "tg_internal.hpp"

namespace tg {

namespace {

constexpr double kNone = -__builtin_huge_val();   // the key of an expert that is not available

// Lane 63's value after six steps: the maximum over the wave.
__device__ __forceinline__ float wave_max_f32(float v) {
#define TG_STEP(ctrl)                                                                                              \
  v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, v), __builtin_bit_cast(int, v), \
                                                                     ctrl, 0xF, 0xF, false)));
  TG_STEP(0x111) TG_STEP(0x112) TG_STEP(0x114) TG_STEP(0x118)   // row_shr 1, 2, 4, 8
  TG_STEP(0x142) TG_STEP(0x143)                                 // row_bcast 15, 31
#undef TG_STEP
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane), hi = __builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double wave_sum(double v) {
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// What the lanes of a wave wrote to LDS is seen by its other lanes.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int DT>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
  if constexpr (DT == kF32) return reinterpret_cast<const float*>(p)[i];
  const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
  if constexpr (DT == kF16) return half_bits_to_float(b);
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}

constexpr int kRouteWaves = 4;   // tokens of a workgroup where there are many

}  // namespace

// One wave per token; lane l holds the V neighbouring experts l V .. l V + V - 1, so that the order of lanes is the
// order of experts.
template <int V, int DT>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(const RouteArgs a) {
  __shared__ double ranked_sh[kRouteWaves][V * 64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int token = blockIdx.x * (blockDim.x >> 6) + wave;
  if (token >= a.tokens) return;
  const float inf = __builtin_huge_valf();
  float l[V], bias[V];
  const int64_t at0 = (int64_t)token * a.ld;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    l[i] = e < a.experts ? logit<DT>(a.logits, at0 + e) : -inf;
    bias[i] = a.bias && e < a.experts ? a.bias[e] : 0.f;
  }
  float most = -inf;
  bool poison = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    poison |= l[i] != l[i] || !(bias[i] < inf) ;
    most = fmaxf(most, l[i]);
  }
  double score[V], key[V];
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) score[i] = 1.0 / (1.0 + exp(-(double)l[i]));
  } else {
    most = wave_max_f32(most);
    poison |= most == inf;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      score[i] = l[i] == -inf ? 0.0 : exp((double)l[i] - (double)most);
      sum += score[i];
    }
    sum = 1.0 / wave_sum(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) score[i] *= sum;
  }
  if (__ballot(poison)) {   // a NaN, or an infinity that leaves no order: the first top_k ids, with weights that say so
    if (lane < a.top_k) {
      a.sel[(int64_t)token * a.top_k + lane] = lane;
      a.weights[(int64_t)token * a.top_k + lane] = __builtin_nanf("");
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = l[i] == -inf || bias[i] == -inf ? kNone : score[i] + (double)bias[i];
  if (a.n_group > 1) {
    // A group's two largest keys. Where a lane's experts lie in one group, each lane leaves its own two largest, and
    // lane g goes over its group's lanes; else over its group's experts.
    const int size = a.experts / a.n_group;
    double* mine = ranked_sh[wave];
    double first = kNone, second = kNone;
    auto take = [&](double v) {
      const double low = fmin(first, v);
      first = fmax(first, v);
      second = fmax(second, low);
    };
    if (V > 1 && size % V == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) take(key[i]);
      mine[2 * lane] = first;
      mine[2 * lane + 1] = second;
      wave_lds_fence();
      first = second = kNone;
      if (lane < a.n_group)
        for (int i = 0; i < size / V; ++i) {
          take(mine[2 * (lane * (size / V) + i)]);
          take(mine[2 * (lane * (size / V) + i) + 1]);
        }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) mine[lane * V + i] = key[i];
      wave_lds_fence();
      if (lane < a.n_group)
        for (int i = 0; i < size; ++i) take(mine[lane * size + i]);
    }
    const double value = a.group_top == 2 && second != kNone ? first + second : first;
    int before = 0;
    for (int i = 0; i < a.n_group; ++i) {
      const double v = lane_value(value, i);
      before += v > value || (v == value && i < lane) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < a.n_group && before < a.topk_group);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (e < a.experts && !((kept >> (e / size)) & 1)) key[i] = kNone;
    }
  }
  if (!a.bias) {            // the same order as the scores', without their rounding
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = key[i] == kNone ? kNone : (double)l[i];
  }
  // top_k rounds: each lane's largest key, and the wave's by its binary32 rounding, which keeps the order; only where
  // several lanes share the largest rounding are their keys compared in full.
  int my_id = -1;           // lane i keeps slot i
  double my_w = 0.0;
  for (int s = 0; s < a.top_k; ++s) {
    double best = key[0], w = score[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
        w = score[i];
      }
    const float near = (float)best;
    const float top = wave_max_f32(near);
    if (top == -inf) break;   // no expert is left: the other slots stay -1 with weight 0
    uint64_t mask = __ballot(near == top);
    int owner = __builtin_ctzll(mask);
    mask &= mask - 1;
    if (mask) {
      double most_key = lane_value(best, owner);
      while (mask) {
        const int o = __builtin_ctzll(mask);
        mask &= mask - 1;
        const double k = lane_value(best, o);
        if (k > most_key) {
          most_key = k;
          owner = o;
        }
      }
    }
    const int id = owner * V + __builtin_amdgcn_readlane(at, owner);
    const double sw = lane_value(w, owner);
    if (lane == s) {
      my_id = id;
      my_w = sw;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane == owner && i == at) key[i] = kNone;
  }
  if (a.renorm) {
    const double total = wave_sum(my_w);
    my_w = total > 0.0 ? my_w / total : 0.0;
  }
  if (lane < a.top_k) {
    a.sel[(int64_t)token * a.top_k + lane] = my_id;
    a.weights[(int64_t)token * a.top_k + lane] = (float)(my_w * (double)a.scale);
  }
}

template <int DT>
static hipError_t launch_route_t(const RouteArgs& a, hipStream_t s) {
  const int waves = a.tokens >= 1024 ? kRouteWaves : 1;
  const dim3 grid((unsigned)((a.tokens + waves - 1) / waves)), block(64 * waves);
  if (a.experts <= 64) hipLaunchKernelGGL((route_kernel<1, DT>), grid, block, 0, s, a);
  else if (a.experts <= 128) hipLaunchKernelGGL((route_kernel<2, DT>), grid, block, 0, s, a);
  else if (a.experts <= 256) hipLaunchKernelGGL((route_kernel<4, DT>), grid, block, 0, s, a);
  else if (a.experts <= 512) hipLaunchKernelGGL((route_kernel<8, DT>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((route_kernel<16, DT>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_moe_route(const RouteArgs& a, int dtype, hipStream_t s) {
  if (dtype == kF32) return launch_route_t<kF32>(a, s);
  if (dtype == kF16) return launch_route_t<kF16>(a, s);
  return launch_route_t<kBf16>(a, s);
}

// ---------------------------------------------------------------------------
// Pairs in expert order, stable, in one launch without a workspace: workgroup e (e == experts: the pairs without an
// expert) reads all ids, counts those before its own and writes its own pairs behind them. Its 16 waves take
// neighbouring stretches, a lane four neighbouring ids at a time, so the order of the pairs is the order of waves,
// steps, lanes and ids.
// ---------------------------------------------------------------------------
constexpr int kGroupSteps = 32;   // steps of 256 ids whose hits a wave keeps: 16 * 32 * 256 = 2^17 pairs

template <bool KEEP>
__global__ __launch_bounds__(1024) void group_kernel(const int32_t* __restrict__ sel, int pairs, int experts, int wide,
                                                     int32_t* __restrict__ offsets, int32_t* __restrict__ order) {
  __shared__ int less_sh[16], same_sh[16];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const uint32_t mine = blockIdx.x;
  const int steps = (pairs + 4095) >> 12;                       // of 256 ids, per wave
  const int begin = wave * steps * 256 + lane * 4;
  auto load = [&](int step, uint32_t(&id)[4]) {                 // ids past the end: beyond every expert
    const int p = begin + step * 256;
    if (wide && p + 4 <= pairs) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(sel + p);
#pragma unroll
      for (int c = 0; c < 4; ++c) id[c] = min(v[c], (uint32_t)experts);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) id[c] = p + c < pairs ? min((uint32_t)sel[p + c], (uint32_t)experts) : 0xFFFFFFFFu;
    }
  };
  uint32_t kept[kGroupSteps / 8] = {};                          // four bits per step: this lane's hits
  int less = 0, same = 0;                                       // of the wave
  auto count = [&](const uint32_t(&id)[4]) {
    uint32_t hits = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      less += __popcll(__ballot(id[c] < mine));
      hits |= id[c] == mine ? 1u << c : 0u;
    }
    return hits;
  };
  if constexpr (KEEP) {
#pragma unroll
    for (int b = 0; b < kGroupSteps / 8; ++b) {
      if (8 * b >= steps) break;
      if (wide && 8 * b + 8 <= steps && wave * steps * 256 + (8 * b + 8) * 256 <= pairs) {
        u32x4 v[8];                                             // eight loads in flight
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const u32x4*>(sel + begin + (8 * b + i) * 256);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t id[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) id[c] = min(v[i][c], (uint32_t)experts);
          kept[b] |= count(id) << (4 * i);
        }
      } else {
        for (int i = 0; i < 8 && 8 * b + i < steps; ++i) {
          uint32_t id[4];
          load(8 * b + i, id);
          kept[b] |= count(id) << (4 * i);
        }
      }
      same += __popc(kept[b]);
    }
  } else {
    for (int i = 0; i < steps; ++i) {
      uint32_t id[4];
      load(i, id);
      same += __popc(count(id));
    }
  }
  same = __builtin_amdgcn_readlane(wave_scan(same), 63);
  if (lane == 0) {
    less_sh[wave] = less;
    same_sh[wave] = same;
  }
  __syncthreads();
  int base = 0, at = 0;
  for (int w = 0; w < 16; ++w) {
    base += less_sh[w];
    if (w < wave) at += same_sh[w];
  }
  if (threadIdx.x == 0) offsets[mine] = base;                   // offsets[experts]: the pairs with an expert
  if (same == 0) return;
  at += base;
  auto put = [&](int step, uint32_t hits, int to) {             // this lane's hits of a step
    while (hits) {
      order[to++] = begin + step * 256 + __builtin_ctz(hits);
      hits &= hits - 1;
    }
  };
  if constexpr (KEEP) {
#pragma unroll
    for (int b = 0; b < kGroupSteps / 8; ++b) {
      if (8 * b >= steps || __ballot(kept[b] != 0) == 0) continue;
      // The lanes' hits of eight steps, summed over the lanes at once: ten bits hold the at most 256 hits of a step.
      int mine3[3], upto[3], total[3];
#pragma unroll
      for (int d = 0; d < 3; ++d) {
        mine3[d] = 0;
#pragma unroll
        for (int i = 0; i < 3 && 3 * d + i < 8; ++i) mine3[d] |= __popc((kept[b] >> (4 * (3 * d + i))) & 15u) << (10 * i);
        upto[d] = wave_scan(mine3[d]);
        total[d] = __builtin_amdgcn_readlane(upto[d], 63);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = i / 3, sh = 10 * (i % 3);
        put(8 * b + i, (kept[b] >> (4 * i)) & 15u, at + (((upto[d] - mine3[d]) >> sh) & 1023));
        at += (total[d] >> sh) & 1023;
      }
    }
  } else {
    for (int i = 0; i < steps; ++i) {
      uint32_t id[4];
      load(i, id);
      uint32_t hits = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) hits |= id[c] == mine ? 1u << c : 0u;
      const int n = __popc(hits), upto = wave_scan(n);
      put(i, hits, at + upto - n);
      at += __builtin_amdgcn_readlane(upto, 63);
    }
  }
}

hipError_t launch_moe_group(int pairs, int experts, const int32_t* sel, int32_t* offsets, int32_t* order, hipStream_t s) {
  const int wide = (uintptr_t)sel % 16 == 0;
  const dim3 grid((unsigned)experts + 1), block(1024);
  if (pairs <= 4096 * kGroupSteps) hipLaunchKernelGGL(group_kernel<true>, grid, block, 0, s, sel, pairs, experts, wide, offsets, order);
  else hipLaunchKernelGGL(group_kernel<false>, grid, block, 0, s, sel, pairs, experts, wide, offsets, order);
  return hipGetLastError();
}

}  // namespace tg

// Routing of tokens to experts: scores, groups, the top_k ids with their weights (moe_route), and the routed pairs in
// expert order (moe_group).
//
// An id is decided by comparing scores: the ids are those of binary64 scores, keys and group values, equal ones in
// the order of the experts; a weight is formed in binary64 and rounded to binary32 once.
#include <type_traits>

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

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#define TG_STEP(ctrl) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xF, 0xF, true));
  TG_STEP(0x111) TG_STEP(0x112) TG_STEP(0x114) TG_STEP(0x118) TG_STEP(0x142) TG_STEP(0x143)
#undef TG_STEP
  return __builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_sum_f32(float v) {
#define TG_STEP(ctrl, rows)                                                                                        \
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, rows, 0xF, false));
  TG_STEP(0x111, 0xF) TG_STEP(0x112, 0xF) TG_STEP(0x114, 0xF) TG_STEP(0x118, 0xF) TG_STEP(0x142, 0xA) TG_STEP(0x143, 0xC)
#undef TG_STEP
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

template <int DT>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
  if constexpr (DT == kF32) return reinterpret_cast<const float*>(p)[i];
  const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
  if constexpr (DT == kF16) return half_bits_to_float(b);
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}

// V neighbouring values, up to 16 bytes at once.
template <int V, int DT>
__device__ __forceinline__ void load_neighbours(const void* p, int64_t at, float (&f)[V]) {
  constexpr int kBytes = V * (DT == kF32 ? 4 : 2), kWords = kBytes >= 16 ? 4 : kBytes / 4;
  if constexpr (kWords == 0) {
    f[0] = logit<DT>(p, at);
  } else {
    constexpr int kEach = kWords * (DT == kF32 ? 1 : 2);    // values of one load
#pragma unroll
    for (int d = 0; d < V / kEach; ++d) {
      const char* from = reinterpret_cast<const char*>(p) + (at + d * kEach) * (DT == kF32 ? 4 : 2);
      uint32_t w[4];
      if constexpr (kWords == 4) {
        const u32x4_any v = *reinterpret_cast<const u32x4_any*>(from);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = v[i];
      } else if constexpr (kWords == 2) {
        const u32x2_any v = *reinterpret_cast<const u32x2_any*>(from);
        w[0] = v[0];
        w[1] = v[1];
      } else {
        w[0] = *reinterpret_cast<const u32_any*>(from);
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const uint32_t word = w[DT == kF32 ? i : i / 2];
        if constexpr (DT == kF32) f[d * kEach + i] = __builtin_bit_cast(float, word);
        else if constexpr (DT == kF16) f[d * kEach + i] = half_bits_to_float((uint16_t)(word >> (16 * (i & 1))));
        else f[d * kEach + i] = __builtin_bit_cast(float, i & 1 ? word & 0xFFFF0000u : word << 16);
      }
    }
  }
}

// Numbers as words of the same order; none is 0.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f + 0.0f);   // -0 and +0 are equal
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t w) {
  return __builtin_bit_cast(float, w & 0x80000000u ? w ^ 0x80000000u : ~w);
}

// The two largest of what it takes; T's least value stands for "none".
template <class T>
struct Best2 {
  T first, second;
  __device__ __forceinline__ explicit Best2(T none) : first(none), second(none) {}
  __device__ __forceinline__ static T larger(T a, T b) { return a > b ? a : b; }
  __device__ __forceinline__ static T smaller(T a, T b) { return a > b ? b : a; }
  __device__ __forceinline__ void take(T v) {
    second = larger(second, smaller(first, v));
    first = larger(first, v);
  }
  __device__ __forceinline__ void take(T f, T s) {           // another's two
    second = larger(larger(second, s), smaller(first, f));
    first = larger(first, f);
  }
};

__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane), hi = __builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double wave_sum(double v) {
  double lane63 = v;
#define TG_STEP(ctrl, rows)                                                                                        \
  {                                                                                                                \
    const uint64_t b = __builtin_bit_cast(uint64_t, lane63);                                                       \
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, ctrl, rows, 0xF, false);                  \
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), ctrl, rows, 0xF, false);                    \
    lane63 += __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);                                                 \
  }
  TG_STEP(0x111, 0xF) TG_STEP(0x112, 0xF) TG_STEP(0x114, 0xF) TG_STEP(0x118, 0xF) TG_STEP(0x142, 0xA) TG_STEP(0x143, 0xC)
#undef TG_STEP
  return lane_value(lane63, 63);
}

// What the lanes of a wave wrote to LDS is seen by its other lanes.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

constexpr int kRouteWaves = 4;   // tokens of a workgroup where there are many

}  // namespace

// The two largest keys of group g in lane g, from every expert's. Where a lane's experts lie in one group, each lane
// leaves its own two largest and lane g goes over its group's lanes; else over its group's experts.
template <int V, class T>
__device__ __forceinline__ Best2<T> group_best(const T (&key)[V], T none, T* mine, int lane, int size, int n_group) {
  Best2<T> best(none);
  if (V > 1 && size % V == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) best.take(key[i]);
    mine[2 * lane] = best.first;
    mine[2 * lane + 1] = best.second;
    wave_lds_fence();
    best = Best2<T>(none);
    if (lane < n_group)
      for (int i = 0; i < size / V; ++i)
        best.take(mine[2 * (lane * (size / V) + i)], mine[2 * (lane * (size / V) + i) + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) mine[lane * V + i] = key[i];
    wave_lds_fence();
    if (lane < n_group)
      for (int i = 0; i < size; ++i) best.take(mine[lane * size + i]);
  }
  wave_lds_fence();                                         // before the place is written again
  return best;
}

// One wave per token; lane l holds the V neighbouring experts l V .. l V + V - 1, so that the order of lanes is the
// order of experts.
//
// The ids are those of binary64 scores, but few comparisons need them: without a bias the keys are the logits themselves,
// and with one the scores are formed in binary32, off by less than 2^-19 (exp and 1/x of the hardware, a unit in the last
// place each, of an argument rounded once: s (1 - s) |l| < 1/4 bounds what that costs a sigmoid, p |ln p| < 0.4 a
// softmax; its sum of up to 22 terms in a row is off by less than 2^-19.5 relative). Keys further apart than two of these
// are in their binary64 order; where some of those found are not (about 2 tokens in 1000 of the 256-expert case
// measured), the experts found are put in order by their binary64 keys, which the lanes form anyway for the weights. A
// token whose groups are not clearly apart is done in binary64 throughout: of 256 experts in 8 groups with normal logits 2
// or 3 tokens in 10000 under a sigmoid; under a softmax, whose group values may all be small, 25 at a standard deviation
// of 1, 6 at 2, 190 at 6 and 700 at 8 (8192 tokens 12-14 us at 1 and 3, 14-15 at 6). Biases far larger than a score widen
// the border: a pair of 1e5 and -1e5 in one of two groups sends 9% of the tokens that way, of 1e8 all.
template <int V, int DT>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(const RouteArgs a) {
  __shared__ double place[kRouteWaves][V * 64 < 128 ? 128 : V * 64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int token = blockIdx.x * (blockDim.x >> 6) + wave;
  if (token >= a.tokens) return;
  const float inf = __builtin_huge_valf();
  float l[V], bias[V];
  const int64_t at0 = (int64_t)token * a.ld;
  if (a.experts % V == 0) { // a lane's experts are all there, or none
    const int e = min(lane * V, a.experts - V);
    load_neighbours<V, DT>(a.logits, at0 + e, l);
    if (a.bias) load_neighbours<V, kF32>(a.bias, e, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = lane * V < a.experts ? l[i] : -inf;
      bias[i] = a.bias && lane * V < a.experts ? bias[i] : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      l[i] = e < a.experts ? logit<DT>(a.logits, at0 + e) : -inf;
      bias[i] = a.bias && e < a.experts ? a.bias[e] : 0.f;
    }
  }
  float most = -inf;
  bool poison = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    poison |= l[i] != l[i] || !(bias[i] < inf);
    most = fmaxf(most, l[i]);
  }
  if (!a.sigmoid) {
    most = wave_max_f32(most);
    poison |= most == inf;
  }
  if (__ballot(poison)) {   // a NaN, or an infinity that leaves no order: the first top_k ids, with weights that say so
    if (lane < a.top_k) {
      a.sel[(int64_t)token * a.top_k + lane] = lane;
      a.weights[(int64_t)token * a.top_k + lane] = __builtin_nanf("");
    }
    return;
  }
  const int size = a.experts / a.n_group;
  auto there = [&](int i) { return l[i] != -inf && bias[i] != -inf; };
  // How many groups stand before a lane's by value, those of lower index among equal ones -> the kept ones as bits.
  auto keep = [&](auto value, int& before) {
    before = 0;
    for (int i = 0; i < a.n_group; ++i) {
      const auto v = lane_value(value, i);
      before += v > value || (v == value && i < lane) ? 1 : 0;
    }
    return __ballot(lane < a.n_group && before < a.topk_group);
  };
  const int inverse = ((1 << 20) + size - 1) / size;        // e / size = e * inverse >> 20 for e < 2^10, size <= 2^10
  const bool one_group = V == 1 || size % V == 0;           // a lane's experts lie in one group
  auto in_kept = [&](uint64_t kept, int i) { return (kept >> ((((lane * V + (one_group ? 0 : i)) * inverse) >> 20) & 63)) & 1; };

  int my_id = -1, found = 0;   // lane i keeps the i-th expert found
  bool sure = true, fuzzy = false;
  {
    uint32_t key[V];        // 0: not available
    if (!a.bias) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = there(i) ? ordered(l[i]) : 0u;
    }
    if (a.bias || a.n_group > 1) {
      constexpr float kLog2e = 1.44269504088896340736f;
      float score[V];
      if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) score[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * l[i]));
      } else {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          score[i] = __builtin_amdgcn_exp2f(kLog2e * (l[i] - most));
          sum += l[i] == -inf ? 0.f : score[i];
        }
        sum = __builtin_amdgcn_rcpf(wave_sum_f32(sum));
#pragma unroll
        for (int i = 0; i < V; ++i) score[i] *= sum;
      }
      uint32_t rank[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        rank[i] = there(i) ? ordered(score[i] + bias[i]) : 0u;
        if (a.bias) key[i] = rank[i];
      }
      if (a.n_group > 1) {
        const Best2<uint32_t> best = group_best<V, uint32_t>(rank, 0u, reinterpret_cast<uint32_t*>(place[wave]), lane, size, a.n_group);
        const bool none = best.first == 0;
        const float one = none ? -inf : unordered(best.first);
        const float two = a.group_top == 2 && best.second != 0 ? unordered(best.second) : 0.f;
        const float value = one + two;
        int before;
        const uint64_t kept = keep(value, before);
        if (a.topk_group < a.n_group) {
          // A value is off by less than its two scores' 2^-18, and each of its roundings (the two keys, their sum, this
          // bound) by 2^-24 of what the keys amount to, which may be far more than their sum. Keys that leave binary32
          // together say nothing of theirs.
          const float both = fabsf(one) + fabsf(two);
          if (__ballot(!none && !(both < 4.f)) == 0) {      // biases of a score's size: only the border is looked at
            const int last = __builtin_ctzll(__ballot(before == a.topk_group - 1));
            const int next = __builtin_ctzll(__ballot(before == a.topk_group));
            sure = !(lane_value(value, last) - lane_value(value, next) <= 2 * (0x1p-18f + 0x1p-20f));
          } else {
            const float off = both < inf ? 0x1p-18f + 0x1p-22f * both : inf, at = both < inf ? value : 0.f;
            const bool in = (kept >> lane) & 1;
            const float least = -wave_max_f32(in && !none ? off - at : -inf);       // of any kept group with experts
            const float most_left = wave_max_f32(!in && !none ? at + off : -inf);   // of any other
            sure = least > most_left;
          }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = in_kept(kept, i) ? key[i] : 0u;
      }
    }
    // A round: the wave's largest key, its first holder, one key less. Up to four experts a lane holds in falling order
    // (equal ones by index: only neighbours change places), so that its first is its largest.
    constexpr bool kSorted = V <= 4;
    uint32_t my_key = 0, order = 0;                         // order: the sorted experts' places in the lane, a byte each
    if constexpr (kSorted) {
      uint32_t at[V];
#pragma unroll
      for (int i = 0; i < V; ++i) at[i] = i;
#pragma unroll
      for (int n = 1; n < V; ++n)
#pragma unroll
        for (int i = n; i > 0; --i) {
          const bool swap = key[i] > key[i - 1];
          const uint32_t most_key = max(key[i], key[i - 1]), first = at[i - 1];
          key[i] = min(key[i], key[i - 1]);
          key[i - 1] = most_key;
          at[i - 1] = swap ? at[i] : first;
          at[i] = swap ? first : at[i];
        }
#pragma unroll
      for (int i = 0; i < V; ++i) order |= at[i] << (8 * i);
    }
    auto largest = [&]() {
      uint32_t m = key[0];
      if constexpr (!kSorted) {
#pragma unroll
        for (int i = 1; i < V; ++i) m = max(m, key[i]);
      }
      return wave_max_u32(m);
    };
    auto round = [&](uint32_t top) {
      int id;
      if constexpr (kSorted) {
        const int owner = __builtin_ctzll(__ballot(key[0] == top));
        id = owner * V + (__builtin_amdgcn_readlane((int)order, owner) & 255);
        const bool mine = lane == owner;
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = mine ? (i + 1 < V ? key[i + 1 < V ? i + 1 : i] : 0u) : key[i];
        order = mine ? order >> 8 : order;
      } else {
        bool hit[V], any = false;
        int first = lane * V;                               // this lane's first expert with that key
#pragma unroll
        for (int i = 0; i < V; ++i) {
          hit[i] = key[i] == top;
          any |= hit[i];
        }
#pragma unroll
        for (int i = V - 1; i >= 0; --i) first = hit[i] ? lane * V + i : first;
        const int owner = __builtin_ctzll(__ballot(any));
        id = __builtin_amdgcn_readlane(first, owner);
        bool open = lane == owner;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          key[i] = open && hit[i] ? 0u : key[i];
          open = open && !hit[i];
        }
      }
      my_id = lane == found ? id : my_id;
      my_key = lane == found ? top : my_key;
      ++found;
    };
    uint32_t top = 0;
    while (sure && found < a.top_k) {
      top = largest();
      if (top == 0) break;  // no expert is left: the other slots stay -1 with weight 0
      round(top);
    }
    if (a.bias && sure && found > 0) {
      // Rounds go on past the top_k-th until the next key is clearly smaller; two keys that are not clearly apart leave
      // the order to binary64.
      auto apart = [](float x, float y) { return x - y > 0x1p-18f + 0x1p-22f * fabsf(y); };
      uint32_t beyond = 0;
      for (;;) {
        beyond = found < a.top_k ? 0u : largest();
        if (beyond == 0 || apart(unordered(__builtin_amdgcn_readlane((int)my_key, found - 1)), unordered(beyond))) break;
        if (found == 64) {
          sure = false;     // more of them than lanes
          break;
        }
        round(beyond);
      }
      const uint32_t after = __shfl_down((int)my_key, 1, 64);
      fuzzy = __ballot(lane + 1 < found && !apart(unordered(my_key), unordered(after))) != 0;
    }
  }
  if (!sure) {              // in binary64 throughout
    double score[V], key[V];
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) score[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    } else {
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
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = there(i) ? score[i] + (double)bias[i] : kNone;
    uint64_t kept = ~0ull;
    if (a.n_group > 1) {
      int before;
      const Best2<double> best = group_best<V, double>(key, kNone, place[wave], lane, size, a.n_group);
      kept = keep(a.group_top == 2 && best.second != kNone ? best.first + best.second : best.first, before);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!a.bias && there(i)) key[i] = l[i];               // the scores' order, without their rounding
      if (a.n_group > 1 && !in_kept(kept, i)) key[i] = kNone;
    }
    my_id = -1;
    fuzzy = false;
    for (int s = 0; s < a.top_k; ++s) {
      double best = key[0];
      int at = 0;
#pragma unroll
      for (int i = 1; i < V; ++i)
        if (key[i] > best) {
          best = key[i];
          at = i;
        }
      const float near = (float)best;                       // keeps the order; equal ones are compared in full
      const float top = wave_max_f32(near);
      if (top == -inf) break;
      uint64_t mask = __ballot(near == top);
      int owner = __builtin_ctzll(mask);
      double most_key = lane_value(best, owner);
      for (mask &= mask - 1; mask; mask &= mask - 1) {
        const int o = __builtin_ctzll(mask);
        const double k = lane_value(best, o);
        if (k > most_key) {
          most_key = k;
          owner = o;
        }
      }
      const int id = owner * V + __builtin_amdgcn_readlane(at, owner);   // read with every lane active
      my_id = lane == s ? id : my_id;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane == owner && i == at) key[i] = kNone;
    }
  }
  double w = 0.0, total = 0.0;
  if (my_id >= 0) {
    const double ml = logit<DT>(a.logits, at0 + my_id);
    w = a.sigmoid ? 1.0 / (1.0 + exp(-ml)) : exp(ml - (double)most);
  }
  if (!a.sigmoid && (fuzzy || !a.renorm)) {
#pragma unroll
    for (int i = 0; i < V; ++i) total += l[i] == -inf ? 0.0 : exp((double)l[i] - (double)most);
    total = wave_sum(total);
    w = my_id >= 0 ? w / total : 0.0;
  }
  int slot = lane;
  if (fuzzy) {              // those found, by their binary64 keys
    const double key = my_id >= 0 ? w + (double)a.bias[my_id] : kNone;
    int before = 0;
    for (int i = 0; i < found; ++i) {
      const double k = lane_value(key, i);
      const int id = __builtin_amdgcn_readlane(my_id, i);
      before += k > key || (k == key && id < my_id) ? 1 : 0;
    }
    slot = lane < found ? before : lane;
  }
  if (a.renorm) {
    total = wave_sum(slot < a.top_k ? w : 0.0);
    w = total > 0.0 ? w / total : 0.0;
  }
  if (slot < a.top_k) {
    a.sel[(int64_t)token * a.top_k + slot] = my_id;
    a.weights[(int64_t)token * a.top_k + slot] = (float)(w * (double)a.scale);
  }
}

// Bound by instruction issue and the rounds' chain of dependent steps: 8192 tokens x 256 experts in 8 groups, top 8, take
// 11.4-12 us back to back (623 vector and 332 scalar instructions a token, of which how many it needs is not shown; each
// round that searches a lane's experts anew costs 0.6 us; 8.9 MB, 1.7 us of them), 65536 tokens 62 us, one token of 128
// experts 3.1 us. Four tokens share a workgroup where
// there are many; one each keeps a short batch spread over the card.
template <int DT>
static hipError_t launch_route_t(const RouteArgs& a, hipStream_t s) {
  const int waves = a.tokens >= 1024 ? kRouteWaves : 1;
  const dim3 grid((unsigned)((a.tokens + waves - 1) / waves)), block(64 * waves);
  const int v = a.experts <= 64 ? 1 : a.experts <= 128 ? 2 : a.experts <= 256 ? 4 : a.experts <= 512 ? 8 : 16;
  if (v == 1) hipLaunchKernelGGL((route_kernel<1, DT>), grid, block, 0, s, a);
  else if (v == 2) hipLaunchKernelGGL((route_kernel<2, DT>), grid, block, 0, s, a);
  else if (v == 4) hipLaunchKernelGGL((route_kernel<4, DT>), grid, block, 0, s, a);
  else if (v == 8) hipLaunchKernelGGL((route_kernel<8, DT>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((route_kernel<16, DT>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_moe_route(const RouteArgs& a, int dtype, hipStream_t s) {
  if (dtype == kF32) return launch_route_t<kF32>(a, s);
  if (dtype == kF16) return launch_route_t<kF16>(a, s);
  return launch_route_t<kBf16>(a, s);
}

// ---------------------------------------------------------------------------
// Pairs in expert order, stable, in one launch without a workspace: workgroup e reads all ids, counts those before its
// own and writes its own pairs behind them. Its 16 waves take neighbouring stretches, a lane four neighbouring ids at a
// time, so the order of the pairs is the order of waves, steps, lanes and ids.
//
// Every workgroup looks at every id, with three vector instructions and two scalar ones, and that bounds it: 131072 pairs
// of 256 experts take 10.0-11.2 us back to back (6 of them to read and count; 14.4 with the steps' hits placed one after
// another), 512 pairs of 128 experts 2.8-3.7 us, 2^18 pairs 24 us, 2^20 pairs 80-85 us for 1.6 us of bytes. A table of
// counts between workgroups would let each look at a part, for a workspace and a second launch of about 3 us: that would
// pay for long lists, from a number of pairs that has not been measured.
// ---------------------------------------------------------------------------
constexpr int kGroupBatches = 4;  // batches of 8 * 256 ids whose hits a wave keeps: 16 * 4 * 2048 = 2^17 pairs

// Four neighbouring ids of a lane: hits doubled four times, each time with whether that id is the workgroup's (NONE: is no
// expert's, >= mine) as the carry of the addition; COUNT: the wave's ids below `mine` are added to less. In one piece, as a
// carry is read two wait states after its comparison at the earliest and the compiler does not see into an addition
// written by hand: here three other instructions or more lie between.
#define TG_EACH(cmp, to)                                                                                             \
  cmp " %[" to "0], %[id0], %[mine]\n\t" cmp " %[" to "1], %[id1], %[mine]\n\t"                                         \
  cmp " %[" to "2], %[id2], %[mine]\n\t" cmp " %[" to "3], %[id3], %[mine]\n\t"
#define TG_PUSH(is) "v_addc_co_u32_e64 %[hits], vcc, %[hits], %[hits], %[" is "]\n\t"
#define TG_PUSHES TG_PUSH("is0") TG_PUSH("is1") TG_PUSH("is2") TG_PUSH("is3")
#define TG_OUT [hits] "+&v"(hits), [is0] "=&s"(is0), [is1] "=&s"(is1), [is2] "=&s"(is2), [is3] "=&s"(is3)
#define TG_LOW [low0] "=&s"(low0), [low1] "=&s"(low1), [low2] "=&s"(low2), [low3] "=&s"(low3)
#define TG_IN [id0] "v"(id[0]), [id1] "v"(id[1]), [id2] "v"(id[2]), [id3] "v"(id[3]), [mine] "s"(mine)
template <bool NONE, bool COUNT>
__device__ __forceinline__ void look_at_four(const u32x4& id, uint32_t mine, uint32_t& hits, int& less) {
  uint64_t is0, is1, is2, is3;
  if constexpr (COUNT) {
    uint64_t low0, low1, low2, low3;
    if constexpr (NONE)
      asm(TG_EACH("v_cmp_ge_u32_e64", "is") TG_EACH("v_cmp_lt_u32_e64", "low") TG_PUSHES : TG_OUT, TG_LOW : TG_IN : "vcc");
    else
      asm(TG_EACH("v_cmp_eq_u32_e64", "is") TG_EACH("v_cmp_lt_u32_e64", "low") TG_PUSHES : TG_OUT, TG_LOW : TG_IN : "vcc");
    less += __popcll(low0) + __popcll(low1) + __popcll(low2) + __popcll(low3);
  } else if constexpr (NONE) {
    asm(TG_EACH("v_cmp_ge_u32_e64", "is") TG_PUSHES : TG_OUT : TG_IN : "vcc");
  } else {
    asm(TG_EACH("v_cmp_eq_u32_e64", "is") TG_PUSHES : TG_OUT : TG_IN : "vcc");
  }
}
#undef TG_EACH
#undef TG_PUSH
#undef TG_PUSHES
#undef TG_OUT
#undef TG_LOW
#undef TG_IN

// The pairs of expert `mine` (NONE: mine == experts, those without one) -> their places, and where they end. KEEP: a
// wave's batches fit kGroupBatches; else they are looked at again for the writing.
template <bool KEEP, bool NONE>
__device__ __forceinline__ int group_pairs(const int32_t* __restrict__ sel, int pairs, int experts, uint32_t mine,
                                           int (&less_sh)[16], int (&same_sh)[16], int32_t* __restrict__ offsets,
                                           int32_t* __restrict__ order) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int steps = (pairs + 4095) >> 12, batches = (steps + 7) >> 3;   // of 256 ids and of 8 steps, per wave
  const int stretch = wave * steps * 256, begin = stretch + lane * 4;
  // Batch b of this lane: a bit for each of its 32 ids that is the workgroup's; the wave's ids before it are added to less.
  int less = 0;
  auto look = [&](int b, auto count) {
    uint32_t hits = 0;
    if (8 * b + 8 <= steps && stretch + (8 * b + 8) * 256 <= pairs) {
      u32x4 v[8];                                             // eight loads in flight
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const u32x4_any*>(sel + begin + (8 * b + i) * 256);
      // A hit is doubled into its place by the addition that adds it: the first of 32 ends on top.
#pragma unroll
      for (int i = 0; i < 8; ++i) look_at_four<NONE, decltype(count)::value>(v[i], mine, hits, less);
      return __brev(hits);
    }
    for (int i = 0; i < 8 && 8 * b + i < steps; ++i) {
      const int p = begin + (8 * b + i) * 256;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool there = p + c < pairs;
        const uint32_t id = there ? (uint32_t)sel[p + c] : 0u;
        less += __popcll(__ballot(there && id < mine));
        hits |= there && (NONE ? id >= mine : id == mine) ? 1u << (4 * i + c) : 0u;
      }
    }
    return hits;
  };
  uint32_t kept[kGroupBatches] = {};
  int same = 0;
  if constexpr (KEEP) {
#pragma unroll
    for (int b = 0; b < kGroupBatches; ++b) {
      if (b >= batches) break;
      int next = b;
      asm volatile("" : "+s"(next) : "v"(less));              // one batch's loads at a time: four would not fit the registers
      kept[b] = look(next, std::true_type{});
      same += __popc(kept[b]);
    }
  } else {
    for (int b = 0; b < batches; ++b) same += __popc(look(b, std::true_type{}));
  }
  same = __builtin_amdgcn_readlane(wave_scan(same), 63);
  if (lane == 0) {
    less_sh[wave] = less;
    same_sh[wave] = same;
  }
  __syncthreads();
  int at = 0, end = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    at += less_sh[w] + (w < wave ? same_sh[w] : 0);
    end += less_sh[w] + same_sh[w];
  }
  at = __builtin_amdgcn_readfirstlane(at);
  end = __builtin_amdgcn_readfirstlane(end);
  if (threadIdx.x == 0) {
    if (!NONE) offsets[mine] = at;
    if (mine + 1 == (uint32_t)experts) offsets[experts] = end;
  }
  auto write = [&](int b, uint32_t hits) {
    if (__ballot(hits != 0) == 0) return;
    // The lanes' hits of eight steps, summed over the lanes at once: word d holds those of steps d and d + 4 in halves,
    // where the hits of the steps before are added in (at most 2048 together).
    uint32_t n = hits - ((hits >> 1) & 0x55555555u), before[4], total[4];
    n = (n & 0x33333333u) + ((n >> 2) & 0x33333333u);         // four bits per step
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t own = (n >> (4 * d)) & 0x000F000Fu, upto = (uint32_t)wave_scan((int)own);
      before[d] = upto - own;
      total[d] = __builtin_amdgcn_readlane((int)upto, 63);
    }
    uint32_t low = 0, high = (total[0] + total[1] + total[2] + total[3]) & 0xFFFFu;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      before[d] += low | high << 16;
      low += total[d] & 0xFFFFu;
      high += total[d] >> 16;
    }
    for (uint32_t left = hits; left; left &= left - 1) {      // every lane's next one
      const int bit = __builtin_ctz(left), step = bit >> 2;
      const uint32_t even = step & 2 ? before[2] : before[0], odd = step & 2 ? before[3] : before[1];
      const uint32_t both = step & 1 ? odd : even;
      const uint32_t nth = (step & 4 ? both >> 16 : both & 0xFFFFu) + __popc((hits >> (4 * step)) & ((1u << (bit & 3)) - 1));
      order[at + nth] = begin + (8 * b + step) * 256 + (bit & 3);
    }
    at += high;
  };
  if constexpr (KEEP) {
#pragma unroll
    for (int b = 0; b < kGroupBatches; ++b) write(b, kept[b]);
  } else if (same != 0) {
    for (int b = 0; b < batches; ++b) write(b, look(b, std::false_type{}));
  }
  return end;
}

template <bool KEEP>
__global__ __launch_bounds__(1024, 8) void group_kernel(const int32_t* __restrict__ sel, int pairs, int experts,
                                                        int32_t* __restrict__ offsets, int32_t* __restrict__ order) {
  __shared__ int less_sh[16], same_sh[16];
  if ((int)blockIdx.x < experts) {
    const int end = group_pairs<KEEP, false>(sel, pairs, experts, blockIdx.x, less_sh, same_sh, offsets, order);
    if ((int)gridDim.x > experts || (int)blockIdx.x + 1 != experts || end == pairs) return;
    __syncthreads();                                          // the counts in LDS have been read
  }
  group_pairs<KEEP, true>(sel, pairs, experts, (uint32_t)experts, less_sh, same_sh, offsets, order);
}

// A workgroup for each expert and one for the pairs without one, unless that one would be alone in a second round of
// compute units: then the last expert's looks for them, if there are any (131072 pairs of 256 experts: 10.0 us, 13.9 with
// the one more; with 2% of the pairs without an expert 19.0 and 17.6).
hipError_t launch_moe_group(int pairs, int experts, const int32_t* sel, int32_t* offsets, int32_t* order, hipStream_t s) {
  const dim3 grid((unsigned)experts + (experts % kComputeUnits != 0)), block(1024);
  if (pairs <= 16 * 2048 * kGroupBatches) hipLaunchKernelGGL(group_kernel<true>, grid, block, 0, s, sel, pairs, experts, offsets, order);
  else hipLaunchKernelGGL(group_kernel<false>, grid, block, 0, s, sel, pairs, experts, offsets, order);
  return hipGetLastError();
}

}  // namespace tg

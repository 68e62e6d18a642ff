// Routing of tokens to experts: scores, groups, the top_k ids with their weights (moe_route), and the routed pairs in
// expert order (moe_group).
//
// An id is decided by comparing scores, so scores, keys and group values are formed in binary64 and equal ones go to
// the lowest index; a weight is rounded to binary32 once.
#include "tg_device.hpp"
#include "tg_internal.hpp"

namespace tg {

namespace {

constexpr double kNone = -__builtin_huge_val();

__device__ __forceinline__ double wave_max(double v) {
  for (int m = 32; m; m >>= 1) v = fmax(v, __shfl_xor(v, m, 64));
  return v;
}

__device__ __forceinline__ double wave_sum(double v) {
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

template <int DT>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
  if constexpr (DT == kF32) return reinterpret_cast<const float*>(p)[i];
  const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
  if constexpr (DT == kF16) return half_bits_to_float(b);
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}

}  // namespace

// One wave per token; lane l holds experts l, l + 64, ...
template <int V, int DT>
__global__ __launch_bounds__(64) void route_kernel(const RouteArgs a) {
  __shared__ double ranked_sh[V * 64];
  __shared__ double value_sh[64];
  const int lane = threadIdx.x, token = blockIdx.x;
  double score[V], ranked[V], key[V];
  bool poison = false;
  double top = kNone;
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    const float l = e < a.experts ? logit<DT>(a.logits, (int64_t)token * a.ld + e) : -__builtin_huge_valf();
    bias[i] = a.bias && e < a.experts ? a.bias[e] : 0.f;
    poison |= l != l || !(bias[i] < __builtin_huge_valf());
    key[i] = l;
    top = fmax(top, key[i]);
  }
  top = wave_max(top);
  if (!a.sigmoid) poison |= top == __builtin_huge_val();
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool none = key[i] == kNone;
    if (a.sigmoid) score[i] = none ? 0.0 : 1.0 / (1.0 + exp(-key[i]));
    else score[i] = none ? 0.0 : exp(key[i] - top);
    sum += score[i];
  }
  if (!a.sigmoid) {
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) score[i] = score[i] / sum;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    ranked[i] = key[i] == kNone || bias[i] == -__builtin_huge_valf() ? kNone : score[i] + (double)bias[i];
    if (a.bias) key[i] = ranked[i];
  }
  if (__ballot(poison)) {   // a NaN, or an infinity that leaves no order: the first top_k ids, with weights that say so
    for (int i = lane; i < a.top_k; i += 64) {
      a.sel[(int64_t)token * a.top_k + i] = i;
      a.weights[(int64_t)token * a.top_k + i] = __builtin_nanf("");
    }
    return;
  }
  if (a.n_group > 1) {
    const int size = a.experts / a.n_group;
#pragma unroll
    for (int i = 0; i < V; ++i) ranked_sh[lane + 64 * i] = ranked[i];
    __syncthreads();
    double value = kNone;
    if (lane < a.n_group) {
      double first = kNone, second = kNone;
      for (int i = 0; i < size; ++i) {
        const double v = ranked_sh[lane * size + i];
        if (v > first) {
          second = first;
          first = v;
        } else if (v > second) {
          second = v;
        }
      }
      value = a.group_top == 2 && second != kNone ? first + second : first;
    }
    value_sh[lane] = value;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < a.n_group; ++i) {
      const double v = value_sh[i];
      before += v > value || (v == value && i < lane) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < a.n_group && before < a.topk_group);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      if (e < a.experts && !((kept >> (e / size)) & 1)) key[i] = kNone;
    }
  }
  int my_id = -1;        // lane i keeps slot i
  double my_w = 0.0;
  for (int s = 0; s < a.top_k; ++s) {
    double best = kNone;
    int at = 1 << 30;
    double w = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > best) {
        best = key[i];
        at = lane + 64 * i;
        w = score[i];
      }
    for (int m = 32; m; m >>= 1) {
      const double ob = __shfl_xor(best, m, 64), ow = __shfl_xor(w, m, 64);
      const int oa = __shfl_xor(at, m, 64);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
        w = ow;
      }
    }
    if (best == kNone) break;   // no expert is left: the other slots stay -1 with weight 0
    if (lane == s) {
      my_id = at;
      my_w = w;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 64 * i == at) key[i] = kNone;
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
  const dim3 grid((unsigned)a.tokens), block(64);
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
// neighbouring stretches, so the order of the pairs is the order of the waves and, in a wave, of the lanes.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(1024) void group_kernel(const int32_t* __restrict__ sel, int pairs, int experts,
                                                     int32_t* __restrict__ offsets, int32_t* __restrict__ order) {
  __shared__ int less_sh[16], same_sh[16];
  const int lane = threadIdx.x & 63, wave = wave_id(), mine = blockIdx.x;
  const int stretch = ((pairs + 15) / 16 + 63) & ~63;
  const int begin = wave * stretch, end = min(begin + stretch, pairs);
  int less = 0, same = 0;
  for (int p = begin; p < end; p += 64) {
    int id = -1;
    const bool in = p + lane < end;
    if (in) id = sel[p + lane];
    if (id < 0 || id >= experts) id = experts;
    less += __popcll(__ballot(in && id < mine));
    same += __popcll(__ballot(in && id == mine));
  }
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
  if (threadIdx.x == 0) offsets[mine] = base;   // offsets[experts]: the number of pairs with an expert
  at += base;
  if (same == 0) return;
  for (int p = begin; p < end; p += 64) {
    int id = -1;
    const bool in = p + lane < end;
    if (in) id = sel[p + lane];
    if (id < 0 || id >= experts) id = experts;
    const uint64_t hit = __ballot(in && id == mine);
    if (in && id == mine) order[at + __popcll(hit & ((1ull << lane) - 1))] = p + lane;
    at += __popcll(hit);
  }
}

hipError_t launch_moe_group(int pairs, int experts, const int32_t* sel, int32_t* offsets, int32_t* order, hipStream_t s) {
  hipLaunchKernelGGL(group_kernel, dim3((unsigned)experts + 1), dim3(1024), 0, s, sel, pairs, experts, offsets, order);
  return hipGetLastError();
}

}  // namespace tg

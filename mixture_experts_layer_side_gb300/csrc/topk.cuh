// Top-k selection and softmax of one token's router logits by one warp,
// shared by the router and the layer for a few tokens.
#pragma once

#include <limits.h>
#include <math.h>
#include <stdint.h>

namespace mok {

constexpr int kMaxRouterExperts = 1024;  // keys held in registers: 32 per lane

// (key, expert) pairs ordered by descending key, then ascending expert.
__device__ __forceinline__ bool ranks_before(float ka, int ea, float kb, int eb) {
  return ka > kb || (ka == kb && ea < eb);
}

// The k largest row[e] + bias[e] (ties to the lower expert, descending key
// order; a NaN key ranks last) and the softmax over the k chosen, unbiased
// logits.  Lane l holds the keys of experts l, l + 32, ... (PER of them at
// most); lane j < k ends with the j-th choice.
template <int PER>
__device__ __forceinline__ void topk_softmax_warp(const float* row, const float* bias, int E, int k, int lane,
                                                  int& my_e, float& my_s) {
  float key[PER];
  const int per_lane = (E + 31) >> 5;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    const float v = (i < per_lane && e < E) ? row[e] + (bias ? bias[e] : 0.0f) : 0.0f;
    key[i] = isnan(v) ? -INFINITY : v;
  }
  uint32_t taken = 0;  // bit i: expert lane + 32 i already chosen
  my_e = -1;
  float my_l = 0.0f;
  for (int j = 0; j < k; ++j) {
    float bk = 0.0f;
    int be = INT_MAX;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      if (i < per_lane && e < E && !((taken >> i) & 1u) && (be == INT_MAX || ranks_before(key[i], e, bk, be))) {
        bk = key[i];
        be = e;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ok = __shfl_xor_sync(0xffffffffu, bk, o);
      const int oe = __shfl_xor_sync(0xffffffffu, be, o);
      if (oe != INT_MAX && (be == INT_MAX || ranks_before(ok, oe, bk, be))) {
        bk = ok;
        be = oe;
      }
    }
    if (be == INT_MAX) break;  // fewer than k experts (the host rules it out)
    if ((be & 31) == lane) taken |= 1u << (be >> 5);
    if (lane == j) {
      my_e = be;
      my_l = row[be];
    }
  }
  float m = lane < k ? my_l : -INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ez = lane < k ? expf(my_l - m) : 0.0f;
  float sum = ez;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  my_s = ez / sum;
}

}  // namespace mok

// Top-k selection and softmax of one token's router logits by one warp,
// shared by the router and the layer for a few tokens.
#pragma once

#include <limits.h>
#include <math.h>
#include <stdint.h>

namespace mok {

constexpr int kMaxRouterExperts = 1024;  // keys held in registers: 32 per lane

// Keys as integers in the same order; -0 and +0 are one key, 0 is below every key.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

// The k largest row[e] + bias[e] (ties to the lower expert, descending key
// order; a NaN key ranks last) and the softmax over the k chosen, unbiased
// logits.  Lane l holds the keys of experts l, l + 32, ... (PER of them at
// most); lane j < k ends with the j-th choice.
template <int PER>
__device__ __forceinline__ void topk_softmax_warp(const float* row, const float* bias, int E, int k, int lane,
                                                  int& my_e, float& my_s) {
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0;  // no expert, or one already chosen
    if (e < E) {
      const float v = row[e] + (bias ? bias[e] : 0.0f);
      key[i] = order_key(isnan(v) ? -INFINITY : v);
    }
  }
  my_e = -1;
  float my_l = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(0xffffffffu, best);
    if (best == 0) break;  // fewer than k experts (the host rules it out)
    int e = INT_MAX;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == best) e = lane + 32 * i;
    e = (int)__reduce_min_sync(0xffffffffu, (unsigned)e);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 32 * i == e) key[i] = 0;
    if (lane == j) {
      my_e = e;
      my_l = row[e];
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

// Dropout's random bits, shared by the kernels that drop (dropout.cu,
// residual.cu): Philox-4x32 with ten rounds, the counter-based generator of
// Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2,
// 3" (SC 2011).  A block of eight consecutive elements takes one 128-bit
// output, 16 bits an element, so nothing is stored between a forward pass and
// its backward pass: both make the same bits from the element's index.
//
// 16 bits and not 32: an output is ten dependent rounds of two wide
// multiplications, and one per four elements, which 32 bits would take, bounds
// bf16 (dropout of 16,384 rows of 7,168: one output a block of eight 84 us, two
// 121; f32, with twice the bytes an element, is as fast with two).  The price is
// that p is a multiple of 2^-16.
#pragma once

#include "mok_internal.cuh"

namespace mok {

struct DropParams {
  uint32_t key0, key1;       // the seed
  uint64_t call;             // number of the call ...
  const int64_t* call_dev;   // ... plus this device word, where it is given
  uint32_t below;            // p * 65536: elements whose bits are below are dropped; 0: dropout is off
  float scale;               // 1 / (1 - p); 0 where all are dropped
};

// The counter's upper half, read once per thread.
__device__ __forceinline__ uint64_t drop_call(const DropParams& d) {
  return d.call_dev ? d.call + (uint64_t)*d.call_dev : d.call;
}

__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t call, uint32_t key0, uint32_t key1) {
  uint4 c = make_uint4((uint32_t)block, (uint32_t)(block >> 32), (uint32_t)call, (uint32_t)(call >> 32));
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c.x * 0xD2511F53u, b = (uint64_t)c.z * 0xCD9E8D57u;
    c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ key0, (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ key1, (uint32_t)a);
    key0 += 0x9E3779B9u;
    key1 += 0xBB67AE85u;
  }
  return c;
}

// Both halves of a word are compared at its upper end, where the bits below them change nothing: 16 bits are not below
// p * 65536 if what they begin is more than p * 2^32 - 1.  (Nothing may be asked where p is 0.)
__device__ __forceinline__ uint32_t drop_most(const DropParams& d) { return (d.below << 16) - 1u; }
// Whether element j of a block is kept.
__device__ __forceinline__ bool drop_kept(const uint4& r, int j, uint32_t most) {
  const uint32_t w = j < 2 ? r.x : j < 4 ? r.y : j < 6 ? r.z : r.w;
  return (j & 1 ? w : w << 16) > most;
}
__device__ __forceinline__ uint4 drop_block(const DropParams& d, uint64_t block, uint64_t call) {
  return philox(block, call, d.key0, d.key1);
}
// Which of the eight elements of a block are kept, element j in bit j.
__device__ __forceinline__ uint32_t drop_keep8(const DropParams& d, uint64_t block, uint64_t call) {
  const uint4 r = drop_block(d, block, call);
  uint32_t keep = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) keep |= drop_kept(r, j, drop_most(d)) ? 1u << j : 0u;
  return keep;
}

}  // namespace mok

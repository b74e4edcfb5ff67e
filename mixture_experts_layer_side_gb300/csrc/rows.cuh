// Eight consecutive elements of a row at a time, at any alignment, for the
// kernels that move rows (residual.cu, dropout.cu).
//
// ALIGNED: they are whole 16-byte vectors.  Otherwise a row starts anywhere:
// a thread loads the aligned vectors that its eight elements lie in and
// shifts them into place, and stores whole vectors made of its own elements
// and its neighbour's; what is left at the ends of a warp's and of a row's
// elements goes one by one.  No byte outside the tensor is touched (a vector
// may hold a neighbouring row's, which are not used).
#pragma once

#include "mok_internal.cuh"

namespace mok {

// 32-bit words of eight elements.
template <typename E>
__host__ __device__ constexpr int words8() { return 2 * sizeof(E); }
// 16-byte vectors that eight elements touch.
template <typename E, bool ALIGNED>
__host__ __device__ constexpr int vectors8() { return words8<E>() / 4 + (ALIGNED ? 0 : 1); }

// Where a tensor begins and ends.
struct Span8 {
  uintptr_t lo, hi;
};
template <typename E>
__device__ __forceinline__ Span8 span_of(const E* p, long rows, long ld, long cols) {
  return {reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p + (rows - 1) * ld + cols)};
}

__device__ __forceinline__ uint32_t misalign(const void* p) { return (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u; }

// Words from byte `m` (0 to 15, a multiple of the element) of c on.  m is the same for a whole row, so each of its four
// distances in words has a branch of its own, and rows that lie on a vector's start go past all of it (8,192 rows of 4,099
// bf16, forward: words moved step by step 128 us, so 115).
template <typename E, int FIRST>
__device__ __forceinline__ void shift_from(const uint32_t (&c)[words8<E>() + 4], uint32_t m, uint32_t (&w)[words8<E>()]) {
#pragma unroll
  for (int i = 0; i < words8<E>(); ++i) {
    if constexpr (sizeof(E) == 2) w[i] = __funnelshift_r(c[i + FIRST], c[i + FIRST + 1], (m & 2) * 8);
    else w[i] = c[i + FIRST];
  }
}
template <typename E>
__device__ __forceinline__ void shift8(const uint32_t (&c)[words8<E>() + 4], uint32_t m, uint32_t (&w)[words8<E>()]) {
  switch (m >> 2) {
    case 0: shift_from<E, 0>(c, m, w); break;
    case 1: shift_from<E, 1>(c, m, w); break;
    case 2: shift_from<E, 2>(c, m, w); break;
    default: shift_from<E, 3>(c, m, w); break;
  }
}

// Zeros in place of the elements from the n-th on.
template <typename E>
__device__ __forceinline__ void keep_first(uint32_t (&w)[words8<E>()], int n) {
#pragma unroll
  for (int i = 0; i < words8<E>(); ++i) {
    if constexpr (sizeof(E) == 2) w[i] = 2 * i >= n ? 0u : 2 * i + 1 >= n ? w[i] & 0xffffu : w[i];
    else w[i] = i >= n ? 0u : w[i];
  }
}

// Whether all vectors of eight elements at p lie in the tensor.
template <typename E>
__device__ __forceinline__ bool whole_vectors(const E* p, uint32_t m, const Span8& span) {
  const uintptr_t base = reinterpret_cast<uintptr_t>(p) - m;
  return base >= span.lo && base + 4 * words8<E>() + (m ? 16 : 0) <= span.hi;
}

// The first n (1 to 8) elements at p, zeros after them.
template <typename E, bool ALIGNED>
__device__ __forceinline__ void load_words(const E* p, int n, const Span8& span, uint32_t (&w)[words8<E>()]) {
  constexpr int W = words8<E>();
  if constexpr (ALIGNED) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else {
    const uint32_t m = misalign(p);
    if (m == 0 && n == 8) {
      load_words<E, true>(p, 8, span, w);
    } else if (whole_vectors(p, m, span)) {
      const uint4* at = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) - m);
      uint32_t c[W + 4];
#pragma unroll
      for (int i = 0; i <= W / 4; ++i) {
        const uint4 v = i < W / 4 || m ? at[i] : make_uint4(0, 0, 0, 0);
        c[4 * i] = v.x, c[4 * i + 1] = v.y, c[4 * i + 2] = v.z, c[4 * i + 3] = v.w;
      }
      shift8<E>(c, m, w);
      if (n < 8) keep_first<E>(w, n);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if constexpr (sizeof(E) == 2) {
          const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
          w[i] = (2 * i < n ? q[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)q[2 * i + 1] << 16 : 0u);
        } else {
          w[i] = i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
        }
      }
    }
  }
}

// Asynchronous copies of what load_words reads into shared memory, vector i at dst + i * apart (16 bytes each), and the
// elements out of it.
__device__ __forceinline__ void copy_ahead(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
template <typename E, bool ALIGNED>
__device__ __forceinline__ void copy_words(uint4* dst, int apart, const E* p, int n, const Span8& span) {
  constexpr int W = words8<E>();
  if constexpr (ALIGNED) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) copy_ahead(dst + i * apart, reinterpret_cast<const uint4*>(p) + i);
  } else {
    const uint32_t m = misalign(p);
    if (whole_vectors(p, m, span)) {
      const uint4* at = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) - m);
#pragma unroll
      for (int i = 0; i <= W / 4; ++i)
        if (i < W / 4 || m) copy_ahead(dst + i * apart, at + i);
    } else {
      for (int e = 0; e < n; ++e) {
        const uint32_t byte = m + e * sizeof(E);
        *reinterpret_cast<E*>(reinterpret_cast<char*>(dst + (byte >> 4) * apart) + (byte & 15)) = p[e];
      }
    }
  }
}
// p: what was copied (its alignment counts)
template <typename E, bool ALIGNED>
__device__ __forceinline__ void copied_words(const uint4* src, int apart, const E* p, int n, uint32_t (&w)[words8<E>()]) {
  constexpr int W = words8<E>();
  if constexpr (ALIGNED) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 v = src[i * apart];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else {
    const uint32_t m = misalign(p);
    if (m == 0) {
      copied_words<E, true>(src, apart, p, n, w);
    } else {
      uint32_t c[W + 4];
#pragma unroll
      for (int i = 0; i <= W / 4; ++i) {
        const uint4 v = src[i * apart];
        c[4 * i] = v.x, c[4 * i + 1] = v.y, c[4 * i + 2] = v.z, c[4 * i + 3] = v.w;
      }
      shift8<E>(c, m, w);
    }
    if (n < 8) keep_first<E>(w, n);
  }
}

// Stores the first n (0 to 8) of eight elements at p.  Unaligned, all lanes of a warp call it together, for elements
// that lie side by side and for addresses of one alignment; `next` is the n of the next lane (0 for the last).
template <typename E, bool ALIGNED>
__device__ __forceinline__ void store_words(E* p, int n, int next, int lane, const uint32_t (&w)[words8<E>()]) {
  constexpr int W = words8<E>();
  const uint32_t m = ALIGNED ? 0u : misalign(p);
  uint32_t single = 0;  // elements that go one by one
  if (ALIGNED || m == 0) {
    if (n == 8) {
#pragma unroll
      for (int i = 0; i < W / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
      single = (1u << n) - 1u;
    }
  } else {
    constexpr int V = 16 / sizeof(E);          // elements of a vector
    const int head = V - (int)(m / sizeof(E));  // own elements ahead of the first vector boundary
    uint32_t c[W + 4], r[W];
#pragma unroll
    for (int i = 0; i < W; ++i) c[i] = w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[W + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
    shift8<E>(c, 16 - m, r);
    single = (1u << n) - 1u;
    // (the lane before has this one's head in its last vector)
    if (lane > 0 && n >= head) single &= ~((1u << head) - 1u);
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const int from = head + i * V;  // own elements of the vector, the neighbour's after the eighth
      const bool last = i == W / 4 - 1;
      if (last ? n == 8 && next >= head : n >= from + V) {
        *reinterpret_cast<uint4*>(reinterpret_cast<char*>(p) + (16 - m) + 16 * i) =
            make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        single &= ~(((1u << V) - 1u) << from);
      }
    }
  }
  if (single) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (!((single >> e) & 1u)) continue;
      if constexpr (sizeof(E) == 2) reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
      else reinterpret_cast<uint32_t*>(p)[e] = w[e];
    }
  }
}

}  // namespace mok

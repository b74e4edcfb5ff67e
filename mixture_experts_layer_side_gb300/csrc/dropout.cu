// Dropout by itself: out_i = x_i / (1 - p) where the element is kept, else 0
// (whatever x_i is).  The bits come from the element's index in row-major
// order (philox.cuh), so the gradient is the same call on the output's
// gradient.  Bound by HBM: one read and one write an element.
#include <algorithm>

#include "residual.cuh"

namespace mok {

namespace {

__device__ __forceinline__ void drop_store(float& v, bool keep, float scale) { v = keep ? v * scale : 0.0f; }
__device__ __forceinline__ void drop_store(__nv_bfloat16& v, bool keep, float scale) {
  v = keep ? __float2bfloat16_rn(__bfloat162float(v) * scale) : __float2bfloat16_rn(0.0f);
}

// A thread takes blocks of eight consecutive elements.  VEC: a block lies in
// one row and is made of whole vectors; otherwise its elements are found one
// by one.
template <typename E, bool VEC>
__global__ void __launch_bounds__(256) dropout_kernel(int64_t rows, int64_t cols, const E* x, int64_t ldx,
                                                      const DropParams d, E* out, int64_t ldo) {
  const int64_t n = rows * cols, blocks = (n + 7) / 8;
  const uint64_t call = drop_call(d);
  for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < blocks; b += (int64_t)gridDim.x * blockDim.x) {
    const uint32_t keep = drop_keep8(d, b, call);
    int64_t r = b * 8 / cols, c = b * 8 - r * cols;
    if constexpr (VEC) {
      alignas(16) E v[8];
      constexpr int kWords = 8 * sizeof(E) / 16;
      const uint4* src = reinterpret_cast<const uint4*>(x + r * ldx + c);
#pragma unroll
      for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(v)[i] = src[i];
#pragma unroll
      for (int e = 0; e < 8; ++e) drop_store(v[e], (keep >> e) & 1u, d.scale);
      uint4* dst = reinterpret_cast<uint4*>(out + r * ldo + c);
#pragma unroll
      for (int i = 0; i < kWords; ++i) dst[i] = reinterpret_cast<const uint4*>(v)[i];
    } else {
      for (int e = 0; e < 8 && b * 8 + e < n; ++e) {
        E v = x[r * ldx + c];
        drop_store(v, (keep >> e) & 1u, d.scale);
        out[r * ldo + c] = v;
        if (++c == cols) c = 0, ++r;
      }
    }
  }
}

template <typename E>
cudaError_t launch(int64_t rows, int64_t cols, const E* x, int64_t ldx, const DropParams& d, E* out, int64_t ldo,
                   cudaStream_t st) {
  // rows without a gap are one long row
  if (ldx == cols && ldo == cols) cols *= rows, rows = 1, ldx = ldo = cols;
  constexpr int kVec = 16 / sizeof(E);
  const bool vec = cols % 8 == 0 && ldx % kVec == 0 && ldo % kVec == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(out) % 16 == 0;
  const int64_t blocks = (rows * cols + 7) / 8;
  const int grid = (int)std::min<int64_t>((blocks + 255) / 256, (int64_t)device_sm_count() * 8);
  if (vec) dropout_kernel<E, true><<<grid, 256, 0, st>>>(rows, cols, x, ldx, d, out, ldo);
  else dropout_kernel<E, false><<<grid, 256, 0, st>>>(rows, cols, x, ldx, d, out, ldo);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dropout(mok_dtype type, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                           const DropParams& d, void* out, int64_t ldo, cudaStream_t st) {
  if (type == MOK_TYPE_BF16)
    return launch(rows, cols, static_cast<const __nv_bfloat16*>(x), ldx, d, static_cast<__nv_bfloat16*>(out), ldo, st);
  return launch(rows, cols, static_cast<const float*>(x), ldx, d, static_cast<float*>(out), ldo, st);
}

}  // namespace mok

// Dropout by itself: out_i = x_i / (1 - p) where the element is kept, else 0
// (whatever x_i is).  The bits come from the element's index in row-major
// order (philox.cuh), so the gradient is the same call on the output's
// gradient.  Bound by HBM: one read and one write an element.
#include <algorithm>

#include "residual.cuh"
#include "rows.cuh"

namespace mok {

namespace {

// Pieces of 256 columns of a row, a warp's at a time: as many in flight at once.
constexpr int kPieces = 2;

// Eight elements with those dropped that `keep` says.
template <typename E>
__device__ __forceinline__ void drop_words(uint32_t (&w)[words8<E>()], uint32_t keep, float scale) {
#pragma unroll
  for (int i = 0; i < words8<E>(); ++i) {
    if constexpr (sizeof(E) == 2) {
      const float a = (keep >> (2 * i)) & 1u ? __uint_as_float(w[i] << 16) * scale : 0.0f;
      const float b = (keep >> (2 * i + 1)) & 1u ? __uint_as_float(w[i] & 0xffff0000u) * scale : 0.0f;
      const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      w[i] = (keep >> i) & 1u ? __float_as_uint(__uint_as_float(w[i]) * scale) : 0u;
    }
  }
}

// ALIGNED: rows of whole vectors and whole blocks of the generator.  Otherwise a lane's elements lie in two blocks, of
// which the second is the next lane's first.
template <typename E, bool ALIGNED>
__global__ void __launch_bounds__(256) dropout_kernel(int64_t rows, int64_t cols, int64_t row_pieces, const E* x, int64_t ldx,
                                                      const DropParams d, E* out, int64_t ldo) {
  const int lane = threadIdx.x & 31;
  const int64_t pieces = rows * row_pieces, warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  const Span8 span = span_of(x, rows, ldx, cols);
  const uint64_t call = drop_call(d);
  for (int64_t p0 = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); p0 < pieces; p0 += kPieces * warps) {
    uint32_t w[kPieces][words8<E>()];
    int64_t row[kPieces], col[kPieces];
    int n[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int64_t piece = p0 + i * warps;
      n[i] = 0;
      if (piece >= pieces) continue;  // (the same for a warp)
      row[i] = rows == 1 ? 0 : piece / row_pieces;
      col[i] = (piece - row[i] * row_pieces) * 256 + lane * 8;
      n[i] = (int)min((int64_t)8, max((int64_t)0, cols - col[i]));
      if (n[i] > 0) load_words<E, ALIGNED>(x + row[i] * ldx + col[i], n[i], span, w[i]);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (p0 + i * warps >= pieces) break;
      const uint64_t first = (uint64_t)(row[i] * cols + col[i]);
      uint32_t keep = drop_keep8(d, first >> 3, call);
      if (d.below == 0) {
        keep = 0xffu;
      } else if constexpr (!ALIGNED) {
        uint32_t after = __shfl_down_sync(0xffffffffu, keep, 1);
        if (lane == 31) after = drop_keep8(d, (first >> 3) + 1, call);
        keep = (keep | after << 8) >> (first & 7);
      }
      drop_words<E>(w[i], keep, d.scale);
      E* to = out + row[i] * ldo + col[i];
      if constexpr (ALIGNED) {
        if (n[i] == 8) store_words<E, true>(to, 8, 8, lane, w[i]);
      } else {
        const int64_t after = cols - col[i] - 8;
        const int next = lane < 31 ? (int)min((int64_t)8, max((int64_t)0, after)) : 0;
        store_words<E, false>(to, n[i], next, lane, w[i]);
      }
    }
  }
}

template <typename E>
cudaError_t launch(int64_t rows, int64_t cols, const E* x, int64_t ldx, const DropParams& d, E* out, int64_t ldo,
                   cudaStream_t st) {
  // rows without a gap are one long row
  if ((ldx == cols && ldo == cols) || rows == 1) cols *= rows, rows = 1, ldx = ldo = cols;
  constexpr int kVec = 16 / sizeof(E);
  const bool aligned = cols % 8 == 0 && ldx % kVec == 0 && ldo % kVec == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(out) % 16 == 0;
  const int64_t row_pieces = (cols + 255) / 256, pieces = rows * row_pieces;
  const int grid = (int)std::min<int64_t>((pieces + 8 * kPieces - 1) / (8 * kPieces), (int64_t)device_sm_count() * 8);
  auto kernel = aligned ? dropout_kernel<E, true> : dropout_kernel<E, false>;
  kernel<<<grid, 256, 0, st>>>(rows, cols, row_pieces, x, ldx, d, out, ldo);
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

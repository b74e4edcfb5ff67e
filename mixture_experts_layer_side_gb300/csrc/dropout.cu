// Dropout by itself: out_i = x_i / (1 - p) where the element is kept, else 0
// (whatever x_i is).  The bits come from the element's index in row-major
// order (philox.cuh), so the gradient is the same call on the output's
// gradient.  Bound by HBM: one read and one write an element.
#include <algorithm>

#include "residual.cuh"
#include "rows.cuh"

namespace mok {

namespace {

// Pieces of 256 elements, a warp's at a time: as many in flight at once.
constexpr int kPieces = 2;

// Eight elements, with zeros in place of those that the block's bits drop.
template <typename E>
__device__ __forceinline__ void drop_words(uint32_t (&w)[words8<E>()], const uint4& bits, uint32_t most, float scale) {
#pragma unroll
  for (int i = 0; i < words8<E>(); ++i) {
    if constexpr (sizeof(E) == 2) {
      const float a = drop_kept(bits, 2 * i, most) ? __uint_as_float(w[i] << 16) * scale : 0.0f;
      const float b = drop_kept(bits, 2 * i + 1, most) ? __uint_as_float(w[i] & 0xffff0000u) * scale : 0.0f;
      const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      w[i] = drop_kept(bits, i, most) ? __float_as_uint(__uint_as_float(w[i]) * scale) : 0u;
    }
  }
}

__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Rows of whole vectors, which are whole blocks of the generator (or one row, whose last block may be a part): a block a
// lane.
template <typename E>
__global__ void __launch_bounds__(256, 5) dropout_kernel(int64_t rows, int64_t cols, int64_t row_pieces, const E* x,
                                                         int64_t ldx, const DropParams d, E* out, int64_t ldo) {
  const int lane = threadIdx.x & 31;
  const int64_t pieces = rows * row_pieces, warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  const uint64_t call = drop_call(d);
  const uint32_t most = drop_most(d);
  for (int64_t p0 = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); p0 < pieces; p0 += kPieces * warps) {
    uint32_t w[kPieces][words8<E>()];
    int64_t row[kPieces], col[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int64_t piece = p0 + i * warps;
      row[i] = rows == 1 ? 0 : piece / row_pieces;
      col[i] = (piece - row[i] * row_pieces) * 256 + lane * 8;
      if (piece >= pieces) col[i] = cols;
      if (col[i] + 8 <= cols) load_words<E, true>(x + row[i] * ldx + col[i], 8, Span8{}, w[i]);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (col[i] >= cols) continue;
      const uint4 bits = d.below ? drop_block(d, (uint64_t)(row[i] * cols + col[i]) >> 3, call) : make_uint4(0, 0, 0, 0);
      if (col[i] + 8 <= cols) {
        if (d.below) drop_words<E>(w[i], bits, most, d.scale);
        store_words<E, true>(out + row[i] * ldo + col[i], 8, 8, lane, w[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (col[i] + j < cols)
            put(out + col[i] + j, d.below && !drop_kept(bits, j, most) ? 0.0f : value(x[col[i] + j]) * d.scale);
      }
    }
  }
}

// Rows of any alignment.  A piece is 32 blocks of the generator, from the one on that the row begins in: a lane makes a
// block's bits and takes every 32nd element, whose bits it asks of the lane that has them, so that a warp's accesses are
// of single elements side by side, which no alignment hinders.  (Vectors that are shifted into place take 204 us for
// 16,384 rows of 7,168 bf16, 7,171 apart; these 185; of 4,099 f32 165, these 105.)
template <typename E>
__global__ void __launch_bounds__(256) dropout_any_kernel(int64_t rows, int64_t cols, int64_t row_pieces, const E* x,
                                                          int64_t ldx, const DropParams d, E* out, int64_t ldo) {
  const int lane = threadIdx.x & 31;
  const int64_t pieces = rows * row_pieces, warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  const uint64_t call = drop_call(d);
  for (int64_t piece = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); piece < pieces; piece += warps) {
    const int64_t row = rows == 1 ? 0 : piece / row_pieces;
    const uint64_t first = (uint64_t)(row * cols);
    const int64_t p = piece - row * row_pieces, c0 = p * 256 + lane - (int64_t)(first & 7);
    const E* from = x + row * ldx + c0;
    E* to = out + row * ldo + c0;
    float v[8];
    bool in[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      in[e] = c0 + 32 * e >= 0 && c0 + 32 * e < cols;
      v[e] = in[e] ? value(from[32 * e]) : 0.0f;
    }
    const uint32_t keep = d.below ? drop_keep8(d, (first >> 3) + (uint64_t)p * 32 + lane, call) : 0xffu;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t of = __shfl_sync(0xffffffffu, keep, 4 * e + (lane >> 3));
      if (in[e]) put(to + 32 * e, (of >> (lane & 7)) & 1u ? v[e] * d.scale : 0.0f);
    }
  }
}

template <typename E>
cudaError_t launch(int64_t rows, int64_t cols, const E* x, int64_t ldx, const DropParams& d, E* out, int64_t ldo,
                   cudaStream_t st) {
  // rows without a gap are one long row
  if ((ldx == cols && ldo == cols) || rows == 1) cols *= rows, rows = 1, ldx = ldo = cols;
  constexpr int kVec = 16 / sizeof(E);
  const bool aligned = (rows == 1 || (cols % 8 == 0 && ldx % kVec == 0 && ldo % kVec == 0)) && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(out) % 16 == 0;
  // (a row of any alignment may begin at the last element of a block)
  const int64_t row_pieces = aligned ? (cols + 255) / 256 : (cols + 7 + 255) / 256, pieces = rows * row_pieces;
  const int each = 8 * (aligned ? kPieces : 1);
  const int grid = (int)std::min<int64_t>((pieces + each - 1) / each, (int64_t)device_sm_count() * 8);
  auto kernel = aligned ? dropout_kernel<E> : dropout_any_kernel<E>;
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

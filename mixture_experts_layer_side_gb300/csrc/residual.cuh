// The join of a block with its residual stream (residual.cu) and dropout by
// itself (dropout.cu), shared declarations.
#pragma once

#include "philox.cuh"

namespace mok {

struct ResidualParams {
  int T, H;
  int G, rows_per_gate;  // gate rows and the rows that each serves (G = 0: no gate)
  float scale, eps;
  DropParams drop;
  const void *w_out, *gate, *w_next;
  // forward: x, y -> xo, n;  backward: x is the forward's xo
  const void *x, *y;
  long ldx, ldy;
  void *xo, *n;
  long ldxo, ldn;
  // backward: gradients of xo and n -> gradients of x and y
  const void *dxo, *dn;
  long lddxo, lddn;
  void *dx, *dy;
  long lddx, lddy;
  float *dw_out, *dw_next;
  void* dgate;
  float* part;  // column sums of the workers (residual.cu)
};

// f32 words that the backward pass keeps its workers' column sums in.
size_t residual_part_floats(int T, int H);
cudaError_t launch_residual_forward(mok_dtype stream, mok_dtype branch, const ResidualParams& p, int* launches,
                                    cudaStream_t st);
cudaError_t launch_residual_backward(mok_dtype stream, mok_dtype branch, const ResidualParams& p, int* launches,
                                     cudaStream_t st);

// rows x cols elements, rows ldx / ldo apart
cudaError_t launch_dropout(mok_dtype type, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                           const DropParams& d, void* out, int64_t ldo, cudaStream_t st);

}  // namespace mok

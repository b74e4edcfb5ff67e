// The dense gated feed-forward block (ffn.cu), shared declarations.
#pragma once

#include "mok_internal.cuh"

namespace mok {

// What one launch of the block's matrix products computes.
enum FfnMode : int {
  FFN_GATE = 0,   // [h | u] = x [W1 | W3];  epilogue a = silu(h) u (and h, u for the backward pass)
  FFN_OUT = 1,    // out = a W2
  FFN_DA = 2,     // da = dout W2^T;         epilogue dh, du
  FFN_DX = 3,     // dx = dh W1^T + du W3^T
  FFN_DW13 = 4,   // dW1 = x^T dh, dW3 = x^T du
  FFN_DW2 = 5,    // dW2 = a^T dout
};

struct FfnParams {
  int M, N;        // rows and columns of the result (FFN_GATE: N = I; FFN_DW13: N = I, twice)
  int K;           // length of the sums (FFN_DX: of each of the two)
  int32_t* hdr;    // workspace header: error and abort words
  __nv_bfloat16* out[3];        // FFN_GATE: a, h, u (h, u may be null); FFN_DA: dh, du; FFN_DW13: dW1, dW3; else [0]
  const __nv_bfloat16 *h, *u;   // FFN_DA
  int after;       // FfnAfter
};

// How a launch stands to the one before it in the stream.
enum FfnAfter : int {
  FFN_AFTER_ALL = 0,   // an ordinary launch
  FFN_READS_IT = 1,    // starts beside it, waits for its end before it reads anything
  FFN_BESIDE_IT = 2,   // reads nothing that it writes: waits for its end at its own end
};

struct FfnOperand {
  const void* p;
  int rows, cols;  // as it lies in memory, dense
};

// a[1], b[1]: the second operands of FFN_GATE (b: W3), FFN_DX (both) and FFN_DW13 (b)
cudaError_t launch_ffn(FfnMode mode, const FfnOperand (&a)[2], const FfnOperand (&b)[2], const FfnParams& p,
                       cudaStream_t st);

}  // namespace mok

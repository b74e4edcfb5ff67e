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
  __nv_bfloat16* out[2];  // FFN_DA: dh, du; FFN_DW13: dW1, dW3; else [0]
  float *h, *u;           // FFN_GATE: kept there (or null); FFN_DA: read (laid out by ffn_kept_floats)
  int after;       // FfnAfter
  int a_rows;      // rows of A that a CTA brings (set by the launch)
  int sms;         // SMs that its tiles may be spread over (0: all)
};

// How a launch stands to the one before it in the stream.  Each lets the next one start when its own start is done, which
// for FFN_READS_IT is after its wait: what may still run beside an FFN_BESIDE_IT are the launches back to the last of
// another kind, that one among them, and what stands before those is over.  So dW1 and dW3, beside dx, may read dh and du,
// as dx waits for dW2, which ends after da; right after dW2 they might not.
enum FfnAfter : int {
  FFN_AFTER_ALL = 0,   // an ordinary launch
  FFN_READS_IT = 1,    // starts beside it, waits for its end (and so for all before it) before it reads anything
  FFN_BESIDE_IT = 2,   // reads nothing that those beside it write, writes nothing that they touch: waits at its own end
};

// Floats that h or u of T rows takes where it is kept: rows in whole 32s.
inline size_t ffn_kept_floats(int T, int I) { return ((size_t)T + 31) / 32 * 32 * (size_t)I; }

struct FfnOperand {
  const void* p;
  int rows, cols;  // as it lies in memory, dense
};

// Two launches of which the second runs beside the first: how many SMs each may spread its tiles over, so that both are
// there at once where they are few (all where they are not).  (1,000 tokens, H 1144, I 680, backward: each by itself on all
// SMs 45 us, shared 32.)
struct FfnSize {
  FfnMode mode;
  int M, N, K;  // as in FfnParams
};
void ffn_share_sms(const FfnSize (&two)[2], int (&sms)[2]);

// a[1], b[1]: the second operands of FFN_GATE (b: W3), FFN_DX (both) and FFN_DW13 (b)
cudaError_t launch_ffn(FfnMode mode, const FfnOperand (&a)[2], const FfnOperand (&b)[2], FfnParams p,
                       cudaStream_t st);

// The forward pass of a token or a few (ffn_rows.cu): two launches.
// At most four tokens: eight are no faster so (H 2048, I 768: 1 token 7.9 us, 4 11.7, 8 15.7, on tensor cores 13.6; H
// 7168, I 2048: 21.9, 30.5, 36.5, and 32.4).
constexpr int kFfnRows = 4;
constexpr size_t kFfnRowsSmem = 110 * 1024;  // two CTAs an SM
struct FfnRowsParams {
  int T, K, N;
  int most_rows;       // of K in a CTA
  const void *in, *W, *W3;
  void* out;
};
bool ffn_rows_take(int T, int H, int I);
cudaError_t launch_ffn_rows(int T, int H, int I, const void* x, const void* W1, const void* W3, const void* W2, float* a,
                            void* out, cudaStream_t st);

}  // namespace mok

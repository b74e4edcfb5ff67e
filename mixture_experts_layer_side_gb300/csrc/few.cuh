// The layer for a few tokens (few.cu), shared declarations.
#pragma once

#include "mok_internal.cuh"

namespace mok {

struct FewLayout {
  size_t header;   // int32 [kHeaderWords]: word 0 the error bits
  size_t logits;   // f32 [T, E] router logits
  size_t xq, xsf;  // MXFP8: codes [T, H] and scales [T, H/32] of x
  size_t a, asf;   // bf16 [T*k, I]; MXFP8: codes, and scales [T*k, I/32]
  size_t total;
};
FewLayout few_layout(const mok_shape& s, mok_precision prec);

struct FewParams {
  int T, H, I, E, k;
  int32_t* hdr;
  const __nv_bfloat16* x;
  const int32_t* idx;
  const float* scores;
  // weights: bf16, or E4M3 codes with E8M0 scales sf*
  const void *W1, *W3, *W2;
  const uint8_t *sf1, *sf3, *sf2;
  __nv_bfloat16* out;
  uint8_t *xq, *xsf;
  void* a;
  uint8_t* asf;
  // router (Wr null: the routing is given)
  const __nv_bfloat16* Wr;
  const float* bias;
  float* logits;
  int32_t* idx_out;
  float* scores_out;
};

// Enqueues one pass; *launches gets the number of kernels.
cudaError_t launch_few(const FewParams& p, bool mx, int* launches, cudaStream_t st);

}  // namespace mok

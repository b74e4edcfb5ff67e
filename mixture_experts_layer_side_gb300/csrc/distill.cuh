// Distillation loss from a teacher's top logits (distill.cu), shared declarations.
#pragma once

#include "mok_internal.cuh"

namespace mok {

struct DistillParams {
  int T, V, K;
  const void* z;   // [T, ldz] logits, bf16 or f32
  long ldz;
  const int32_t* ids;
  const float* vals;
  float tau, inv_tau;
  const float* lse_in;  // backward alone
  const float* dloss;
  float* loss;
  float* lse;        // may be null in the step
  float2* sums;      // [T] largest logit and sum of the row, for a step in two launches; else null
  void* dz;        // [T, lddz]
  long lddz;
  int in_place;    // the gradient's rows lie where the logits are
  int32_t* hdr;
};

// what one call computes
enum DistillMode : int { DISTILL_FORWARD = 0, DISTILL_BACKWARD = 1, DISTILL_STEP = 2 };
cudaError_t launch_distill(DistillMode mode, mok_dtype type, const DistillParams& p, int* launches, cudaStream_t st);

}  // namespace mok

// The layer for a few tokens (few.cu), shared declarations.
#pragma once

#include "mok_internal.cuh"

namespace mok {

// Tokens side by side in one tile (the N of its MMAs); an expert with more
// rows takes several units.
inline int few_unit_rows(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }

// The counters' place and number depend on H, I, E and k alone, so that a
// workspace serves calls of fewer tokens: every counter is zero between calls.
struct FewLayout {
  size_t header;   // int32 [kHeaderWords]: word 0 the error bits
  size_t tiles;    // int32 [units, I/128]: arrivals at the tiles of a
  size_t logits;   // f32 [parts, T, E] router logits, in parts along H (room for any smaller T's)
  size_t xq, xsf;  // MXFP8: codes [T, H] and scales [T, H/32] of x
  size_t a, asf;   // bf16 [2][T*k, I] (a, and what its rounding left); MXFP8: codes, and scales [T*k, I/32]
  size_t part;     // f32 [4 per CTA][2][unit rows][128] sums of tiles split along K
  size_t y;        // f32 [T*k, H]
  size_t total;
};
FewLayout few_layout(const mok_shape& s, mok_precision prec);

struct FewMaps {
  CUtensorMap w[3];   // W1, W3, W2
  CUtensorMap sf[3];  // MXFP8: their scales
};

// What a GEMM's cut (few.cu) has of the call's sizes.
struct FewShape {
  int group_shift, supers, kb;
};

struct FewParams {
  FewShape gemm[2];
  int T, H, I, E, k;
  int unit_rows, stages;
  int area;             // bytes of shared memory ahead of the control block: the stages, before them the router's sums
  int32_t* hdr;
  int32_t* tile_count;  // [units, I/128]
  int max_units;        // capacity of the unit table
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
  float* part;
  float* y;
  // router (Wr null: the routing is given)
  const __nv_bfloat16* Wr;
  const float* bias;
  int logit_tokens, h_parts, h_rows;  // logits: tokens side by side, parts along H, rows of Wr per part
  float* logits;
  int32_t* idx_out;
  float* scores_out;
};

// Enqueues one pass; *launches gets the number of kernels.
cudaError_t launch_few(FewParams p, bool mx, int* launches, cudaStream_t st);

}  // namespace mok

// Token embedding and its gradient (embed.cu), shared declarations.
#pragma once

#include "mok_internal.cuh"

namespace mok {

struct EmbedLayout {
  size_t header;            // int32 [kHeaderWords]: word 0 the error bits
  size_t key[2], pos[2];    // int32 [N]: (id, token) pairs between the sort's passes
  size_t part;              // f32 [2 * chunks, H]: sums of segments that cross chunks
  size_t total;
};
EmbedLayout embed_layout(int V, int H, int N);

struct EmbedParams {
  int V, H, N;
  const int32_t* ids;
  float scale;
  int32_t* hdr;
  // lookup
  const void* table;
  void* out;
  // gradient
  int32_t pad_id;
  const void* dx;
  void* dtable;
  int accumulate;
  int32_t *key[2], *pos[2];
  float* part;
};

cudaError_t launch_embed_forward(mok_dtype type, const EmbedParams& p, int* launches, cudaStream_t st);
cudaError_t launch_embed_backward(mok_dtype dx_type, mok_dtype grad_type, const EmbedParams& p, int* launches,
                                  cudaStream_t st);

}  // namespace mok

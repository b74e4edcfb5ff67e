// Top-k softmax router on either side of the layer (the selection is the
// schedule's input; "Mixture-of-Kittens (MoK)", "Use the functional API").
// The logits GEMM and the two backward GEMMs run on the tcgen05 GEMM core
// (GM_DENSE); the kernels here are the small HBM-bound steps around them:
//   pad_weights   Wr [H, E] -> [H, Epad] (zero columns up to a 128 multiple)
//   topk_softmax  per token: the k largest logit + bias keys (ties to the
//                 lower expert, descending key order), softmax over the k
//                 chosen unbiased logits
//   logit_grad    per token: dL[idx_j] = s_j (ds_j - sum_i s_i ds_i), zero
//                 elsewhere, as bf16 rows of the backward GEMMs' operand
//   take_cols     f32 [rows, Epad] -> [rows, E]
// The router gradient reaches the weights through the layer's score
// gradient ("Cursor Open-Sources Mixture-of-Kittens (MoK)", the paragraph
// after "Three design decisions that matter": router weight gradients from
// the SonicMoE-style score gradient in the SwiGLU backward).
#include "mok_internal.cuh"
#include "topk.cuh"

namespace mok {

namespace {

__global__ void __launch_bounds__(256) pad_weights_kernel(int H, int E, int Epad, const __nv_bfloat16* __restrict__ w,
                                                          __nv_bfloat16* __restrict__ wp) {
  const long n = (long)H * Epad;
  for (long i = blockIdx.x * (long)blockDim.x + threadIdx.x; i < n; i += (long)gridDim.x * blockDim.x) {
    const int h = (int)(i / Epad), e = (int)(i - (long)h * Epad);
    wp[i] = e < E ? w[(long)h * E + e] : __float2bfloat16(0.0f);
  }
}

// One warp per token.
__global__ void __launch_bounds__(256) topk_softmax_kernel(int T, int E, int Epad, int k,
                                                           const float* __restrict__ logits,
                                                           const float* __restrict__ bias, int32_t* __restrict__ idx,
                                                           float* __restrict__ scores) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= T) return;
  int e;
  float s;
  topk_softmax_warp<kMaxRouterExperts / 32>(logits + (long)t * Epad, bias, E, k, lane, e, s);
  if (lane < k) {
    idx[(long)t * k + lane] = e;
    scores[(long)t * k + lane] = s;
  }
}

// One warp per row of dL [Tpad, Epad] (rows past T are zero).
__global__ void __launch_bounds__(256) logit_grad_kernel(int T, int Tpad, int E, int Epad, int k,
                                                         const int32_t* __restrict__ idx, const float* __restrict__ s,
                                                         const float* __restrict__ ds, __nv_bfloat16* __restrict__ dl) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= Tpad) return;
  __nv_bfloat16* row = dl + (long)t * Epad;
  for (int e = lane; e < Epad; e += 32) row[e] = __float2bfloat16(0.0f);
  __syncwarp();
  if (t >= T) return;
  const float sj = lane < k ? s[(long)t * k + lane] : 0.0f;
  const float dsj = lane < k ? ds[(long)t * k + lane] : 0.0f;
  float dot = sj * dsj;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if (lane < k) {
    const int e = idx[(long)t * k + lane];
    if (e >= 0 && e < E) row[e] = __float2bfloat16(sj * (dsj - dot));
  }
}

__global__ void __launch_bounds__(256) take_cols_kernel(int rows, int E, int Epad, const float* __restrict__ src,
                                                        float* __restrict__ dst) {
  const long n = (long)rows * E;
  for (long i = blockIdx.x * (long)blockDim.x + threadIdx.x; i < n; i += (long)gridDim.x * blockDim.x) {
    const int r = (int)(i / E), e = (int)(i - (long)r * E);
    dst[i] = src[(long)r * Epad + e];
  }
}

int elementwise_grid(long items) {
  long blocks = (items + 255) / 256;
  const long cap = (long)device_sm_count() * 16;
  if (blocks > cap) blocks = cap;
  return (int)(blocks < 1 ? 1 : blocks);
}

}  // namespace

cudaError_t launch_router_pad_weights(int H, int E, int Epad, const __nv_bfloat16* w, __nv_bfloat16* wp,
                                      cudaStream_t st) {
  pad_weights_kernel<<<elementwise_grid((long)H * Epad), 256, 0, st>>>(H, E, Epad, w, wp);
  return cudaGetLastError();
}

cudaError_t launch_router_topk(int T, int E, int Epad, int k, const float* logits, const float* bias, int32_t* idx,
                               float* scores, cudaStream_t st) {
  if (E > kMaxRouterExperts || k > 32) return cudaErrorInvalidValue;
  topk_softmax_kernel<<<(T + 7) / 8, 256, 0, st>>>(T, E, Epad, k, logits, bias, idx, scores);
  return cudaGetLastError();
}

cudaError_t launch_router_logit_grad(int T, int Tpad, int E, int Epad, int k, const int32_t* idx, const float* s,
                                     const float* ds, __nv_bfloat16* dl, cudaStream_t st) {
  logit_grad_kernel<<<(Tpad + 7) / 8, 256, 0, st>>>(T, Tpad, E, Epad, k, idx, s, ds, dl);
  return cudaGetLastError();
}

cudaError_t launch_router_take_cols(int rows, int E, int Epad, const float* src, float* dst, cudaStream_t st) {
  take_cols_kernel<<<elementwise_grid((long)rows * E), 256, 0, st>>>(rows, E, Epad, src, dst);
  return cudaGetLastError();
}

}  // namespace mok

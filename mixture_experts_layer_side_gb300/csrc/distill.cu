// Distillation loss from a teacher's top logits.  For a row of V student
// logits z and the teacher's K listed (id_j, v_j), temperature tau:
//
//   p = softmax over the list of v / tau          (entries of id -1 left out)
//   lse = log sum_v exp(z_v / tau),   log q_v = z_v / tau - lse
//   loss = sum_j p_j (log p_j - log q_(id_j)) = KL(p || q)
//   dz_v = (dloss / tau) (q_v - sum_{j: id_j = v} p_j)
//
// An entry of p_j = 0 adds nothing; a row whose list is empty has loss 0 and
// gradient 0.  One CTA per row: the row's maximum and sum in one pass over
// the row, each thread keeping a running pair, joined in a fixed tree.
#include "distill.cuh"

namespace mok {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float value(const __nv_bfloat16* z, long i) { return __bfloat162float(z[i]); }
__device__ __forceinline__ float value(const float* z, long i) { return z[i]; }
__device__ __forceinline__ void put(__nv_bfloat16* z, long i, float v) { z[i] = __float2bfloat16(v); }
__device__ __forceinline__ void put(float* z, long i, float v) { z[i] = v; }

// (m, s) stands for s * exp(m); -inf, 0 for nothing
__device__ __forceinline__ void join(float& m, float& s, float mo, float so) {
  const float top = fmaxf(m, mo);
  const float base = top == -INFINITY ? 0.0f : top;
  s = s * expf(m - base) + so * expf(mo - base);
  m = top;
}

template <typename F>
__device__ __forceinline__ float block_reduce(float v, float* red, F f) {
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < kWarps; ++i) v = f(v, red[i]);
  return v;
}

struct Row {
  int32_t ids[MOK_DISTILL_MAX_TOP];
  float p[MOK_DISTILL_MAX_TOP];
  float red[kWarps], red2[kWarps];
};

// The teacher's list in shared memory; returns the sum of p (1, or 0 for an
// empty list).  Thread j holds entry j; log_p of its own entry.
__device__ float load_list(const DistillParams& q, long t, Row& r, float& p, float& log_p) {
  const int j = threadIdx.x;
  int id = -1;
  float v = -INFINITY;
  if (j < q.K) {
    id = q.ids[t * q.K + j];
    if (id >= q.V || id < -1) {
      atomicOr(q.hdr + kHdrError, MOK_ERRBIT_BAD_INDEX);
      id = -1;
    }
    if (id >= 0) v = q.vals[t * q.K + j] * q.inv_tau;
  }
  const float top = block_reduce(v, r.red, [](float a, float b) { return fmaxf(a, b); });
  const float base = top == -INFINITY ? 0.0f : top;
  const float e = id >= 0 ? expf(v - base) : 0.0f;
  const float total = block_reduce(e, r.red, [](float a, float b) { return a + b; });
  p = total > 0.0f || isnan(total) ? e / total : 0.0f;
  log_p = p > 0.0f ? logf(p) : 0.0f;
  if (j < q.K) {
    r.ids[j] = id;
    r.p[j] = p;
  }
  __syncthreads();
  return total > 0.0f || isnan(total) ? 1.0f : 0.0f;
}

template <typename Z>
__global__ void __launch_bounds__(kThreads) distill_forward_kernel(DistillParams q) {
  __shared__ Row r;
  const long t = blockIdx.x;
  const Z* z = static_cast<const Z*>(q.z) + t * q.ldz;
  float p, log_p;
  load_list(q, t, r, p, log_p);
  float m = -INFINITY, s = 0.0f;
  for (int v = threadIdx.x; v < q.V; v += kThreads) join(m, s, value(z, v) * q.inv_tau, 1.0f);
  for (int o = 16; o > 0; o >>= 1) {
    const float mo = __shfl_xor_sync(0xffffffffu, m, o), so = __shfl_xor_sync(0xffffffffu, s, o);
    join(m, s, mo, so);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    r.red[threadIdx.x >> 5] = m;
    r.red2[threadIdx.x >> 5] = s;
  }
  __syncthreads();
  m = r.red[0];
  s = r.red2[0];
  for (int i = 1; i < kWarps; ++i) join(m, s, r.red[i], r.red2[i]);
  const float lse = m + logf(s);
  float l = 0.0f;
  if (p > 0.0f || isnan(p)) l = p * (log_p - (value(z, r.ids[threadIdx.x]) * q.inv_tau - lse));
  l = block_reduce(l, r.red, [](float a, float b) { return a + b; });
  if (threadIdx.x == 0) {
    q.loss[t] = l;
    q.lse[t] = lse;
  }
}

template <typename Z>
__global__ void __launch_bounds__(kThreads) distill_backward_kernel(DistillParams q) {
  __shared__ Row r;
  const long t = blockIdx.x;
  const Z* z = static_cast<const Z*>(q.z) + t * q.ldz;
  Z* dz = static_cast<Z*>(q.dz) + t * q.lddz;
  float p, log_p;
  const float any = load_list(q, t, r, p, log_p);
  if (any == 0.0f) {
    for (int v = threadIdx.x; v < q.V; v += kThreads) put(dz, v, 0.0f);
    return;
  }
  const float lse = q.lse_in[t], g = q.dloss[t] * q.inv_tau;
  // the listed columns: this thread's, if it is the first of its id
  const int id = threadIdx.x < q.K ? r.ids[threadIdx.x] : -1;
  float at = 0.0f;
  bool mine = id >= 0;
  if (mine) {
    float sum = 0.0f;
    for (int j = 0; j < q.K; ++j)
      if (r.ids[j] == id) {
        sum += r.p[j];
        mine = mine && j >= (int)threadIdx.x;
      }
    at = g * (expf(value(z, id) * q.inv_tau - lse) - sum);
  }
  __syncthreads();  // the listed logits are read before a gradient in their place overwrites them
  for (int v = threadIdx.x; v < q.V; v += kThreads) put(dz, v, g * expf(value(z, v) * q.inv_tau - lse));
  __syncthreads();
  if (mine) put(dz, id, at);
}

template <typename Z>
cudaError_t launch(DistillMode mode, DistillParams p, int* launches, cudaStream_t st) {
  *launches = 0;
  if (mode != DISTILL_BACKWARD) {
    distill_forward_kernel<Z><<<p.T, kThreads, 0, st>>>(p);
    *launches += 1;
  }
  if (mode != DISTILL_FORWARD) {
    if (mode == DISTILL_STEP) p.lse_in = p.lse;
    distill_backward_kernel<Z><<<p.T, kThreads, 0, st>>>(p);
    *launches += 1;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_distill(DistillMode mode, mok_dtype type, const DistillParams& p, int* launches, cudaStream_t st) {
  return type == MOK_TYPE_BF16 ? launch<__nv_bfloat16>(mode, p, launches, st) : launch<float>(mode, p, launches, st);
}

}  // namespace mok

// The dense gated feed-forward block for a token or a few (T <= kFfnRows):
// two products of a few rows with a large matrix, bound by the read of the
// weights.  No tensor core: a weight is used once a token, and what counts is
// that every SM has enough of the read on its way from the first moment on.
//
// A cluster of CTAs has 128 columns of the result (gate: 64 of h and the same
// of u), each CTA a range of K, whose rows its 16 half-warps take in turn:
// 16 lanes read 256 bytes of a row, eight rows ahead.  The half-warps' sums
// meet in shared memory, the CTAs' through the cluster's, and every CTA
// finishes a share of the columns.  All sums are f32 and in a fixed order; a
// stays f32 between the two launches, of which the second starts beside the
// first.
//
// 1 token, H 7168, I 2048: 21.9 us, 4.0 TB/s of weights (13.0 at the rate of a
// copy; the rest is two starts, the joins and the second launch's wait).  On
// tensor cores (ffn.cu) it takes 32.4, through the routed few-token kernel
// with one expert 30.
#include <algorithm>
#include <atomic>

#include "ffn.cuh"
#include "tc.cuh"

namespace mok {

namespace {

constexpr int kRowThreads = 256;
constexpr int kWorkers = kRowThreads / 16;  // half-warps
constexpr int kCols = 128;                  // columns of a cluster: eight a lane
constexpr int kRowsAhead = 8;

typedef unsigned long long f2;
__device__ __forceinline__ f2 pair2(float a, float b) {
  f2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
__device__ __forceinline__ float ld_cluster(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// TM: room for tokens.  GATE: in is x (bf16) [T, K], the weights W1 and W3, out a (f32) [T, N]; otherwise in is a, the
// weights W2, out bf16 [T, N].
template <int TM, bool GATE>
__global__ void __launch_bounds__(kRowThreads, 2) ffn_rows_kernel(const FfnRowsParams p) {
  extern __shared__ float shared[];
  const int t = threadIdx.x, worker = t >> 4, lane = t & 15;
  const int ctas = (int)gridDim.y, cta = blockIdx.y;  // a cluster's, along K
  const int k0 = (int)((long)p.K * cta / ctas), rows = (int)((long)p.K * (cta + 1) / ctas) - k0;
  float* x = shared;  // [rows][TM]
  float* sums = shared + (size_t)p.most_rows * TM;  // [kWorkers][TM][kCols]
  // this lane's eight columns of the weight, and of the sums
  const int col = GATE ? blockIdx.x * (kCols / 2) + (lane & 7) * 8 : blockIdx.x * kCols + lane * 8;
  const bool in = col < p.N;
  const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(GATE && lane >= 8 ? p.W3 : p.W) + (long)k0 * p.N + (in ? col : 0);

  uint4 ahead[kRowsAhead];
  auto fetch = [&](int r) {
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
      const int row = r + i * kWorkers;
      if (in && row < rows) ahead[i] = __ldcs(reinterpret_cast<const uint4*>(w + (long)row * p.N));
    }
  };
  fetch(worker);  // (weights wait for no one)
  if (!GATE) griddep_wait();
  for (int i = t; i < rows * TM; i += kRowThreads) {
    const int r = i / TM, token = i - r * TM;
    float v = 0.0f;
    if (token < p.T) {
      const long at = (long)token * p.K + k0 + r;
      v = GATE ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.in)[at]) : __ldcg(static_cast<const float*>(p.in) + at);
    }
    x[i] = v;
  }
  __syncthreads();
  f2 acc[TM][4];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = 0;
  for (int r = worker; r < rows; r += kRowsAhead * kWorkers) {
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
      const int row = r + i * kWorkers;
      if (row >= rows) break;
      const uint32_t u[4] = {ahead[i].x, ahead[i].y, ahead[i].z, ahead[i].w};
      f2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = pair2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
      const int coming = row + kRowsAhead * kWorkers;
      if (in && coming < rows) ahead[i] = __ldcs(reinterpret_cast<const uint4*>(w + (long)coming * p.N));
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        const float f = x[row * TM + m];
        const f2 ff = pair2(f, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][j] = fma2(ff, v[j], acc[m][j]);
      }
    }
  }
  if (GATE) griddep_launch_dependents();
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    f2* to = reinterpret_cast<f2*>(sums + (worker * TM + m) * kCols + lane * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) to[j] = in ? acc[m][j] : 0;
  }
  __syncthreads();
  // the CTA's sums, where its first worker's were
  for (int i = t; i < TM * kCols; i += kRowThreads) {
    float v = sums[i];
#pragma unroll
    for (int k = 1; k < kWorkers; ++k) v += sums[k * TM * kCols + i];
    sums[i] = v;
  }
  __syncwarp();  // (the cluster's barrier is of the aligned form)
  cluster_sync();
  // each CTA finishes every ctas-th result
  constexpr int kResults = GATE ? kCols / 2 : kCols;
  for (int i = t * ctas + cta; i < TM * kResults; i += kRowThreads * ctas) {
    const int m = i / kResults, c = i - m * kResults;
    const int n = blockIdx.x * kResults + c;
    if (m >= p.T || n >= p.N) continue;
    float h = 0.0f, u = 0.0f;
    for (int k = 0; k < ctas; ++k) {
      h += ld_cluster(mapa_shared(sums + m * kCols + c, (uint32_t)k));
      if (GATE) u += ld_cluster(mapa_shared(sums + m * kCols + kResults + c, (uint32_t)k));
    }
    if (GATE) static_cast<float*>(p.out)[(long)m * p.N + n] = h / (1.0f + __expf(-h)) * u;
    else static_cast<__nv_bfloat16*>(p.out)[(long)m * p.N + n] = __float2bfloat16_rn(h);
  }
  __syncwarp();
  cluster_sync();  // (no CTA leaves while another reads its sums)
}

// Rows of K that a CTA has at most, in whole fours (what follows them in shared memory stands on a boundary of sixteen).
int rows_of_cta(int K, int ctas) { return ((K + ctas - 1) / ctas + 3) / 4 * 4; }

size_t rows_smem(int most_rows, int tm) { return (size_t)(most_rows + kWorkers * kCols) * tm * 4; }

// CTAs of a cluster: enough for two on every SM, of 64 rows of K at least.
int rows_ctas(int K, int blocks, int sms) {
  int c = 1;
  while (c < 8 && blocks * c * 2 <= 2 * sms && K / (2 * c) >= 64) c *= 2;
  return c;
}

template <int TM, bool GATE>
cudaError_t launch_rows(FfnRowsParams p, cudaStream_t st) {
  const int blocks = GATE ? (p.N + kCols / 2 - 1) / (kCols / 2) : (p.N + kCols - 1) / kCols;
  const int ctas = rows_ctas(p.K, blocks, device_sm_count());
  p.most_rows = rows_of_cta(p.K, ctas);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem((const void*)ffn_rows_kernel<TM, GATE>, kFfnRowsSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = (unsigned)ctas;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)ctas);
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = rows_smem(p.most_rows, TM);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = GATE ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, ffn_rows_kernel<TM, GATE>, p);
}

template <int TM>
cudaError_t run_rows(const FfnRowsParams& gate, const FfnRowsParams& out, cudaStream_t st) {
  const cudaError_t e = launch_rows<TM, true>(gate, st);
  return e == cudaSuccess ? launch_rows<TM, false>(out, st) : e;
}

}  // namespace

bool ffn_rows_take(int T, int H, int I) {
  // (K of either product; a range of it and the half-warps' sums lie in shared memory)
  const int sms = device_sm_count(), tm = T <= 1 ? 1 : T <= 2 ? 2 : 4;
  if (T > kFfnRows || sms == 0) return false;
  const int g = rows_ctas(H, (I + kCols / 2 - 1) / (kCols / 2), sms), o = rows_ctas(I, (H + kCols - 1) / kCols, sms);
  return rows_smem(rows_of_cta(H, g), tm) <= kFfnRowsSmem && rows_smem(rows_of_cta(I, o), tm) <= kFfnRowsSmem;
}

cudaError_t launch_ffn_rows(int T, int H, int I, const void* x, const void* W1, const void* W3, const void* W2, float* a,
                            void* out, cudaStream_t st) {
  const FfnRowsParams gate = {T, H, I, 0, x, W1, W3, a}, second = {T, I, H, 0, a, W2, nullptr, out};
  if (T <= 1) return run_rows<1>(gate, second, st);
  if (T <= 2) return run_rows<2>(gate, second, st);
  return run_rows<4>(gate, second, st);
}

}  // namespace mok

// The layer for a few tokens (T <= MOK_FEW_MAX_TOKENS): routed SwiGLU experts
// and combine, with or without the router, for serving steps.
//
//   h = x_t W1_e,  u = x_t W3_e,  a = silu(h) * u,  y = a W2_e,  e = idx[t, j]
//   out_t = sum_j s[t, j] y_(t, j)
//
// One thread per output column walks the contraction: consecutive threads
// read consecutive columns of a weight row.
#include <cuda_fp8.h>

#include "few.cuh"
#include "mx.cuh"

namespace mok {

namespace {

__device__ __forceinline__ float e4m3_value(uint8_t q) {
  __nv_fp8_e4m3 v;
  v.__x = q;
  return static_cast<float>(v);
}

// E8M0 scale: 2^(code - 127); 2^-127 is a subnormal float
__device__ __forceinline__ float e8m0_value(uint8_t s) {
  return s ? __int_as_float((int)s << 23) : __int_as_float(0x00400000);
}

// MXFP8: x [T, H] as the values its quantisation along H stands for.
__global__ void few_quant_x_kernel(int nblocks, const __nv_bfloat16* __restrict__ x, uint8_t* __restrict__ q,
                                   uint8_t* __restrict__ sf) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= nblocks) return;
  float v[32];
  for (int i = 0; i < 32; ++i) v[i] = __bfloat162float(x[(long)b * 32 + i]);
  uint32_t codes[8];
  sf[b] = mx_quant32(v, codes);
  for (int i = 0; i < 8; ++i) reinterpret_cast<uint32_t*>(q + (long)b * 32)[i] = codes[i];
}

template <bool MX>
__device__ __forceinline__ float row_value(const void* rows, const uint8_t* sf, long row, int K, int i) {
  if (MX)
    return e4m3_value(static_cast<const uint8_t*>(rows)[row * K + i]) * e8m0_value(sf[row * (K / 32) + i / 32]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(rows)[row * K + i]);
}

template <bool MX>
__device__ __forceinline__ float weight_value(const void* w, const uint8_t* sf, long e, int K, int N, int i, int n) {
  if (MX)
    return e4m3_value(static_cast<const uint8_t*>(w)[(e * K + i) * N + n]) *
           e8m0_value(sf[(e * (K / 32) + i / 32) * N + n]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[(e * K + i) * N + n]);
}

// a of one routed row f and 128 intermediate columns
template <bool MX>
__global__ void __launch_bounds__(128) few_hidden_kernel(FewParams p) {
  const int f = blockIdx.y, n = blockIdx.x * 128 + threadIdx.x;
  const int e = p.idx[f];
  if (e < 0 || e >= p.E) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(p.hdr + kHdrError, MOK_ERRBIT_BAD_INDEX);
    return;
  }
  const long t = f / p.k;
  float h = 0.0f, u = 0.0f;
  for (int i = 0; i < p.H; ++i) {
    const float xv = row_value<MX>(MX ? (const void*)p.xq : p.x, p.xsf, t, p.H, i);
    h = fmaf(xv, weight_value<MX>(p.W1, p.sf1, e, p.H, p.I, i, n), h);
    u = fmaf(xv, weight_value<MX>(p.W3, p.sf3, e, p.H, p.I, i, n), u);
  }
  const float a = h / (1.0f + __expf(-h)) * u;
  if (MX) {
    // a warp's 32 columns are one block
    const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(a))));
    const int X = mx_block_exponent(amax);
    static_cast<uint8_t*>(p.a)[(long)f * p.I + n] = (uint8_t)mx_cvt_e4m3x2(a * mx_exp2_int(-X), 0.0f);
    if ((threadIdx.x & 31) == 0) p.asf[(long)f * (p.I / 32) + n / 32] = (uint8_t)(X + 127);
  } else {
    static_cast<__nv_bfloat16*>(p.a)[(long)f * p.I + n] = __float2bfloat16(a);
  }
}

// out of one token and 128 columns: y of its k experts, combined in f32 in
// increasing j and rounded once
template <bool MX>
__global__ void __launch_bounds__(128) few_out_kernel(FewParams p) {
  const int t = blockIdx.y, n = blockIdx.x * 128 + threadIdx.x;
  float acc = 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const long f = (long)t * p.k + j;
    const int e = p.idx[f];
    if (e < 0 || e >= p.E) continue;
    float y = 0.0f;
    for (int i = 0; i < p.I; ++i)
      y = fmaf(row_value<MX>(p.a, p.asf, f, p.I, i), weight_value<MX>(p.W2, p.sf2, e, p.I, p.H, i, n), y);
    acc = fmaf(p.scores[f], y, acc);
  }
  p.out[(long)t * p.H + n] = __float2bfloat16(acc);
}

// Router logits of one token: a warp per 32 experts, x row and Wr column-wise.
__global__ void __launch_bounds__(256) few_logits_kernel(FewParams p) {
  const int t = blockIdx.y, e = blockIdx.x * 256 + threadIdx.x;
  if (e >= p.E) return;
  float l = 0.0f;
  for (int i = 0; i < p.H; ++i)
    l = fmaf(__bfloat162float(p.x[(long)t * p.H + i]), __bfloat162float(p.Wr[(long)i * p.E + e]), l);
  p.logits[(long)t * p.E + e] = l;
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace

FewLayout few_layout(const mok_shape& s, mok_precision prec) {
  FewLayout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  const size_t R = (size_t)s.T * s.k;
  L.header = take(kHeaderWords * 4);
  L.logits = take((size_t)s.T * s.E * 4);
  L.xq = prec == MOK_MXFP8 ? take((size_t)s.T * s.H) : 0;
  L.xsf = prec == MOK_MXFP8 ? take((size_t)s.T * (s.H / 32)) : 0;
  L.a = take(R * s.I * (prec == MOK_MXFP8 ? 1 : 2));
  L.asf = prec == MOK_MXFP8 ? take(R * (s.I / 32)) : 0;
  L.total = off;
  return L;
}

cudaError_t launch_few(const FewParams& p, bool mx, int* launches, cudaStream_t st) {
  int n = 0;
  if (p.Wr) {
    few_logits_kernel<<<dim3((p.E + 255) / 256, p.T), 256, 0, st>>>(p);
    cudaError_t e = launch_router_topk(p.T, p.E, p.E, p.k, p.logits, p.bias, p.idx_out, p.scores_out, st);
    if (e != cudaSuccess) return e;
    n += 2;
  }
  const dim3 g1(p.I / 128, p.T * p.k), g2(p.H / 128, p.T);
  if (mx) {
    const int nb = p.T * (p.H / 32);
    few_quant_x_kernel<<<(nb + 127) / 128, 128, 0, st>>>(nb, p.x, p.xq, p.xsf);
    few_hidden_kernel<true><<<g1, 128, 0, st>>>(p);
    few_out_kernel<true><<<g2, 128, 0, st>>>(p);
    n += 3;
  } else {
    few_hidden_kernel<false><<<g1, 128, 0, st>>>(p);
    few_out_kernel<false><<<g2, 128, 0, st>>>(p);
    n += 2;
  }
  *launches = n;
  return cudaGetLastError();
}

}  // namespace mok

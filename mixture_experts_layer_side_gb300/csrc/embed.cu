// Token embedding and its gradient.
//
//   x_n = scale * table[id_n]
//   dtable_v = scale * sum of dx_n over the tokens n with id_n = v, in
//   ascending n (f32), rounded once; added to dtable_v when accumulating
//
// The gradient goes by tokens sorted by id: a stable radix sort of (id,
// token) pairs, then sums over runs of equal ids.  No float atomics: the
// order of each sum is fixed by the input.
//
// The sort is one cluster of kSortCtas CTAs: the pairs of a few thousand to
// a few million tokens are small beside dx, and a cluster's barriers and
// distributed shared memory join its histograms without a launch or a
// device-wide barrier per pass.
#include <cooperative_groups.h>

#include "embed.cuh"

namespace mok {

namespace cg = cooperative_groups;

namespace {

constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigits = 1024;
constexpr int kChunk = 32;  // sorted tokens per summing block

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

template <typename T>
__global__ void __launch_bounds__(256) embed_lookup_kernel(EmbedParams p) {
  const int n = blockIdx.x;
  const int id = p.ids[n];
  const bool ok = id >= 0 && id < p.V;
  if (!ok && id != p.pad_id && threadIdx.x == 0) atomicOr(p.hdr + kHdrError, MOK_ERRBIT_BAD_INDEX);
  const T* src = static_cast<const T*>(p.table) + (long)(ok ? id : 0) * p.H;
  T* dst = static_cast<T*>(p.out) + (long)n * p.H;
  for (int c = threadIdx.x; c < p.H; c += 256) put(dst + c, ok ? p.scale * to_f(src[c]) : 0.0f);
}

// Stable least-significant-digit radix sort of the tokens by id; a token
// that takes no part (padding, or an id outside [0, V)) gets key V and goes
// last.  `bits` per pass, `passes` passes; the sorted pairs end in key/pos
// [passes & 1].  Warp w of CTA r owns the contiguous range w of range r, so
// (CTA, warp, place in the range) is the order of the pairs.
__global__ void __launch_bounds__(kSortThreads) __cluster_dims__(kSortCtas, 1, 1)
    embed_sort_kernel(EmbedParams p, int bits, int passes) {
  extern __shared__ int sm[];
  int* hist = sm;                                // [kSortWarps][digits]
  const int digits = 1 << bits;
  int* tot = hist + kSortWarps * digits;         // [digits] this CTA's counts
  int* warp_sum = tot + digits;                  // [kSortWarps]
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // ranges in whole groups of 32 pairs
  const int groups = (p.N + 31) / 32;
  const int per_warp = (groups + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps);
  const long first = (long)(rank * kSortWarps + warp) * per_warp * 32;
  const long last = first + (long)per_warp * 32 < p.N ? first + (long)per_warp * 32 : p.N;

  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * bits;
    const int32_t* kin = p.key[pass & 1];
    const int32_t* pin = p.pos[pass & 1];
    int32_t* kout = p.key[(pass + 1) & 1];
    int32_t* pout = p.pos[(pass + 1) & 1];
    auto key_at = [&](long i) {
      if (pass > 0) return kin[i];
      const int id = p.ids[i];
      if (id == p.pad_id) return p.V;
      if (id < 0 || id >= p.V) {
        atomicOr(p.hdr + kHdrError, MOK_ERRBIT_BAD_INDEX);
        return p.V;
      }
      return id;
    };
    for (int d = threadIdx.x; d < kSortWarps * digits; d += kSortThreads) hist[d] = 0;
    __syncthreads();
    int* mine = hist + warp * digits;
    for (long i = first + lane; i - lane < last; i += 32) {
      const bool in = i < last;
      const int d = in ? (key_at(i) >> shift) & (digits - 1) : digits;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      if (in && (same & ((1u << lane) - 1u)) == 0) mine[d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    // exclusive sums over the warps, and the CTA's totals
    for (int d = threadIdx.x; d < digits; d += kSortThreads) {
      int run = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = hist[w * digits + d];
        hist[w * digits + d] = run;
        run += c;
      }
      tot[d] = run;
    }
    cluster.sync();
    // digits is at most the number of threads: thread d holds digit d
    int all = 0, before = 0;
    if (threadIdx.x < digits)
      for (int r = 0; r < kSortCtas; ++r) {
        const int c = cluster.map_shared_rank(tot, r)[threadIdx.x];
        if (r < rank) before += c;
        all += c;
      }
    int incl = all;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int base = incl - all + before;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    if (threadIdx.x < digits)
      for (int w = 0; w < kSortWarps; ++w) hist[w * digits + threadIdx.x] += base;
    __syncthreads();
    for (long i = first + lane; i - lane < last; i += 32) {
      const bool in = i < last;
      const int k = in ? key_at(i) : 0;
      const int d = in ? (k >> shift) & (digits - 1) : digits;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      const int ahead = __popc(same & ((1u << lane) - 1u));
      int at = 0;
      if (in) at = mine[d] + ahead;
      __syncwarp();
      if (in && ahead == 0) mine[d] += __popc(same);
      __syncwarp();
      if (in) {
        kout[at] = k;
        pout[at] = pass > 0 ? pin[i] : (int32_t)i;
      }
    }
    // the pass's pairs are visible to the whole cluster, and no CTA's counts
    // are overwritten while another still reads them
    cluster.sync();
  }
}

// One block sums a chunk of kChunk sorted tokens over a slab of columns.  A
// run of equal ids inside the chunk is finished here; one that crosses the
// chunk's start or end leaves its part in part[2c] (the run that began
// earlier) or part[2c + 1] (the one that began here and goes on).
template <typename D, typename G>
__global__ void __launch_bounds__(256) embed_sum_kernel(EmbedParams p, const int32_t* __restrict__ key,
                                                        const int32_t* __restrict__ pos) {
  const int c0 = blockIdx.x * kChunk;
  const int n = min(kChunk, p.N - c0);
  const int col = blockIdx.y * 256 + threadIdx.x;
  if (col >= p.H || key[c0] >= p.V) return;
  const bool from_before = c0 > 0 && key[c0 - 1] == key[c0];
  float acc = 0.0f;
  bool began_before = from_before;
  for (int i = 0; i < n; ++i) {
    const int k = key[c0 + i];
    if (k >= p.V) break;
    acc += to_f(static_cast<const D*>(p.dx)[(long)pos[c0 + i] * p.H + col]);
    const bool goes_on = c0 + i + 1 < p.N && key[c0 + i + 1] == k;
    if (goes_on && i + 1 < n) continue;
    if (began_before)
      p.part[(long)(2 * blockIdx.x) * p.H + col] = acc;
    else if (goes_on)
      p.part[(long)(2 * blockIdx.x + 1) * p.H + col] = acc;
    else {
      G* g = static_cast<G*>(p.dtable) + (long)k * p.H + col;
      put(g, p.accumulate ? fmaf(p.scale, acc, to_f(*g)) : p.scale * acc);
    }
    acc = 0.0f;
    began_before = false;
  }
}

// Joins the runs that cross chunks: the block of the chunk where such a run
// began adds its parts in order.
template <typename G>
__global__ void __launch_bounds__(256) embed_join_kernel(EmbedParams p, const int32_t* __restrict__ key) {
  const int c0 = blockIdx.x * kChunk;
  const int end = c0 + kChunk;
  if (end >= p.N) return;
  const int k = key[end - 1];
  // a run that goes on past this chunk, and began in it
  if (k >= p.V || key[end] != k || (key[c0] == k && c0 > 0 && key[c0 - 1] == k)) return;
  const int col = blockIdx.y * 256 + threadIdx.x;
  if (col >= p.H) return;
  float acc = p.part[(long)(2 * blockIdx.x + 1) * p.H + col];
  for (int c = blockIdx.x + 1; c * kChunk < p.N && key[c * kChunk] == k; ++c) acc += p.part[(long)(2 * c) * p.H + col];
  G* g = static_cast<G*>(p.dtable) + (long)k * p.H + col;
  put(g, p.accumulate ? fmaf(p.scale, acc, to_f(*g)) : p.scale * acc);
}

template <typename D, typename G>
cudaError_t launch_backward(const EmbedParams& p, int* launches, cudaStream_t st) {
  *launches = 0;
  if (!p.accumulate) {
    const cudaError_t e = cudaMemsetAsync(p.dtable, 0, (size_t)p.V * p.H * sizeof(G), st);
    if (e != cudaSuccess) return e;
  }
  if (p.N == 0) return cudaSuccess;
  // keys are 0 .. V
  int key_bits = 1;
  while (key_bits < 31 && (1 << key_bits) <= p.V) ++key_bits;
  const int passes = (key_bits + 9) / 10, bits = (key_bits + passes - 1) / passes;
  const size_t smem = ((size_t)(kSortWarps + 1) * (1 << bits) + kSortWarps) * 4;
  cudaError_t e =
      cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)(((size_t)(kSortWarps + 1) * kMaxDigits + kSortWarps) * 4));
  if (e != cudaSuccess) return e;
  embed_sort_kernel<<<kSortCtas, kSortThreads, smem, st>>>(p, bits, passes);
  const dim3 grid((p.N + kChunk - 1) / kChunk, (p.H + 255) / 256);
  embed_sum_kernel<D, G><<<grid, 256, 0, st>>>(p, p.key[passes & 1], p.pos[passes & 1]);
  embed_join_kernel<G><<<grid, 256, 0, st>>>(p, p.key[passes & 1]);
  *launches = 3;
  return cudaGetLastError();
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace

EmbedLayout embed_layout(int V, int H, int N) {
  (void)V;
  EmbedLayout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  L.header = take(kHeaderWords * 4);
  for (int i = 0; i < 2; ++i) {
    L.key[i] = take((size_t)N * 4);
    L.pos[i] = take((size_t)N * 4);
  }
  L.part = take((size_t)((N + kChunk - 1) / kChunk) * 2 * H * 4);
  L.total = off;
  return L;
}

cudaError_t launch_embed_forward(mok_dtype type, const EmbedParams& p, int* launches, cudaStream_t st) {
  *launches = 0;
  if (p.N == 0) return cudaSuccess;
  if (type == MOK_TYPE_BF16)
    embed_lookup_kernel<__nv_bfloat16><<<p.N, 256, 0, st>>>(p);
  else
    embed_lookup_kernel<float><<<p.N, 256, 0, st>>>(p);
  *launches = 1;
  return cudaGetLastError();
}

cudaError_t launch_embed_backward(mok_dtype dx_type, mok_dtype grad_type, const EmbedParams& p, int* launches,
                                  cudaStream_t st) {
  if (dx_type == MOK_TYPE_BF16)
    return grad_type == MOK_TYPE_BF16 ? launch_backward<__nv_bfloat16, __nv_bfloat16>(p, launches, st)
                                      : launch_backward<__nv_bfloat16, float>(p, launches, st);
  return grad_type == MOK_TYPE_BF16 ? launch_backward<float, __nv_bfloat16>(p, launches, st)
                                    : launch_backward<float, float>(p, launches, st);
}

}  // namespace mok

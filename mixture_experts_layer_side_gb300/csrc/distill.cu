// Distillation loss from a teacher's top logits.  For a row of V student
// logits z and the teacher's K listed (id_j, v_j), temperature tau:
//
//   p = softmax over the list of v / tau          (entries of id -1 left out)
//   lse = log sum_v exp(z_v / tau),   log q_v = z_v / tau - lse
//   loss = sum_j p_j (log p_j - log q_(id_j)) = KL(p || q)
//   dz_v = (dloss / tau) (q_v - sum_{j: id_j = v} p_j)
//
// An entry of p_j = 0 adds nothing; a row whose list is empty has loss 0 and
// gradient 0.  Every operation is bound by the row's bytes: the forward reads
// it once, the backward reads and writes it once, and the step, which needs
// the row's sum before it can write, keeps the row on the chip in between:
//
//  * Rows are read in 16-byte vectors of the address grid (a row of any
//    alignment has at most one part-filled vector at each end).
//  * Each thread keeps a running maximum m and sum of exp2((z - m) c), c =
//    log2(e) / tau; threads, warps and CTAs join theirs in a fixed tree.
//  * A row is shared by a cluster of up to 8 CTAs, which exchange their
//    (m, sum) through distributed shared memory: a few rows still fill the
//    GPU.  In the step a CTA brings its share, 32 KB where eight are enough,
//    to shared memory with bulk copies, where it stays between the sum and the
//    gradient; seven such CTAs an SM are in different phases, so that loads
//    and stores overlap.  (Shares held in registers let two CTAs an SM run:
//    876 us for 4,096 rows of 131,072 bf16.)
//  * The teacher's list (at most MOK_DISTILL_MAX_TOP entries) is a warp's
//    work, hidden behind the row's loads.  Listed columns are stored after
//    the rest of their vectors, by the thread that is the first with that id.
//
// Rows too long for eight CTAs' shared memory (more than about 800,000 bf16)
// take the forward and then the backward.
#include <cooperative_groups.h>

#include "distill.cuh"
#include "tc.cuh"

namespace mok {

namespace cg = cooperative_groups;

namespace {

constexpr int kMaxShare = 8;  // CTAs a row
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Vectors of a type: 16 bytes.
template <typename Z>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float top(const uint4& v) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ float value(__nv_bfloat16 z) { return __bfloat162float(z); }
  static __device__ __forceinline__ __nv_bfloat16 from(float f) { return __float2bfloat16(f); }
  static __device__ __forceinline__ uint4 lowest() { return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float top(const uint4& v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static __device__ __forceinline__ float value(float z) { return z; }
  static __device__ __forceinline__ float from(float f) { return f; }
  static __device__ __forceinline__ uint4 lowest() { return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u); }
};

// A row on the grid of 16-byte vectors: vector i holds elements
// [i * kN - head, i * kN - head + kN), those outside [0, V) not the row's.
template <typename Z>
struct RowGrid {
  Z* z;
  int V, head, vecs;
  __device__ __forceinline__ RowGrid(const void* p, long at, int V_) : V(V_) {
    z = static_cast<Z*>(const_cast<void*>(p)) + at;
    head = (int)((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(Z));
    vecs = (V + head + Vec<Z>::kN - 1) / Vec<Z>::kN;
  }
  __device__ __forceinline__ int first(int i) const { return i * Vec<Z>::kN - head; }
  __device__ __forceinline__ bool whole(int i) const { return first(i) >= 0 && first(i) + Vec<Z>::kN <= V; }
  // -inf outside the row
  __device__ __forceinline__ uint4 load(int i) const {
    if (whole(i)) return __ldcs(reinterpret_cast<const uint4*>(z + first(i)));
    uint4 v = Vec<Z>::lowest();
    Z* e = reinterpret_cast<Z*>(&v);
#pragma unroll
    for (int k = 0; k < Vec<Z>::kN; ++k) {
      const int c = first(i) + k;
      if (c >= 0 && c < V) e[k] = z[c];
    }
    return v;
  }
};

// (m, s) stands for s * 2^(m c); (-inf, 0) for nothing.  Differences are
// taken before the product with c, so that rows of the type's lowest value
// stay finite.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ void join(float& m, float& s, float mo, float so, float c) {
  const float top = fmaxf(m, mo), base = finite_max(top);
  s = s * fast_exp2((m - base) * c) + so * fast_exp2((mo - base) * c);
  m = top;
}

// N vectors into a thread's running pair
template <typename Z, int N>
__device__ __forceinline__ void take(const uint4 (&v)[N], float& m, float& s, float c) {
  float top = Vec<Z>::top(v[0]);
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, Vec<Z>::top(v[i]));
  if (top > m) {
    s *= fast_exp2((m - top) * c);
    m = top;
  }
  const float base = finite_max(m);
  float sum[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float f[Vec<Z>::kN];
    Vec<Z>::unpack(v[i], f);
#pragma unroll
    for (int k = 0; k < Vec<Z>::kN; ++k) sum[k & 1] += fast_exp2((f[k] - base) * c);
  }
  s += sum[0] + sum[1];
}

template <int WARPS>
struct Shared {
  int32_t ids[MOK_DISTILL_MAX_TOP];
  float p[MOK_DISTILL_MAX_TOP];
  float m[WARPS], s[WARPS];
  float share_m[kMaxShare], share_s[kMaxShare];
  float loss[WARPS];
  int any;
};

// An entry's id, or -1 where it is left out.
__device__ __forceinline__ int entry_id(const DistillParams& q, long t, int j, bool tell) {
  const int id = q.ids[t * q.K + j];
  if (id >= -1 && id < q.V) return id;
  if (tell) atomicOr(q.hdr + kHdrError, MOK_ERRBIT_BAD_INDEX);
  return -1;
}

// The teacher's probabilities, by one warp.  NaN values make them NaN.
template <int W>
__device__ __forceinline__ void teacher(const DistillParams& q, long t, Shared<W>& sh, int lane) {
  float top = -INFINITY;
  bool nan = false;
  for (int j = lane; j < q.K; j += 32) {
    const int id = entry_id(q, t, j, true);
    const float v = id >= 0 ? q.vals[t * q.K + j] * q.inv_tau : -INFINITY;
    sh.ids[j] = id;
    sh.p[j] = v;
    nan |= isnan(v);
    top = fmaxf(top, v);
  }
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  nan = __any_sync(0xffffffffu, nan);
  const float base = top == -INFINITY ? 0.0f : top;
  float total = 0.0f;
  for (int j = lane; j < q.K; j += 32) {
    const float e = expf(sh.p[j] - base);  // exp(-inf) = 0 for what is left out
    sh.p[j] = e;
    total += e;
  }
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const bool any = total > 0.0f || nan || isnan(total);
  for (int j = lane; j < q.K; j += 32) sh.p[j] = any ? sh.p[j] / total : 0.0f;
  if (lane == 0) sh.any = any;
}

// The CTA's pair from its threads', the same in every thread.
template <int W>
__device__ __forceinline__ void join_block(float& m, float& s, float c, Shared<W>& sh) {
  for (int o = 16; o > 0; o >>= 1) {
    const float mo = __shfl_xor_sync(0xffffffffu, m, o), so = __shfl_xor_sync(0xffffffffu, s, o);
    join(m, s, mo, so, c);
  }
  if ((threadIdx.x & 31) == 0) {
    sh.m[threadIdx.x >> 5] = m;
    sh.s[threadIdx.x >> 5] = s;
  }
  __syncthreads();
  // W lanes of every warp join the warps' pairs
  static_assert(W <= 32 && (W & (W - 1)) == 0, "a group of lanes holds the warps' pairs");
  m = sh.m[threadIdx.x & (W - 1)];
  s = sh.s[threadIdx.x & (W - 1)];
  for (int o = W / 2; o > 0; o >>= 1) {
    const float mo = __shfl_xor_sync(0xffffffffu, m, o), so = __shfl_xor_sync(0xffffffffu, s, o);
    join(m, s, mo, so, c);
  }
}

// The row's pair from its CTAs', the same in every thread.
template <int W>
__device__ __forceinline__ void join_shares(float& m, float& s, float c, Shared<W>& sh, int rank, int shares) {
  if (shares == 1) return;
  cg::cluster_group cluster = cg::this_cluster();
  if (threadIdx.x < shares) {
    *cluster.map_shared_rank(&sh.share_m[rank], threadIdx.x) = m;
    *cluster.map_shared_rank(&sh.share_s[rank], threadIdx.x) = s;
  }
  cluster.sync();
  m = sh.share_m[0];
  s = sh.share_s[0];
  for (int i = 1; i < shares; ++i) join(m, s, sh.share_m[i], sh.share_s[i], c);
}

// The row's loss and log-sum-exp from its pair (all threads of one CTA; after a
// barrier that follows teacher()).
template <typename Z, int W>
__device__ __forceinline__ void store_loss(const DistillParams& q, long t, Shared<W>& sh, const Z* logits, float m,
                                           float s) {
  const float base = finite_max(m), log_s = logf(s);
  float l = 0.0f;
  for (int j = threadIdx.x; j < q.K; j += W * 32) {
    const float p = sh.p[j];
    if (p > 0.0f || isnan(p)) l += p * (logf(p) - ((Vec<Z>::value(logits[j]) - base) * q.inv_tau - log_s));
  }
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if ((threadIdx.x & 31) == 0) sh.loss[threadIdx.x >> 5] = l;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < W; ++w) l += sh.loss[w];
    q.loss[t] = l;
    if (q.lse) q.lse[t] = fmaf(base, q.inv_tau, log_s);
  }
}

// The student's logits at the listed columns, while the row still holds them.
template <typename Z>
__device__ __forceinline__ void read_listed(const DistillParams& q, long t, const Z* z, Z* logits, int threads) {
  for (int j = threadIdx.x; j < q.K; j += threads) {
    const int id = entry_id(q, t, j, false);
    if (id >= 0) logits[j] = z[id];
  }
}

constexpr int kThreads = 512;

template <typename Z>
__global__ void __launch_bounds__(kThreads) distill_forward_kernel(DistillParams q, int shares) {
  __shared__ Shared<kThreads / 32> sh;
  __shared__ Z logits[MOK_DISTILL_MAX_TOP];
  const long t = blockIdx.x / shares;
  const int rank = blockIdx.x % shares;
  const float c = q.inv_tau * kLog2e;
  const RowGrid<Z> row(q.z, t * q.ldz, q.V);
  if (rank == 0) {
    read_listed(q, t, row.z, logits, kThreads);
    if (threadIdx.x >= kThreads - 32) teacher(q, t, sh, threadIdx.x & 31);
  }
  const int v1 = (int)((long)row.vecs * (rank + 1) / shares);
  float m = -INFINITY, s = 0.0f;
  constexpr int kAhead = 4;
  for (int v = (int)((long)row.vecs * rank / shares) + threadIdx.x; v < v1; v += kAhead * kThreads) {
    uint4 x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = v + i * kThreads < v1 ? row.load(v + i * kThreads) : Vec<Z>::lowest();
    take<Z, kAhead>(x, m, s, c);
  }
  join_block(m, s, c, sh);
  join_shares(m, s, c, sh, rank, shares);
  if (rank == 0) store_loss(q, t, sh, logits, m, s);
}

// The gradient of a share of a row, and with STEP the sum before it.  Without
// STEP the shares are CTAs of their own.  Shared memory: the share's vectors.
constexpr int kGradThreads = 256;
constexpr int kPieces = 4;  // copies of a share, so that the sum begins with the first

template <typename Z, bool STEP>
__global__ void __launch_bounds__(kGradThreads, 7) distill_gradient_kernel(DistillParams q, int shares) {
  extern __shared__ __align__(128) uint8_t share_smem[];
  __shared__ Shared<kGradThreads / 32> sh;
  __shared__ Z logits[MOK_DISTILL_MAX_TOP];
  __shared__ uint64_t full[kPieces];
  constexpr int kN = Vec<Z>::kN;
  uint4* x = reinterpret_cast<uint4*>(share_smem);
  const long t = blockIdx.x / shares;
  const int rank = blockIdx.x % shares;
  const float c = q.inv_tau * kLog2e;
  const RowGrid<Z> row(q.z, t * q.ldz, q.V), grad(q.dz, t * q.lddz, q.V);
  const int v0 = (int)((long)row.vecs * rank / shares), n = (int)((long)row.vecs * (rank + 1) / shares) - v0;
  // bulk copies take whole vectors; a part-filled one at the row's ends goes by hand
  const int lead = n > 0 && !row.whole(v0) ? 1 : 0, tail = n > lead && !row.whole(v0 + n - 1) ? 1 : 0;
  const int whole = n - lead - tail, piece = (whole + kPieces - 1) / kPieces;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPieces; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
    for (int i = 0; i < kPieces; ++i) {
      const int at = i * piece, len = max(0, min(piece, whole - at));
      mbar_arrive_expect_tx(&full[i], len * 16);
      if (len) bulk_load(x + lead + at, row.z + row.first(v0 + lead + at), len * 16, &full[i]);
    }
  }
  if (lead && threadIdx.x == 32) x[0] = row.load(v0);
  if (tail && threadIdx.x == 64) x[n - 1] = row.load(v0 + n - 1);
  read_listed(q, t, row.z, logits, kGradThreads);
  if (threadIdx.x >= kGradThreads - 32) teacher(q, t, sh, threadIdx.x & 31);
  __syncthreads();
  // the copies always arrive (the limit is there for what no one foresaw: the sum would be of other values)
  auto arrived = [&](int i) { return mbar_drain(&full[i], 0, kWaitLimitNs); };
  bool fine = true;

  // q_v = 2^((z_v - base) c - log_s)
  float base, log_s;
  if constexpr (STEP) {
    float m = -INFINITY, sum = 0.0f;
    for (int i = 0; i < kPieces; ++i) {
      fine &= arrived(i);
      // piece i, with the vectors that went by hand beside the first and the last
      const int b = i == 0 ? 0 : lead + i * piece, e = i == kPieces - 1 ? n : min(n, lead + (i + 1) * piece);
      constexpr int kAhead = 2;
      for (int v = b + threadIdx.x; v < e; v += kAhead * kGradThreads) {
        uint4 y[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) y[k] = v + k * kGradThreads < e ? x[v + k * kGradThreads] : Vec<Z>::lowest();
        take<Z, kAhead>(y, m, sum, c);
      }
    }
    join_block(m, sum, c, sh);
    // (the logits that other CTAs list are read before the barrier in here, and overwritten after it)
    join_shares(m, sum, c, sh, rank, shares);
    base = finite_max(m);
    log_s = log2f(sum);
    if (rank == 0) store_loss(q, t, sh, logits, m, sum);
  } else {
    for (int i = 0; i < kPieces; ++i) fine &= arrived(i);
    base = q.lse_in[t] / q.inv_tau;
    log_s = 0.0f;
  }
  if (!fine && threadIdx.x == 0) atomicOr(q.hdr + kHdrError, MOK_ERRBIT_TIMEOUT);
  const float g = q.dloss[t] * q.inv_tau;
  const bool any = sh.any, same = row.head == grad.head;
  for (int i = threadIdx.x; i < n; i += kGradThreads) {
    const int v = v0 + i;
    float f[kN];
    Vec<Z>::unpack(x[i], f);
#pragma unroll
    for (int k = 0; k < kN; ++k) f[k] = any ? g * fast_exp2(fmaf(f[k] - base, c, -log_s)) : 0.0f;
    if (same && row.whole(v)) {
      __stcs(reinterpret_cast<uint4*>(grad.z + row.first(v)), Vec<Z>::pack(f));
    } else {
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int col = row.first(v) + k;
        if (col >= 0 && col < q.V) grad.z[col] = Vec<Z>::from(f[k]);
      }
    }
  }
  if (!any) return;
  // the listed columns of this share, each stored by the first entry that has it
  __syncthreads();
  for (int j = threadIdx.x; j < q.K; j += kGradThreads) {
    const int id = sh.ids[j];
    const int v = (id + row.head) / kN;
    if (id < 0 || v < v0 || v >= v0 + n) continue;
    float sum = 0.0f;
    bool mine = true;
    for (int i = 0; i < q.K; ++i)
      if (sh.ids[i] == id) {
        sum += sh.p[i];
        mine = mine && i >= j;
      }
    if (mine) grad.z[id] = Vec<Z>::from(g * (fast_exp2(fmaf(Vec<Z>::value(logits[j]) - base, c, -log_s)) - sum));
  }
}

int sm_count() {
  const int n = device_sm_count();
  return n > 0 ? n : 1;
}

template <typename... Args>
cudaError_t launch_shares(void (*kernel)(Args...), long rows, int shares, bool cluster, int threads, size_t smem,
                          cudaStream_t st, Args... args) {
  if (rows * shares > 0x7fffffffl) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * shares));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = shares;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster && shares > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Vectors of the longest row on its grid.
template <typename Z>
long row_vectors(const DistillParams& p) {
  const int kN = Vec<Z>::kN;
  const bool aligned = (reinterpret_cast<uintptr_t>(p.z) & 15) == 0 && (p.T == 1 || p.ldz % kN == 0);
  return ((long)p.V + (aligned ? 0 : kN - 1) + kN - 1) / kN;
}

template <typename Z>
cudaError_t launch_forward(const DistillParams& p, int* launches, cudaStream_t st) {
  // a CTA a row, or more while SMs are left and each keeps two vectors a thread
  int shares = 1;
  const long vecs = row_vectors<Z>(p);
  while (shares < kMaxShare && (long)p.T * shares < 2l * sm_count() && vecs >= 4l * kThreads * shares) shares *= 2;
  *launches += 1;
  return launch_shares(distill_forward_kernel<Z>, p.T, shares, true, kThreads, 0, st, p, shares);
}

constexpr long kShareVecs = 2048;   // 32 KB: seven CTAs an SM
constexpr long kMostVecs = 13312;   // 208 KB: what a CTA can hold at most

template <typename Z, bool STEP>
cudaError_t launch_gradient(const DistillParams& p, int shares, int* launches, cudaStream_t st) {
  const long vecs = row_vectors<Z>(p);
  const size_t smem = (size_t)((vecs + shares - 1) / shares) * 16;
  auto kernel = distill_gradient_kernel<Z, STEP>;
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostVecs * 16);
    if (e != cudaSuccess) return e;
  }
  *launches += 1;
  return launch_shares(kernel, p.T, shares, STEP, kGradThreads, smem, st, p, shares);
}

template <typename Z>
cudaError_t launch(DistillMode mode, DistillParams p, int* launches, cudaStream_t st) {
  *launches = 0;
  if (mode == DISTILL_FORWARD) return launch_forward<Z>(p, launches, st);
  const long vecs = row_vectors<Z>(p);
  if (mode == DISTILL_STEP) {
    int shares = 1;
    while (shares < kMaxShare && vecs > kShareVecs * shares) shares *= 2;
    while (shares < kMaxShare && (long)p.T * shares < 2l * sm_count() && vecs >= 2l * kGradThreads * shares) shares *= 2;
    if (vecs <= kMostVecs * shares) return launch_gradient<Z, true>(p, shares, launches, st);
    const cudaError_t e = launch_forward<Z>(p, launches, st);
    if (e != cudaSuccess) return e;
    p.lse_in = p.lse;
  }
  return launch_gradient<Z, false>(p, (int)((vecs + kShareVecs - 1) / kShareVecs), launches, st);
}

}  // namespace

cudaError_t launch_distill(DistillMode mode, mok_dtype type, const DistillParams& p, int* launches, cudaStream_t st) {
  return type == MOK_TYPE_BF16 ? launch<__nv_bfloat16>(mode, p, launches, st) : launch<float>(mode, p, launches, st);
}

}  // namespace mok

// Distillation loss from a teacher's top logits.  For a row of V student
// logits z and the teacher's K listed (id_j, v_j), temperature tau:
//
//   p = softmax over the list of v / tau          (entries of id -1 left out)
//   lse = log sum_v exp(z_v / tau),   log q_v = z_v / tau - lse
//   loss = sum_j p_j (log p_j - log q_(id_j)) = KL(p || q)
//   dz_v = (dloss / tau) (q_v - sum_{j: id_j = v} p_j)
//
// An entry of p_j = 0 adds nothing; a row whose list is empty has loss 0 and
// gradient 0.  Every operation is bound by the row's bytes -- the forward
// reads it once, the backward reads and writes it once, and the step, which
// needs the row's sum before it can write, keeps the row on the chip in
// between -- with the instructions of an element close behind:
//
//  * A sum is kept as (m, s), s * 2^(m c), m the largest logit so far and c =
//    log2(e) / tau; a term is 2^((z - m) c) -- the difference first, so that
//    the largest term is 1 exactly and rows of the type's lowest value stay
//    finite.  Differences, products and sums go two at a time (f32x2).
//    Threads, warps and CTAs join their pairs in a fixed tree.
//  * Rows are read in 16-byte vectors of the address grid (a row of any
//    alignment has at most one part-filled vector at each end).
//  * A row is shared by a cluster of up to 8 CTAs, which exchange their pairs
//    through distributed shared memory: a few rows still fill the GPU.  In
//    the step a CTA brings its share, 32 or 64 KB where eight are enough, to shared
//    memory with bulk copies, where it stays between the sum and the gradient;
//    six CTAs of 32 KB an SM are in different phases, so that loads and stores
//    overlap: 393 us for 4,096 rows of 131,072 bf16, loss and gradient, 82% of
//    the rate of a copy.  (Twice the threads a CTA: 412; a CTA a row of its own
//    that streams it twice, the second time from L2: 471.)
//  * The teacher's list (at most MOK_DISTILL_MAX_TOP entries) is a warp's
//    work, hidden behind the row's copies.  Listed columns are stored after
//    the rest, by the first entry that has them.
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

// ---------------------------------------------------------------- pairs of floats
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pair(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(F2 p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p.v));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 exp2_2(F2 a) {
  float lo, hi;
  split(a, lo, hi);
  return pair(fast_exp2(lo), fast_exp2(hi));
}

// ---------------------------------------------------------------- vectors of 16 bytes
template <typename Z>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, F2 (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 pack(const F2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      split(f[i], lo, hi);
      w[i] = pack_bf16x2(lo, hi);
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
  static __device__ __forceinline__ uint4 lowest() {
    return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, F2 (&f)[2]) {
    f[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 pack(const F2 (&f)[2]) {
    float a, b, c, d;
    split(f[0], a, b);
    split(f[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  }
  static __device__ __forceinline__ float top(const uint4& v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static __device__ __forceinline__ float value(float z) { return z; }
  static __device__ __forceinline__ float from(float f) { return f; }
  static __device__ __forceinline__ uint4 lowest() {
    return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
  }
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
  // a part-filled vector: -inf outside the row
  __device__ __noinline__ uint4 load_part(int i) const {
    uint4 v = Vec<Z>::lowest();
    Z* e = reinterpret_cast<Z*>(&v);
#pragma unroll 1
    for (int k = 0; k < Vec<Z>::kN; ++k) {
      const int c = first(i) + k;
      if (c >= 0 && c < V) e[k] = z[c];
    }
    return v;
  }
};

// The elements of a vector, col the first's, that lie in [0, V).
template <typename Z>
__device__ __noinline__ void row_store(Z* z, int V, int col, uint4 v) {
  const Z* e = reinterpret_cast<const Z*>(&v);
#pragma unroll 1
  for (int k = 0; k < Vec<Z>::kN; ++k)
    if (col + k >= 0 && col + k < V) z[col + k] = e[k];
}

// Zeros in a share of a gradient row, on the row's own grid.
template <typename Z>
__device__ __forceinline__ void zero_share(const RowGrid<Z>& grad, int rank, int shares, int threads) {
  const int most = (grad.vecs + shares - 1) / shares, v1 = min(grad.vecs, (rank + 1) * most);
  const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll 4
  for (int v = rank * most + threadIdx.x; v < v1; v += threads) {
    if (grad.whole(v))
      __stcs(reinterpret_cast<uint4*>(grad.z + grad.first(v)), none);
    else
      row_store(grad.z, grad.V, grad.first(v), none);
  }
}

// ---------------------------------------------------------------- sums
struct Sum {
  float m, s;  // s * 2^(m c); (-inf, 0) for nothing
};

// 2^((from - to) c) for from <= to; 0 for a sum of nothing
__device__ __forceinline__ float rescale(float from, float to, float c) {
  return from == -INFINITY ? 0.0f : fast_exp2((from - to) * c);
}
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.0f : m; }

// N vectors into a thread's sum
template <typename Z, int N>
__device__ __forceinline__ void take(const uint4 (&v)[N], Sum& sum, float c) {
  float top = Vec<Z>::top(v[0]);
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, Vec<Z>::top(v[i]));
  if (top > sum.m) {
    sum.s *= rescale(sum.m, top, c);
    sum.m = top;
  }
  const float base = -finite_max(sum.m);
  const F2 b2 = pair(base, base), c2 = pair(c, c);
  F2 acc[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    F2 f[Vec<Z>::kN / 2];
    Vec<Z>::unpack(v[i], f);
#pragma unroll
    for (int k = 0; k < Vec<Z>::kN / 2; ++k) acc[k & 1] = add2(acc[k & 1], exp2_2(mul2(add2(f[k], b2), c2)));
  }
  float a, b;
  split(add2(acc[0], acc[1]), a, b);
  sum.s += a + b;
}

template <int WIDTH>
__device__ __forceinline__ void join_lanes(Sum& a, float c) {
  float top = a.m;
#pragma unroll
  for (int o = WIDTH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  a.s *= a.m == top ? 1.0f : rescale(a.m, top, c);  // (a NaN sum stays one: 0 * NaN)
  a.m = top;
#pragma unroll
  for (int o = WIDTH / 2; o > 0; o >>= 1) a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
}

// ---------------------------------------------------------------- what a CTA shares
template <int WARPS>
struct Shared {
  Sum warp[WARPS];
  Sum share[kMaxShare];
  int any;
};

// The list, in dynamic shared memory.
struct List {
  int32_t* ids;   // [K]
  float* p;       // [K]
  float* logits;  // [K] the student's, at the ids
};
__host__ __device__ constexpr size_t list_bytes(int K) { return (size_t)K * 12; }
__device__ __forceinline__ List list_at(uint8_t* smem, int K) {
  List l;
  l.ids = reinterpret_cast<int32_t*>(smem);
  l.p = reinterpret_cast<float*>(l.ids + K);
  l.logits = l.p + K;
  return l;
}

// By one warp, in three steps of which the others wait for the first alone:
// the ids and values (-inf for what is left out) --
// returns whether there is anything to learn from: an entry above -inf.
__device__ __forceinline__ bool read_list(const DistillParams& q, long t, const List& l, int lane) {
  bool any = false;
#pragma unroll 1
  for (int j = lane; j < q.K; j += 32) {
    int id = q.ids[t * q.K + j];
    float v = q.vals[t * q.K + j];
    if (id < -1 || id >= q.V) {
      atomicOr(q.hdr + kHdrError, MOK_ERRBIT_BAD_INDEX);
      id = -1;
    }
    if (id < 0) v = -INFINITY;
    l.ids[j] = id;
    l.p[j] = v;
    any |= v != -INFINITY;  // a NaN value counts: it makes the row NaN
  }
  return __any_sync(0xffffffffu, any);
}

// The student's logits at the ids, while the row still holds them.
template <typename Z>
__device__ __forceinline__ void read_logits(const DistillParams& q, const Z* z, const List& l, int lane) {
#pragma unroll 4
  for (int j = lane; j < q.K; j += 32) l.logits[j] = l.ids[j] >= 0 ? Vec<Z>::value(z[l.ids[j]]) : 0.0f;
}

// The teacher's probabilities in place of its values, for a list that has any.
// (The difference first: a value over tau may be past f32 where the difference is 0.)
__device__ __forceinline__ void softmax_list(const DistillParams& q, const List& l, int lane) {
  float top = -INFINITY;
#pragma unroll 1
  for (int j = lane; j < q.K; j += 32) top = fmaxf(top, l.p[j]);
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float base = top == -INFINITY ? 0.0f : top;
  float total = 0.0f;
#pragma unroll 1
  for (int j = lane; j < q.K; j += 32) {
    const float e = expf((l.p[j] - base) * q.inv_tau);  // exp(-inf) = 0 for what is left out
    l.p[j] = e;
    total += e;
  }
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
#pragma unroll 1
  for (int j = lane; j < q.K; j += 32) l.p[j] /= total;
  __syncwarp();
}

// The cluster's CTAs tell one another that they run (begin), before any writes
// into another's shared memory (wait): a CTA that has not begun has none.
__device__ __forceinline__ void cluster_begin(int shares) {
  if (shares > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_begun() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// The row's sum from those of the threads of its CTAs, the same in every
// thread.  The first W warps hold sums; others only take part in the barriers.
template <int W>
__device__ __forceinline__ void join_row(Sum& a, float c, Shared<W>& sh, int rank, int shares) {
  join_lanes<32>(a, c);
  if ((threadIdx.x & 31) == 0 && threadIdx.x < W * 32) sh.warp[threadIdx.x >> 5] = a;
  __syncthreads();
  static_assert(W <= 32 && (W & (W - 1)) == 0, "a group of lanes holds the warps' sums");
  a = sh.warp[threadIdx.x & (W - 1)];
  join_lanes<W>(a, c);
  if (shares == 1) return;
  cg::cluster_group cluster = cg::this_cluster();
  cluster_begun();
  if (threadIdx.x < shares) *cluster.map_shared_rank(&sh.share[rank], threadIdx.x) = a;
  cluster.sync();
  const int i = threadIdx.x & (kMaxShare - 1);
  a.m = -INFINITY;
  a.s = 0.0f;
  if (i < shares) a = sh.share[i];
  join_lanes<kMaxShare>(a, c);
}

// The row's loss and log-sum-exp from its sum, by the warp that read the list.
__device__ __forceinline__ void store_loss(const DistillParams& q, long t, const List& list, bool any, Sum a, int lane) {
  const float base = finite_max(a.m), log_s = logf(a.s);
  float l = 0.0f;
#pragma unroll 1
  for (int j = lane; any && j < q.K; j += 32) {
    const float p = list.p[j];
    if (p > 0.0f || isnan(p)) l += p * (logf(p) - ((list.logits[j] - base) * q.inv_tau - log_s));
  }
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) {
    q.loss[t] = l;
    if (q.lse) q.lse[t] = fmaf(base, q.inv_tau, log_s);
    if (q.sums) q.sums[t] = make_float2(base, a.s);
  }
}

// The kN elements from element `by` on of two neighbouring vectors.
template <typename Z>
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int by) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const int words = sizeof(Z) == 2 ? by >> 1 : by;
  if (words & 2)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (words & 1)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  if (sizeof(Z) == 2 && (by & 1))
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The gradients of the listed columns in vectors [v0, v1) in place of their
// logits; returns a bit for each of the lane's entries that is the first of
// its column.  e_j q_base - sum of p: where there is one token its e_j is the
// sum, and the division says 1 exactly.
template <typename Z, bool STEP>
__device__ __forceinline__ uint32_t list_gradients(const DistillParams& q, const List& list, int head, int v0, int v1,
                                                   float base, float q_base, float sum, float g, float c, int lane) {
  uint32_t mine = 0;
#pragma unroll 1
  for (int j = lane; j < q.K; j += 32) {
    const int id = list.ids[j], v = (id + head) / Vec<Z>::kN;
    if (id < 0 || v < v0 || v >= v1) continue;
    float p = 0.0f;
    bool first = true;
#pragma unroll 8
    for (int i = 0; i < q.K; ++i) {
      const bool same_id = list.ids[i] == id;
      p += same_id ? list.p[i] : 0.0f;
      first = first && !(same_id && i < j);
    }
    const float e_j = fast_exp2((list.logits[j] - base) * c);
    list.logits[j] = g * ((STEP ? e_j / sum : e_j * q_base) - p);
    mine |= (uint32_t)first << (j >> 5);
  }
  return mine;
}

// A vector's gradient.
template <typename Z>
struct Gradient {
  F2 b2, c2, s2;
  __device__ __forceinline__ Gradient(float base, float c, float scale)
      : b2(pair(-base, -base)), c2(pair(c, c)), s2(pair(scale, scale)) {}
  __device__ __forceinline__ uint4 operator()(const uint4& v) const {
    F2 f[Vec<Z>::kN / 2];
    Vec<Z>::unpack(v, f);
#pragma unroll
    for (int k = 0; k < Vec<Z>::kN / 2; ++k) f[k] = mul2(s2, exp2_2(mul2(add2(f[k], b2), c2)));
    return Vec<Z>::pack(f);
  }
};

// All kernels: workers, and a last warp for the list.
// Forward: 1,000 rows of 50,001 bf16 20 to 23 us (GPUs differ), 65 to 75% of
// the rate of a copy; of 128 workers 22, of 512 26 where 256 take 20.  4,096
// rows of 131,072: 150 us, all of it; the gradient of them alone 339, 95%.
constexpr int kForwardWorkers = 256;
constexpr int kGradWorkers = 128;

template <typename Z>
__global__ void __launch_bounds__(kForwardWorkers + 32) distill_forward_kernel(DistillParams q, int shares, int most) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared<kForwardWorkers / 32> sh;
  cluster_begin(shares);
  const long t = blockIdx.x / shares;
  const int rank = blockIdx.x % shares;
  const float c = q.inv_tau * kLog2e;
  const RowGrid<Z> row(q.z, t * q.ldz, q.V);
  const List list = list_at(smem, q.K);
  Sum a{-INFINITY, 0.0f};
  if (threadIdx.x >= kForwardWorkers) {
    if (rank == 0) {
      const int lane = threadIdx.x & 31;
      const bool any = read_list(q, t, list, lane);
      if (any) {
        read_logits(q, row.z, list, lane);
        softmax_list(q, list, lane);
      }
      if (lane == 0) sh.any = any;
    }
  } else {
    const int v0 = min(rank * most, row.vecs), v1 = min(v0 + most, row.vecs);
    // the part-filled vectors at the row's ends apart
    const int b = v1 > v0 && !row.whole(v0) ? v0 + 1 : v0, e = v1 > b && !row.whole(v1 - 1) ? v1 - 1 : v1;
    if ((b > v0 && threadIdx.x == 0) || (e < v1 && threadIdx.x == 32)) {
      const uint4 x[1] = {row.load_part(threadIdx.x == 0 ? v0 : e)};
      take<Z, 1>(x, a, c);
    }
    constexpr int kAhead = 4;
    const uint4* from = reinterpret_cast<const uint4*>(row.z + row.first(0));
    for (int v = b + threadIdx.x; v < e; v += kAhead * kForwardWorkers) {
      uint4 x[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        x[i] = v + i * kForwardWorkers < e ? __ldcs(from + v + i * kForwardWorkers) : Vec<Z>::lowest();
      take<Z, kAhead>(x, a, c);
    }
  }
  join_row(a, c, sh, rank, shares);
  if (rank == 0 && threadIdx.x >= kForwardWorkers) store_loss(q, t, list, sh.any, a, threadIdx.x & 31);
}

// The gradient of a share of a row, and with STEP the sum before it.  Without
// STEP the shares are CTAs of their own.  Shared memory: the share's vectors,
// then the list.
constexpr int kPieces = 2;  // copies of a share, so that the sum begins with the first

template <typename Z, bool STEP>
__global__ void __launch_bounds__(kGradWorkers + 32) distill_gradient_kernel(DistillParams q, int shares, int most) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared<kGradWorkers / 32> sh;
  __shared__ uint64_t full[kPieces];
  if (STEP) cluster_begin(shares);
  constexpr int kN = Vec<Z>::kN;
  uint4* x = reinterpret_cast<uint4*>(smem);
  const List list = list_at(smem + (size_t)most * 16, q.K);
  const long t = blockIdx.x / shares;
  const int rank = blockIdx.x % shares, lane = threadIdx.x & 31;
  const bool worker = threadIdx.x < kGradWorkers;
  // the gradient takes the logits' place: then a logit is read before any is overwritten
  const bool in_place = q.in_place;
  const float c = q.inv_tau * kLog2e;
  const RowGrid<Z> row(q.z, t * q.ldz, q.V), grad(q.dz, t * q.lddz, q.V);
  const int v0 = min(rank * most, row.vecs), n = min(most, row.vecs - v0);
  // bulk copies take whole vectors [b, e); a part-filled one at the row's ends goes by hand
  const int b = n > 0 && !row.whole(v0) ? 1 : 0, e = n > b && !row.whole(v0 + n - 1) ? n - 1 : n;
  const int piece = (e - b + kPieces - 1) / kPieces;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPieces; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
#pragma unroll 1
    for (int i = 0; i < kPieces; ++i) {
      const int at = b + i * piece, len = max(0, min(piece, e - at));
      mbar_arrive_expect_tx(&full[i], len * 16);
      if (len) bulk_load(x + at, row.z + row.first(v0 + at), len * 16, &full[i]);
    }
  }
  __syncthreads();

  Sum a{-INFINITY, 0.0f};
  bool fine = true;
  const bool first_part = threadIdx.x == 32 && b > 0, last_part = threadIdx.x == 64 && e < n;
  if (!worker) {
    const bool any = read_list(q, t, list, lane);
    if (lane == 0) sh.any = any;
    if (in_place && any) read_logits(q, row.z, list, lane);
  } else {
    // a part-filled vector stays with the thread that brings it
    if (first_part) x[0] = row.load_part(v0);
    if (last_part) x[n - 1] = row.load_part(v0 + n - 1);
    if (STEP && (first_part || last_part)) {
      const uint4 y[1] = {first_part ? x[0] : x[n - 1]};
      take<Z, 1>(y, a, c);
    }
#pragma unroll 1
    for (int i = 0; i < kPieces; ++i) {
      // the copies always arrive; a wait that gave up all the same is told to the caller
      if (!mbar_try_wait(&full[i], 0)) fine &= mbar_drain(&full[i], 0, kWaitLimitNs);
      if (!STEP) continue;
      const int p1 = min(e, b + (i + 1) * piece);
      constexpr int kAhead = 4;
#pragma unroll 1
      for (int v = b + i * piece + threadIdx.x; v < p1; v += kAhead * kGradWorkers) {
        uint4 y[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) y[k] = v + k * kGradWorkers < p1 ? x[v + k * kGradWorkers] : Vec<Z>::lowest();
        take<Z, kAhead>(y, a, c);
      }
    }
  }
  if (!fine && lane == 0) atomicOr(q.hdr + kHdrError, MOK_ERRBIT_TIMEOUT);

  // q_v = 2^((z_v - base) c) q_base
  float base, q_base;
  if constexpr (STEP) {
    // (in place, the logits that other CTAs list are read before the barrier in here, and overwritten after it)
    join_row(a, c, sh, rank, shares);
    base = finite_max(a.m);
    q_base = 1.0f / a.s;
  } else {
    __syncthreads();
    if (q.sums) {
      const float2 s = q.sums[t];
      base = s.x;
      q_base = 1.0f / s.y;
    } else {
      // z / tau - lse = (z - lse tau) / tau: base is that logit, q_base what its rounding left
      const double z0 = (double)q.lse_in[t] * (double)q.tau;
      base = (float)z0;
      const float left = isinf(base) ? 0.0f : (float)((double)base - z0);
      q_base = left == 0.0f ? 1.0f : fast_exp2(left * c);
    }
  }
  const float g = q.dloss[t] * q.inv_tau;
  const bool any = sh.any, same = row.head == grad.head;
  const float scale = g * q_base;
  const Gradient<Z> gradient(base, c, scale);
  uint32_t mine = 0;  // list warp: its entries that are the first of a column of this share
  if (!worker) {
    if (any) {
      if (!in_place) read_logits(q, row.z, list, lane);
      softmax_list(q, list, lane);
    }
    if (STEP && rank == 0) store_loss(q, t, list, any, a, lane);
    if (any) mine = list_gradients<Z, STEP>(q, list, row.head, v0, v0 + n, base, q_base, a.s, g, c, lane);
  } else if (any && same) {
    uint4* out = reinterpret_cast<uint4*>(grad.z + row.first(v0 + b));
#pragma unroll 4
    for (int i = threadIdx.x; i < e - b; i += kGradWorkers) __stcs(out + i, gradient(x[b + i]));
    if (first_part) row_store(grad.z, q.V, row.first(v0), gradient(x[0]));
    if (last_part) row_store(grad.z, q.V, row.first(v0 + n - 1), gradient(x[n - 1]));
  } else if (any) {
    // a gradient of another alignment: the vectors of its grid that lie in
    // this share's columns, each out of two of the logits', and its few
    // elements before and after them
    const int c0 = max(0, row.first(v0)), c1 = min(q.V, row.first(v0 + n));
    const int g0 = (c0 + grad.head + kN - 1) / kN, g1 = max(g0, (c1 + grad.head) / kN);
    const int shift = (grad.first(g0) - row.first(v0)) & (kN - 1);
#pragma unroll 2
    for (int v = g0 + threadIdx.x; v < g1; v += kGradWorkers) {
      const int i = (grad.first(v) - row.first(v0)) / kN;
      __stcs(reinterpret_cast<uint4*>(grad.z + grad.first(v)), gradient(shifted<Z>(x[i], x[i + 1], shift)));
    }
    const int before = min(grad.first(g0), c1) - c0, after = max(c0 + before, grad.first(g1));
    for (int k = threadIdx.x; k < before + max(0, c1 - after); k += kGradWorkers) {
      const int col = k < before ? c0 + k : after + k - before;
      const float z = Vec<Z>::value(reinterpret_cast<const Z*>(x)[col - row.first(v0)]);
      grad.z[col] = Vec<Z>::from(scale * fast_exp2((z - base) * c));
    }
  } else {
    zero_share(grad, rank, shares, kGradWorkers);  // a row without a list
  }
  if (!any) return;
  // the listed columns of this share, over what the rest of their vectors stored there
  __syncthreads();
  if (!worker)
#pragma unroll 1
    for (int j = lane; j < q.K; j += 32)
      if ((mine >> (j >> 5)) & 1u) grad.z[list.ids[j]] = Vec<Z>::from(list.logits[j]);
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
  while (shares < kMaxShare && (long)p.T * shares < 2l * sm_count() && vecs >= 4l * kForwardWorkers * shares)
    shares *= 2;
  *launches += 1;
  return launch_shares(distill_forward_kernel<Z>, p.T, shares, true, kForwardWorkers + 32, list_bytes(p.K), st, p,
                       shares, (int)((vecs + shares - 1) / shares));
}

constexpr long kShareVecs = 2048;   // 32 KB: six CTAs an SM
// 64 KB, where it makes a row one CTA, or in f32, and rows fill the GPU.  4,096
// rows of 32,000 bf16 with lists of 8: 88 us, in two shares 94 (of 64: 99 and
// 103); f32 with lists of 64 196, in four 202 (of 8: 171 and 170).  Else more
// CTAs overlap better: 2,048 rows of 65,536 bf16 in two 102, in four 101; 256
// rows of 32,000 in one 17.5, in shares of 32 KB 14.9.
constexpr long kLongShareVecs = 4096;
constexpr long kMostVecs = 13312;   // 208 KB: what a CTA can hold at most

template <typename Z, bool STEP>
cudaError_t launch_gradient(const DistillParams& p, int shares, int* launches, cudaStream_t st) {
  const int most = (int)((row_vectors<Z>(p) + shares - 1) / shares);
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem((const void*)distill_gradient_kernel<Z, STEP>,
                                   kMostVecs * 16 + list_bytes(MOK_DISTILL_MAX_TOP), allowed);
  if (e != cudaSuccess) return e;
  *launches += 1;
  return launch_shares(distill_gradient_kernel<Z, STEP>, p.T, shares, STEP, kGradWorkers + 32,
                       (size_t)most * 16 + list_bytes(p.K), st, p, shares, most);
}

template <typename Z>
cudaError_t launch(DistillMode mode, DistillParams p, int* launches, cudaStream_t st) {
  *launches = 0;
  float2* const sums = p.sums;
  p.sums = nullptr;
  if (mode == DISTILL_FORWARD) return launch_forward<Z>(p, launches, st);
  const long vecs = row_vectors<Z>(p);
  if (mode == DISTILL_STEP) {
    const bool is_long = p.T >= 2l * sm_count() && (vecs <= kLongShareVecs || sizeof(Z) == 4);
    const long share = is_long ? kLongShareVecs : kShareVecs;
    int shares = 1;
    while (shares < kMaxShare && vecs > share * shares) shares *= 2;
    while (shares < kMaxShare && (long)p.T * shares < 2l * sm_count() && vecs >= 4l * kGradWorkers * shares) shares *= 2;
    if (vecs <= kMostVecs * shares) return launch_gradient<Z, true>(p, shares, launches, st);
    // (with the sums themselves in between: lse may be past f32 where the step's gradient is not)
    p.sums = sums;
    const cudaError_t e = launch_forward<Z>(p, launches, st);
    if (e != cudaSuccess) return e;
  }
  return launch_gradient<Z, false>(p, (int)((vecs + kShareVecs - 1) / kShareVecs), launches, st);
}

}  // namespace

cudaError_t launch_distill(DistillMode mode, mok_dtype type, const DistillParams& p, int* launches, cudaStream_t st) {
  return type == MOK_TYPE_BF16 ? launch<__nv_bfloat16>(mode, p, launches, st) : launch<float>(mode, p, launches, st);
}

}  // namespace mok

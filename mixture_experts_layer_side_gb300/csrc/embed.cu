// Token embedding and its gradient.
//
//   x_n = scale * table[id_n]
//   dtable_v = scale * sum of dx_n over the tokens n with id_n = v, in
//   ascending n (f32), rounded once; added to dtable_v when accumulating
//
// Both are bound by the rows' bytes.
//
// The lookup: a warp brings 2 KB of a row, four 16-byte loads a lane (16,384
// tokens of 7,168 bf16, Zipf ids: 55 us, 8.6 TB/s with the frequent rows in L2).
//
// The gradient goes by tokens sorted by id: a stable radix sort of (id,
// token) pairs, then sums over runs of equal ids.  No float is added to by
// two threads: the order of each sum is fixed by the input.
//
//  * Up to kRankTokens tokens are placed by counting the pairs before each of
//    them, 16 threads a token: no pass waits for another.  (With the sums of
//    1,024 bf16 columns: 2,048 tokens 15 us, by the radix sort 23; 8,192
//    tokens 36 and 31.  Of 8 threads a token: 2,048 tokens 17.5 us, 4,096 23.1,
//    where 16 take 15.2 and 20.4, and 32 14.2 and 17.1.)
//  * More are sorted by one cluster of kSortCtas CTAs: the pairs of a few
//    thousand to a few million tokens are small beside dx, and a cluster's
//    barriers and distributed shared memory join its histograms without a
//    launch or a device-wide barrier per pass (16,384 tokens: 17 us).  When the
//    gradient is written whole, the other SMs write the zeros of the rows that
//    no token has meanwhile.
//  * The sums: a block takes kChunk sorted tokens and a slab of columns, eight
//    tokens' loads in flight.  A run of equal ids that crosses chunks leaves
//    its parts to a last launch, so that a token that is everywhere is summed
//    by as many blocks as its rows fill.
//  * Accumulating, the rows whose runs end among the eight tokens are loaded
//    with them, so that nothing waits for a row alone.  (16,384 uniform ids in
//    131,072 f32 rows: 196 us; by reductions at L2 233.)
//
// 8,192 tokens of 2,048 bf16 columns into a table of 65,536 rows, written
// whole: 83 us.  The zeros are the most of it: the launch that writes them
// beside the sort takes 67 (3.7 TB/s; beside the counting of one token 49, where
// a memset of the table takes 38), and the sums and the last launch, 13 and 8 by
// themselves, wait for all of it.
// 16,384 tokens of 7,168 (Zipf ids) added to f32 rows: 119 us, 71% of the rate
// of a copy; beside the sums, the sort takes 17 and the last launch under 10.
#include <cooperative_groups.h>
#include <limits.h>

#include "embed.cuh"
#include "tc.cuh"

namespace mok {

namespace cg = cooperative_groups;

namespace {

constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigits = 1024;
constexpr int kQuarter = 4;  // lanes that add up a digit's counts; 8 digits of them are a warp
constexpr int kChunk = 32;  // sorted tokens per summing block

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

template <typename T>
struct Vec;  // 16 bytes
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
};
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// Whether an id is the padding's.  (What says that there is none is no id either.)
__device__ __forceinline__ bool is_pad(const EmbedParams& p, int id) {
  return id == p.pad_id && id != MOK_EMBED_NO_PAD;
}

// VEC: rows of whole aligned vectors; else one element a lane.  A warp brings
// kLookup pieces of 32 vectors (elements) of one row.
constexpr int kLookup = 4;  // (of 2: 58 us where 4 and 8 take 55)
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) embed_lookup_kernel(EmbedParams p, int pieces) {
  constexpr int kN = VEC ? Vec<T>::kN : 1;
  const long w = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int n = (int)(w / pieces), c0 = (int)(w - (long)n * pieces) * (32 * kLookup) + lane;
  if (n >= p.N) return;
  const int id = p.ids[n], cols = p.H / kN;
  const bool ok = id >= 0 && id < p.V;
  if (!ok && !is_pad(p, id) && c0 == 0) atomicOr(p.hdr + kHdrError, MOK_ERRBIT_BAD_INDEX);
  const T* src = static_cast<const T*>(p.table) + (long)(ok ? id : 0) * p.H;
  T* dst = static_cast<T*>(p.out) + (long)n * p.H;
  if constexpr (VEC) {
    uint4 v[kLookup];
#pragma unroll
    for (int i = 0; i < kLookup; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (ok && c0 + 32 * i < cols) v[i] = __ldg(reinterpret_cast<const uint4*>(src) + c0 + 32 * i);
    }
#pragma unroll
    for (int i = 0; i < kLookup; ++i) {
      float f[kN];
      Vec<T>::unpack(v[i], f);
#pragma unroll
      for (int k = 0; k < kN; ++k) f[k] = ok ? f[k] * p.scale : 0.0f;
      if (c0 + 32 * i < cols) __stcs(reinterpret_cast<uint4*>(dst) + c0 + 32 * i, pack(f));
    }
  } else {
    for (int i = 0; i < kLookup; ++i) {
      const int c = c0 + 32 * i;
      if (c < cols) put(dst + c, ok ? p.scale * to_f(src[c]) : 0.0f);
    }
  }
}

// Zeros in the rows of this CTA's range that no token has: the ids are read
// once to mark the rows that are taken (a bit each, in shared memory).
constexpr int kMarkRows = 1 << 18;  // rows marked at a time
constexpr int kZeroBytes = 16384;
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ void zero_rows(const EmbedParams& p, uint32_t* taken, int grad_bytes, int c, int ctas) {
  const int lo = (int)((long)p.V * c / ctas), hi = (int)((long)p.V * (c + 1) / ctas);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long row_bytes = (long)p.H * grad_bytes;
  uint8_t* out = static_cast<uint8_t*>(p.dtable);
  const bool vec = row_bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  uint4* zeros = reinterpret_cast<uint4*>(taken + kMarkRows / 32);
  for (int i = threadIdx.x; i < kZeroBytes / 16; i += kSortThreads) zeros[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_shared();
  for (int r0 = lo; r0 < hi; r0 += kMarkRows) {
    const int n = min(kMarkRows, hi - r0);
    __syncthreads();
    for (int i = threadIdx.x; i < (n + 31) / 32; i += kSortThreads) taken[i] = 0;
    __syncthreads();
#pragma unroll 8
    for (int i = threadIdx.x; i < p.N; i += kSortThreads) {
      const int id = p.ids[i];
      const unsigned r = (unsigned)id - (unsigned)r0;
      if (r < (unsigned)n && id != p.pad_id) atomicOr(&taken[r >> 5], 1u << (r & 31));
    }
    __syncthreads();
    if (vec) {
      // bulk stores of a zeroed buffer, a row a thread
      for (int r = threadIdx.x; r < n; r += kSortThreads) {
        if ((taken[r >> 5] >> (r & 31)) & 1u) continue;
        uint8_t* row = out + (r0 + r) * row_bytes;
        for (long at = 0; at < row_bytes; at += kZeroBytes)
          bulk_store(row + at, zeros, (uint32_t)(row_bytes - at < kZeroBytes ? row_bytes - at : kZeroBytes));
      }
    } else {
      for (int r = warp; r < n; r += kSortWarps) {
        if ((taken[r >> 5] >> (r & 31)) & 1u) continue;
        uint8_t* row = out + (r0 + r) * row_bytes;
        for (int i = lane; i < p.H; i += 32) {
          if (grad_bytes == 2)
            reinterpret_cast<uint16_t*>(row)[i] = 0;
          else
            reinterpret_cast<uint32_t*>(row)[i] = 0;
        }
      }
    }
  }
  bulk_commit();
  bulk_wait<0>();
}

// The key of token i in the sort: its id, or V (which goes last) for one that
// takes no part -- padding, or an id outside [0, V).
__device__ __forceinline__ int key_of(const EmbedParams& p, long i, bool tell) {
  const int id = p.ids[i];
  if (is_pad(p, id)) return p.V;
  if (id >= 0 && id < p.V) return id;
  if (tell) atomicOr(p.hdr + kHdrError, MOK_ERRBIT_BAD_INDEX);
  return p.V;
}

// Few tokens: a token's place is the number of pairs before it, a pair being
// one word, key over token (of `bits` bits).  A CTA places kRankShare tokens,
// kRankLanes threads each a share of the pairs; CTAs past `ranks` write zeros.
constexpr int kRankTokens = 4096;
constexpr int kRankLanes = 16, kRankShare = kSortThreads / kRankLanes;
__global__ void __launch_bounds__(kSortThreads) embed_rank_kernel(EmbedParams p, int bits, int ranks, int grad_bytes) {
  extern __shared__ __align__(16) uint32_t pairs[];
  griddep_launch_dependents();
  if (blockIdx.x >= ranks) {
    zero_rows(p, pairs, grad_bytes, blockIdx.x - ranks, gridDim.x - ranks);
    return;
  }
  // to whole vectors, with pairs that come before none
  const int padded = (p.N + 3) & ~3;
  for (int i = threadIdx.x; i < padded; i += kSortThreads)
    pairs[i] = i < p.N ? (uint32_t)key_of(p, i, blockIdx.x == 0) << bits | i : 0xffffffffu;
  __syncthreads();
  const int i = blockIdx.x * kRankShare + threadIdx.x / kRankLanes, lane = threadIdx.x % kRankLanes;
  const uint32_t pair = i < p.N ? pairs[i] : 0;
  int before = 0;
#pragma unroll 4
  for (int j = lane * 4; j < padded; j += kRankLanes * 4) {
    const uint4 k = *reinterpret_cast<const uint4*>(pairs + j);
    before += (k.x < pair) + (k.y < pair) + (k.z < pair) + (k.w < pair);
  }
#pragma unroll
  for (int o = kRankLanes / 2; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (i < p.N && lane == 0) {
    p.key[0][before] = (int32_t)(pair >> bits);
    p.pos[0][before] = i;
  }
}

// Stable least-significant-digit radix sort of the tokens by id; a token
// that takes no part (padding, or an id outside [0, V)) gets key V and goes
// last.  `bits` per pass, `passes` passes; the sorted pairs end in key/pos
// [passes & 1].  Warp w of CTA r owns the contiguous range w of range r, so
// (CTA, warp, place in the range) is the order of the pairs.
__global__ void __launch_bounds__(kSortThreads) __cluster_dims__(kSortCtas, 1, 1)
    embed_sort_kernel(EmbedParams p, int bits, int passes, int grad_bytes) {
  extern __shared__ int sm[];
  griddep_launch_dependents();
  if (blockIdx.x >= kSortCtas) {
    zero_rows(p, reinterpret_cast<uint32_t*>(sm), grad_bytes, blockIdx.x - kSortCtas, gridDim.x - kSortCtas);
    return;
  }
  int* hist = sm;                                // [kSortWarps][digits]
  const int digits = 1 << bits;
  int* tot = hist + kSortWarps * digits;         // [digits] this CTA's counts
  int* base = tot + digits;                      // [digits] where the CTA's pairs of a digit go
  int* warp_sum = base + digits;                 // [kSortWarps]
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
    auto key_at = [&](long i) { return pass > 0 ? kin[i] : key_of(p, i, true); };
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
    // exclusive sums over the warps, and the CTA's totals: kQuarter lanes a
    // digit, each a share of the warps
    for (int i = threadIdx.x; i < digits * kQuarter; i += kSortThreads) {
      const int d = i / kQuarter, w0 = (i % kQuarter) * (kSortWarps / kQuarter);
      int c[kSortWarps / kQuarter], sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps / kQuarter; ++w) c[w] = hist[(w0 + w) * digits + d];
#pragma unroll
      for (int w = 0; w < kSortWarps / kQuarter; ++w) {
        const int v = c[w];
        c[w] = sum;
        sum += v;
      }
      int before = sum;
#pragma unroll
      for (int o = 1; o < kQuarter; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o, kQuarter);
        if (i % kQuarter >= o) before += v;
      }
      if (i % kQuarter == kQuarter - 1) tot[d] = before;
      before -= sum;
#pragma unroll
      for (int w = 0; w < kSortWarps / kQuarter; ++w) hist[(w0 + w) * digits + d] = c[w] + before;
    }
    cluster.sync();
    // digits is at most the number of threads: thread d holds digit d
    int all = 0, before = 0;
    if (threadIdx.x < digits) {
      int c[kSortCtas];
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r) c[r] = cluster.map_shared_rank(tot, r)[threadIdx.x];
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r) {
        if (r < rank) before += c[r];
        all += c[r];
      }
    }
    int incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    // the digits before this warp's
    int ahead = lane < warp ? warp_sum[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
    if (threadIdx.x < digits) base[threadIdx.x] = incl - all + before + ahead;
    __syncthreads();
    for (long i = first + lane; i - lane < last; i += 32) {
      const bool in = i < last;
      const int k = in ? key_at(i) : 0;
      const int d = in ? (k >> shift) & (digits - 1) : digits;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      const int ahead = __popc(same & ((1u << lane) - 1u));
      int at = 0;
      if (in) at = base[d] + mine[d] + ahead;
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

// N values of a row of the gradient as they were; what is added to them, or 0.
template <typename G, int N>
__device__ __forceinline__ void load_row(const G* g, float (&f)[N]) {
  if constexpr (N == 1) {
    f[0] = to_f(*g);
  } else if constexpr (sizeof(G) == 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(g + i));
      f[i] = v.x;
      f[i + 1] = v.y;
      f[i + 2] = v.z;
      f[i + 3] = v.w;
    }
  } else {
    // bf16: N is 8, or 4 where dx is f32
    const uint32_t* w = reinterpret_cast<const uint32_t*>(g);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      f[i] = __uint_as_float(w[i / 2] << 16);
      f[i + 1] = __uint_as_float(w[i / 2] & 0xffff0000u);
    }
  }
}

// N values of a row of the gradient: scale * acc + was, rounded once.
template <typename G, int N, bool ADD>
__device__ __forceinline__ void finish(const EmbedParams& p, G* g, const float (&acc)[N], const float (&was)[N]) {
  float f[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    f[i] = p.scale * acc[i];
    if constexpr (ADD) f[i] += was[i];
  }
  if constexpr (N == 1) {
    put(g, f[0]);
  } else if constexpr (sizeof(G) == 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      __stcs(reinterpret_cast<float4*>(g + i), make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]));
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(g);
#pragma unroll
    for (int i = 0; i < N; i += 2) w[i / 2] = pack_bf16x2(f[i], f[i + 1]);
  }
}

// One block sums a chunk of kChunk sorted tokens over a slab of columns.  A
// run of equal ids inside the chunk is finished here; one that crosses the
// chunk's start or end leaves its part in part[2c] (the run that began
// earlier) or part[2c + 1] (the one that began here and goes on).  VEC: a
// thread has the columns of one 16-byte vector of dx, else one column.
// (Started while the sort still writes the pairs: key and pos are no
// __restrict__ pointers here and in the join, which would allow reads ahead of
// griddep_wait and past coherence.)
constexpr int kSumThreads = 128;
template <typename D, typename G, bool VEC, bool ADD>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(EmbedParams p, const int32_t* key,
                                                                const int32_t* pos) {
  constexpr int kN = VEC ? Vec<D>::kN : 1;
  __shared__ int keys[kChunk + 2], at[kChunk];  // keys[1 + i]; the neighbours' at the ends
  griddep_launch_dependents();
  griddep_wait();
  const long c0 = (long)blockIdx.x * kChunk;
  if (threadIdx.x < kChunk + 2) {
    const long i = c0 - 1 + threadIdx.x;
    keys[threadIdx.x] = i >= 0 && i < p.N ? key[i] : p.V;
  }
  if (threadIdx.x < kChunk && c0 + threadIdx.x < p.N) at[threadIdx.x] = pos[c0 + threadIdx.x];
  __syncthreads();
  const int col = (blockIdx.y * kSumThreads + threadIdx.x) * kN;
  if (col >= p.H) return;
  float acc[kN];
#pragma unroll
  for (int k = 0; k < kN; ++k) acc[k] = 0.0f;
  // (tokens that take no part have key V and come last)
  bool began_before = keys[1] < p.V && keys[0] == keys[1];
  constexpr int kAhead = 8;  // (16,384 tokens of 7,168 accumulated: 119 us, of four 122, of two 128)
#pragma unroll 1
  for (int i0 = 0; i0 < kChunk; i0 += kAhead) {
    if (keys[1 + i0] >= p.V) break;
    uint4 v[kAhead];
    float was[kAhead][kN];  // ADD: the rows whose runs end here, before
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if constexpr (ADD) {
        const int k = keys[1 + i0 + i];
        if (k < p.V && keys[2 + i0 + i] != k) load_row(static_cast<const G*>(p.dtable) + (long)k * p.H + col, was[i]);
      }
      v[i] = make_uint4(0, 0, 0, 0);
      if (keys[1 + i0 + i] < p.V) {
        const D* from = static_cast<const D*>(p.dx) + (long)at[i0 + i] * p.H + col;
        if constexpr (VEC)
          v[i] = __ldcs(reinterpret_cast<const uint4*>(from));
        else
          v[i].x = __float_as_uint(to_f(*from));
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = keys[1 + i0 + i];
      if (k >= p.V) break;
      float f[kN];
      if constexpr (VEC)
        Vec<D>::unpack(v[i], f);
      else
        f[0] = __uint_as_float(v[i].x);
#pragma unroll
      for (int c = 0; c < kN; ++c) acc[c] += f[c];
      const bool last = i0 + i + 1 == kChunk, goes_on = keys[2 + i0 + i] == k;
      if (goes_on && !last) continue;
      if (began_before || goes_on) {
        float* to = p.part + (2l * blockIdx.x + (began_before ? 0 : 1)) * p.H + col;
#pragma unroll
        for (int c = 0; c < kN; ++c) to[c] = acc[c];
      } else {
        finish<G, kN, ADD>(p, static_cast<G*>(p.dtable) + (long)k * p.H + col, acc, was[i]);
      }
#pragma unroll
      for (int c = 0; c < kN; ++c) acc[c] = 0.0f;
      began_before = false;
    }
  }
}

// Joins the runs that cross chunks: the block of the chunk where such a run
// began adds its parts in order.
template <typename G, bool VEC, bool ADD>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(EmbedParams p, const int32_t* key) {
  constexpr int kN = VEC ? 4 : 1;
  griddep_wait();
  const long c0 = (long)blockIdx.x * kChunk, end = c0 + kChunk;
  if (end >= p.N) return;
  const int k = key[end - 1];
  // a run that goes on past this chunk, and began in it
  if (k >= p.V || key[end] != k || (c0 > 0 && key[c0 - 1] == k)) return;
  // the chunks past this one that the run reaches: every warp looks 32 ahead
  int chunks = 1;
  for (bool more = true; more;) {
    const long i = end + (long)(chunks + (threadIdx.x & 31)) * kChunk;
    const uint32_t same = __ballot_sync(0xffffffffu, i < p.N && key[i] == k);
    more = same == 0xffffffffu;
    chunks += more ? 32 : __ffs(~same) - 1;
  }
  const int col = (blockIdx.y * kSumThreads + threadIdx.x) * kN;
  if (col < p.H) {
    float acc[kN], was[kN];
    G* to = static_cast<G*>(p.dtable) + (long)k * p.H + col;
    if constexpr (ADD) load_row(to, was);
    const float* from = p.part + (2l * blockIdx.x + 1) * p.H + col;
#pragma unroll
    for (int c = 0; c < kN; ++c) acc[c] = from[c];
    from += p.H;  // the next chunk's first part; then every other row
#pragma unroll 8
    for (int i = 0; i < chunks; ++i) {
      if constexpr (VEC) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(from + 2l * i * p.H));
        acc[0] += v.x;
        acc[1] += v.y;
        acc[2] += v.z;
        acc[3] += v.w;
      } else {
        acc[0] += from[2l * i * p.H];
      }
    }
    finish<G, kN, ADD>(p, to, acc, was);
  }
}

template <typename... Args>
cudaError_t launch_after(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t st, Args... args) {
  // programmatic dependent launch: the kernel's start hides behind the end of the one before
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename D, typename G, bool VEC, bool ADD>
cudaError_t launch_sums(const EmbedParams& p, int sorted, cudaStream_t st) {
  const unsigned chunks = (unsigned)((p.N + kChunk - 1) / kChunk);
  const int slab = kSumThreads * (VEC ? Vec<D>::kN : 1);
  const int32_t* key = p.key[sorted];
  const int32_t* pos = p.pos[sorted];
  cudaError_t e =
      launch_after(embed_sum_kernel<D, G, VEC, ADD>, dim3(chunks, (p.H + slab - 1) / slab), kSumThreads, st, p, key, pos);
  if (e != cudaSuccess) return e;
  const int joined = kSumThreads * (VEC ? 4 : 1);
  return launch_after(embed_join_kernel<G, VEC, ADD>, dim3(chunks, (p.H + joined - 1) / joined), kSumThreads, st, p, key);
}

bool rows_of_vectors(const void* p, int H, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (long)H * bytes % 16 == 0;
}

template <typename D, typename G>
cudaError_t launch_backward(const EmbedParams& p, int* launches, cudaStream_t st) {
  *launches = 0;
  if (p.N == 0) return p.accumulate ? cudaSuccess : cudaMemsetAsync(p.dtable, 0, (size_t)p.V * p.H * sizeof(G), st);
  const int sms = device_sm_count();
  int sorted = 0;  // where the pairs end
  int token_bits = 0;
  while ((1 << token_bits) < p.N) ++token_bits;
  if (p.N <= kRankTokens && p.V < (1ll << (32 - token_bits))) {
    // (both kinds of CTA fit an SM together)
    const int ranks = (p.N + kRankShare - 1) / kRankShare, zero = p.accumulate ? 0 : sms > 0 ? sms : 1;
    constexpr size_t kBytes = kMarkRows / 8 + kZeroBytes;
    static_assert(kRankTokens * 4 <= kBytes, "the keys fit");
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem((const void*)embed_rank_kernel, kBytes, allowed);
    if (e != cudaSuccess) return e;
    embed_rank_kernel<<<ranks + zero, kSortThreads, kBytes, st>>>(p, token_bits, ranks, (int)sizeof(G));
  } else {
    // keys are 0 .. V
    int key_bits = 3;  // (8 digits at least: kQuarter lanes each fill a warp)
    while (key_bits < 31 && (1 << key_bits) <= p.V) ++key_bits;
    const int passes = (key_bits + 9) / 10, bits = (key_bits + passes - 1) / passes;
    constexpr size_t kMost = ((size_t)(kSortWarps + 2) * kMaxDigits + kSortWarps) * 4;
    static_assert(kMarkRows / 8 + kZeroBytes <= kMost, "what marks and zeros rows fits the sort's shared memory");
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem((const void*)embed_sort_kernel, kMost, allowed);
    if (e != cudaSuccess) return e;
    // the zeros of the rows that no token has: by the clusters beside the sort's
    const int zero = p.accumulate ? 0 : sms > 2 * kSortCtas ? sms / kSortCtas - 1 : 1;
    embed_sort_kernel<<<kSortCtas * (1 + zero), kSortThreads, kMost, st>>>(p, bits, passes, (int)sizeof(G));
    sorted = passes & 1;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // a thread's vector of dx may be half of one of the gradient, or two
  const bool vec = rows_of_vectors(p.dx, p.H, sizeof(D)) && rows_of_vectors(p.dtable, p.H, sizeof(G));
  if (p.accumulate)
    e = vec ? launch_sums<D, G, true, true>(p, sorted, st) : launch_sums<D, G, false, true>(p, sorted, st);
  else
    e = vec ? launch_sums<D, G, true, false>(p, sorted, st) : launch_sums<D, G, false, false>(p, sorted, st);
  *launches = 3;
  return e;
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

template <typename T>
static cudaError_t launch_lookup(const EmbedParams& p, cudaStream_t st) {
  const bool vec = rows_of_vectors(p.table, p.H, sizeof(T)) && rows_of_vectors(p.out, p.H, sizeof(T));
  const int cols = vec ? p.H / Vec<T>::kN : p.H;
  const int pieces = (cols + 32 * kLookup - 1) / (32 * kLookup);
  const long blocks = ((long)p.N * pieces + 7) / 8;
  if (blocks > 0x7fffffffl) return cudaErrorInvalidValue;
  if (vec)
    embed_lookup_kernel<T, true><<<(unsigned)blocks, 256, 0, st>>>(p, pieces);
  else
    embed_lookup_kernel<T, false><<<(unsigned)blocks, 256, 0, st>>>(p, pieces);
  return cudaGetLastError();
}

cudaError_t launch_embed_forward(mok_dtype type, const EmbedParams& p, int* launches, cudaStream_t st) {
  *launches = 0;
  if (p.N == 0) return cudaSuccess;
  *launches = 1;
  return type == MOK_TYPE_BF16 ? launch_lookup<__nv_bfloat16>(p, st) : launch_lookup<float>(p, st);
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

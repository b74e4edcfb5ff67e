// The join of a block with its residual stream, forward and backward: the
// kernels, whose instances are spread over residual_*.cu.
//
//   z  = y r_y w_out,  r_y = (mean y^2 + eps)^(-1/2)      (or z = y)
//   d  = dropout(z)
//   x' = x + scale gate d
//   n  = x' r w_next,  r = (mean x'^2 + eps)^(-1/2)
//
// and from dx' and dn, with xh = x' r and yh = y r_y,
//
//   t  = dn w_next,  dx = dx' + r (t - xh mean(t xh)),     dw_next = sum_rows dn xh
//   db = scale dx,                                         dgate   = sum_rows db d
//   dz = dropout(db gate)
//   t' = dz w_out,   dy = r_y (t' - yh mean(t' yh)),       dw_out  = sum_rows dz yh
//
// Both passes are bound by HBM: every row is read once, kept on the chip
// between its sums and its outputs, and written once.  All arithmetic is in
// 32 bits; each output is rounded once.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "residual.cuh"
#include "rows.cuh"
#include "tc.cuh"

namespace mok {
namespace residual {

// ------------------------------------------------------------------ pairs
// Two f32 in a register pair: one instruction multiplies or adds both.  What
// bounds these kernels beside HBM is the number of instructions an element,
// and half of an unpacked one's are such.
typedef unsigned long long f2;

__device__ __forceinline__ f2 pair(float a, float b) {
  f2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ f2 both(float a) { return pair(a, a); }
__device__ __forceinline__ void split(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ float lo(f2 v) {
  float a, b;
  split(v, a, b);
  return a;
}
__device__ __forceinline__ float hi(f2 v) {
  float a, b;
  split(v, a, b);
  return b;
}
__device__ __forceinline__ float sum(f2 v) { return lo(v) + hi(v); }
__device__ __forceinline__ f2 mul(f2 a, f2 b) {
  f2 v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ f2 fma(f2 a, f2 b, f2 c) {
  f2 v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}

// ------------------------------------------------------------------ rows
// A row belongs to a team of NT threads (a warp, or a whole CTA), 8 NG
// elements each: thread t holds the eight from (g NT + t) 8 on.  ALIGNED: every row of
// every tensor is made of whole 16-byte vectors.
//
// In the last group a thread may have fewer elements, or none: then it works
// on the row's first ones beside their owner, and leaves them out of sums and
// stores, so that no branch stands around a group.
struct Place {
  int t, nt;
  int last;  // the first column of the thread's last group
  int n;     // how many of its elements there are (0: none), and of the next lane's (0 past the warp)
  int next;
  int held;  // how many it works on
};
template <int NG>
__device__ __forceinline__ Place place(int t, int nt, int H) {
  const int c = ((NG - 1) * nt + t) * 8;
  const int n = min(8, max(0, H - c)), next = (t & 31) < 31 ? min(8, max(0, H - c - 8)) : 0;
  return Place{t, nt, n > 0 ? c : 0, n, next, n > 0 ? n : min(8, H)};
}
template <int NG>
__device__ __forceinline__ int first_column(const Place& a, int g) {
  return g == NG - 1 ? a.last : (g * a.nt + a.t) * 8;
}
template <int NG>
__device__ __forceinline__ bool counts(const Place& a, int g) { return g < NG - 1 || a.n > 0; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E>
__device__ __forceinline__ E from_f32(float v) {
  if constexpr (sizeof(E) == 4) return v;
  else return __float2bfloat16_rn(v);
}

// Eight elements as four pairs.
struct Eight {
  f2 v[4];
};
__device__ __forceinline__ float squares(const Eight& a) {
  f2 s = mul(a.v[0], a.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma(a.v[i], a.v[i], s);
  return sum(s);
}
__device__ __forceinline__ Eight zeros() { return Eight{{0, 0, 0, 0}}; }
__device__ __forceinline__ Eight ones() { return Eight{{both(1.0f), both(1.0f), both(1.0f), both(1.0f)}}; }

template <typename E>
__device__ __forceinline__ Eight unpack(const uint32_t (&w)[words8<E>()]) {
  Eight r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 2) r.v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else r.v[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  return r;
}

// A tensor of rows and where it ends (its ends matter where rows are not aligned).
template <typename E>
struct Rows {
  E* p;
  long ld;
  Span8 span;
  __device__ __forceinline__ E* operator[](long row) const { return p + row * ld; }
};
template <typename E>
__device__ __forceinline__ Rows<const E> rows_in(const void* p, long ld, long rows, int H) {
  const E* q = static_cast<const E*>(p);
  return {q, ld, span_of(q, rows, ld, H)};
}
template <typename E>
__device__ __forceinline__ Rows<E> rows_out(void* p, long ld) {
  return {static_cast<E*>(p), ld, {0, 0}};
}

template <bool ALIGNED, int NG, typename E>
__device__ __forceinline__ Eight load8(const E* row, const Span8& span, int g, const Place& a) {
  uint32_t w[words8<E>()];
  load_words<E, ALIGNED>(row + first_column<NG>(a, g), g < NG - 1 ? 8 : a.held, span, w);
  return unpack<E>(w);
}
template <bool ALIGNED, int NG, typename E>
__device__ __forceinline__ Eight load8(const Rows<const E>& r, long row, int g, const Place& a) {
  return load8<ALIGNED, NG>(r[row], r.span, g, a);
}
template <bool ALIGNED, int NG, typename E>
__device__ __forceinline__ void store8(E* row, int g, const Place& a, const Eight& v) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) split(v.v[i], f[2 * i], f[2 * i + 1]);
  uint32_t w[words8<E>()];
#pragma unroll
  for (int i = 0; i < words8<E>(); ++i) {
    if constexpr (sizeof(E) == 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      w[i] = __float_as_uint(f[i]);
    }
  }
  E* at = row + first_column<NG>(a, g);
  if constexpr (ALIGNED) {
    if (counts<NG>(a, g)) store_words<E, true>(at, 8, 8, 0, w);
  } else {
    const int lane = a.t & 31;
    store_words<E, false>(at, g < NG - 1 ? 8 : a.n, g < NG - 1 ? (lane < 31 ? 8 : 0) : a.next, lane, w);
  }
}

// A row of f32 in shared memory, on a vector boundary and as long as whole vectors.
template <int NG>
__device__ __forceinline__ Eight shared8(const float* row, int g, const Place& a) {
  const float* at = row + first_column<NG>(a, g);
  const int n = g < NG - 1 ? 8 : a.held;
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = e < n ? at[e] : 0.0f;
  return Eight{{pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7])}};
}

__device__ __forceinline__ float product(const Eight& a, const Eight& b) {
  f2 s = mul(a.v[0], b.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma(a.v[i], b.v[i], s);
  return sum(s);
}

// ------------------------------------------------------------------ teams
// A team of 32 threads is one of the CTA's warps; a larger one is the CTA.
__device__ __forceinline__ void team_sync(int nt) {
  if (nt > 32) __syncthreads();
  else __syncwarp();
}

// Eight sums over a warp in nine exchanges: lanes 4 i .. 4 i + 3 have the i-th.
__device__ __forceinline__ float warp_sum8(const float (&v)[8], int lane) {
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 16;
    a[i] = up ? v[4 + i] : v[i];
    a[i] += __shfl_xor_sync(0xffffffffu, up ? v[i] : v[4 + i], 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 8;
    b[i] = up ? a[2 + i] : a[i];
    b[i] += __shfl_xor_sync(0xffffffffu, up ? a[i] : a[2 + i], 8);
  }
  const bool up = lane & 4;
  float s = up ? b[1] : b[0];
  s += __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 4);
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  return s + __shfl_xor_sync(0xffffffffu, s, 1);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums over the team, in a fixed order.  Two areas of shared memory in turn
// (`which`), so that one barrier a sum is enough: an area is written again
// only after the barrier of the sum between.
struct Slots {
  float4 eight[2][32][2];
};
__device__ __forceinline__ void team_sum8(float (&v)[8], int t, int nt, Slots& slots, int& which) {
  const int lane = t & 31;
  float s = warp_sum8(v, lane);
  if (nt > 32) {
    float4(*area)[2] = slots.eight[which];
    which ^= 1;
    if ((lane & 3) == 0) reinterpret_cast<float*>(area[t >> 5])[lane >> 2] = s;
    __syncthreads();
    const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float4 x = lane < (nt >> 5) ? area[lane][0] : none, y = lane < (nt >> 5) ? area[lane][1] : none;
    const float u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    s = warp_sum8(u, lane);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(0xffffffffu, s, 4 * i);
}
__device__ __forceinline__ float team_sum(float v, int t, int nt, Slots& slots, int& which) {
  v = warp_sum(v);
  if (nt == 32) return v;
  float* area = reinterpret_cast<float*>(slots.eight[which]);
  which ^= 1;
  if ((t & 31) == 0) area[t >> 5] = v;
  __syncthreads();
  return warp_sum((t & 31) < (nt >> 5) ? area[t & 31] : 0.0f);
}

// ------------------------------------------------------------------ dropout
// Eight elements' keep bits.  ALIGNED: the row's elements from a multiple of
// eight are one of the generator's blocks.  Otherwise they lie in two, and the
// team makes the row's blocks together, a byte each, in `bytes` (shared, (H +
// 14) / 8 + 1 of them), of which every thread picks its bits.
__device__ __forceinline__ void keep_bytes(const DropParams& d, uint64_t call, uint64_t first, int H, int t, int nt,
                                           uint8_t* bytes) {
  const uint64_t b0 = first >> 3;
  const int n = (int)(((first + H - 1) >> 3) - b0) + 1;
  team_sync(nt);
  for (int i = t; i < n; i += nt) bytes[i] = (uint8_t)drop_keep8(d, b0 + i, call);
  team_sync(nt);
}
struct KeepBits {
  uint32_t bits;
  __device__ __forceinline__ bool operator()(int j) const { return (bits >> j) & 1u; }
};
struct KeepBlock {
  uint4 r;
  uint32_t most;
  __device__ __forceinline__ bool operator()(int j) const { return drop_kept(r, j, most); }
};
// (Words need no bits made of them first, but registers, of which threads with four groups have none to spare: 8,192 rows
// of 7,168 bf16, two groups, backward with dropout: bits 212 us, words 188; 4,096 of 12,288, four: 293 and 401, and
// 265 and 366 where the same kernel is called without dropout.)
template <bool ALIGNED, int NG>
using Keep = std::conditional_t<ALIGNED && NG <= 2, KeepBlock, KeepBits>;
template <bool ALIGNED, int NG>
__device__ __forceinline__ Keep<ALIGNED, NG> keep8(const DropParams& d, uint64_t call, uint64_t first, int g, const Place& a,
                                                   const uint8_t* bytes) {
  const int c = first_column<NG>(a, g);
  if constexpr (ALIGNED && NG <= 2) {
    return {drop_block(d, (first + c) >> 3, call), drop_most(d)};
  } else if constexpr (ALIGNED) {
    return {drop_keep8(d, (first + c) >> 3, call)};
  } else {
    const uint32_t at = (uint32_t)(first & 7) + c;
    uint32_t keep = bytes[at >> 3] >> (at & 7);
    // (the byte after is there if one of its elements is the row's)
    if ((at & 7) + (g < NG - 1 ? 8 : a.held) > 8) keep |= (uint32_t)bytes[(at >> 3) + 1] << (8 - (at & 7));
    return {keep};
  }
}
// (a dropped element is 0 whatever it was)
template <typename K>
__device__ __forceinline__ void drop8(Eight& v, const K& keep) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    split(v.v[i], a, b);
    v.v[i] = pair(keep(2 * i) ? a : 0.0f, keep(2 * i + 1) ? b : 0.0f);
  }
}

// ------------------------------------------------------------------ rows ahead
// A thread's elements of the rows to come lie in shared memory, brought there
// by its own 16-byte asynchronous copies, so that no register and no barrier
// stands between HBM and the rows at work: a plane of 16 bytes a thread per
// stage, tensor, group and vector that its eight elements touch.
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most n (uniform, 0 to 3) of the thread's last groups are on their way.
__device__ __forceinline__ void copies_wait(int n) {
  if (n == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// `at`: the tensor's first plane of the stage, this thread's 16 bytes.
template <bool ALIGNED, int NG, typename E>
__device__ __forceinline__ void row_ahead(uint4* at, const Rows<const E>& r, long row, const Place& a) {
  const E* from = r[row];
#pragma unroll
  for (int g = 0; g < NG; ++g)
    copy_words<E, ALIGNED>(at + g * vectors8<E, ALIGNED>() * a.nt, a.nt, from + first_column<NG>(a, g),
                           g < NG - 1 ? 8 : a.held, r.span);
}
// Group g of a row that was brought ahead.
template <bool ALIGNED, int NG, typename E>
__device__ __forceinline__ Eight held8(const uint4* at, const Rows<const E>& r, long row, int g, const Place& a) {
  uint32_t w[words8<E>()];
  copied_words<E, ALIGNED>(at + g * vectors8<E, ALIGNED>() * a.nt, a.nt, r[row] + first_column<NG>(a, g),
                           g < NG - 1 ? 8 : a.held, w);
  return unpack<E>(w);
}

// The same of rows that are not aligned, put back in place as whole vectors for those who read it again (8,192 rows of
// 4,099 bf16, backward: shifted twice 283 us, once 255).
template <int NG, typename E>
__device__ __forceinline__ Eight placed8(uint4* at, const Rows<const E>& r, long row, int g, const Place& a) {
  uint4* v = at + g * vectors8<E, false>() * a.nt;
  uint32_t w[words8<E>()];
  copied_words<E, false>(v, a.nt, r[row] + first_column<NG>(a, g), g < NG - 1 ? 8 : a.held, w);
#pragma unroll
  for (int i = 0; i < words8<E>() / 4; ++i) v[i * a.nt] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  return unpack<E>(w);
}
template <typename E>
__device__ __forceinline__ Eight again8(const uint4* at, const Rows<const E>& r, int g, const Place& a) {
  uint32_t w[words8<E>()];
  copied_words<E, true>(at + g * vectors8<E, false>() * a.nt, a.nt, r.p, 8, w);
  return unpack<E>(w);
}

// ------------------------------------------------------------------ what a call has
// A kernel that has to ask row by row what there is spends as many
// instructions on that as on the elements (8,192 rows of 7,168 bf16, backward:
// 197 us, with the answers compiled in 123).  So the usual combinations have
// kernels of their own, named by these bits (with x and y, their gradients
// and the gradient of x' all there); any other is asked for.
enum Parts { kAnything = -1, kNext = 1, kOut = 2, kDrop = 4 };

// ------------------------------------------------------------------ forward
constexpr int kTeamRows = 8;  // rows, a warp each, in a CTA where a warp holds a row

// AHEAD: the rows come through shared memory, `stages` rows ahead; otherwise
// straight from global memory.
template <typename S, typename B, bool ALIGNED, int NG, bool AHEAD, int PARTS>
__global__ void __launch_bounds__(512, NG <= 2 ? 2 : 1) residual_forward_kernel(const ResidualParams p, int stages) {
  extern __shared__ uint4 shared[];
  __shared__ Slots slots;
  const int t = threadIdx.x, nt = blockDim.x, H = p.H;
  const int team = blockIdx.x * blockDim.y + threadIdx.y, teams = gridDim.x * blockDim.y;
  if (team >= p.T) return;  // (a whole team: a warp of its own, or the whole CTA)
  const bool has_y = PARTS != kAnything || p.y, has_out = PARTS == kAnything ? p.w_out != nullptr : PARTS & kOut;
  const bool to_next = PARTS == kAnything ? p.n != nullptr : PARTS & kNext;
  const bool drops = PARTS == kAnything ? p.drop.below != 0 : PARTS & kDrop;
  const Place a = place<NG>(t, nt, H);
  const float rH = 1.0f / (float)H;
  constexpr int kS = NG * vectors8<S, ALIGNED>(), kB = NG * vectors8<B, ALIGNED>(), kStage = kS + kB;  // planes
  uint4* mine = shared + threadIdx.y * (AHEAD ? stages * kStage * nt : 0) + t;
  uint8_t* bytes = reinterpret_cast<uint8_t*>(shared + blockDim.y * (AHEAD ? stages * kStage * nt : 0)) +
                   threadIdx.y * ((H + 14) / 8 + 1);
  const auto xs = rows_in<S>(p.x, p.ldx, p.T, H);
  const auto ys = rows_in<B>(p.y, p.ldy, p.T, H), gates = rows_in<B>(p.gate, H, p.G, H);
  const auto w_out = rows_in<B>(p.w_out, H, 1, H), w_next = rows_in<B>(p.w_next, H, 1, H);
  const auto xo = rows_out<S>(p.xo, p.ldxo);
  const auto n = rows_out<B>(p.n, p.ldn);
  auto ahead = [&](long row, int stage) {
    if (row < p.T) {
      row_ahead<ALIGNED, NG>(mine + stage * kStage * nt, xs, row, a);
      if (has_y) row_ahead<ALIGNED, NG>(mine + (stage * kStage + kS) * nt, ys, row, a);
    }
    copies_commit();
  };
  if constexpr (AHEAD)
    for (int i = 0; i < stages; ++i) ahead(team + (long)i * teams, i);
  const uint64_t call = drops ? drop_call(p.drop) : 0;
  const float scale = drops ? p.scale * p.drop.scale : p.scale;
  int stage = 0, which = 0;
  for (long row = team; row < p.T; row += teams) {
    Eight x[NG];
    auto get_x = [&](int g) {
      if constexpr (AHEAD) return held8<ALIGNED, NG>(mine + stage * kStage * nt, xs, row, g, a);
      else return load8<ALIGNED, NG>(xs, row, g, a);
    };
    if constexpr (AHEAD) copies_wait(stages - 1);
    if (has_y) {
      Eight z[NG];
      if constexpr (!AHEAD) {
        // (all of a row's loads together)
#pragma unroll
        for (int g = 0; g < NG; ++g) x[g] = get_x(g);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if constexpr (AHEAD) z[g] = held8<ALIGNED, NG>(mine + (stage * kStage + kS) * nt, ys, row, g, a);
        else z[g] = load8<ALIGNED, NG>(ys, row, g, a);
      }
      float factor = scale;
      if (has_out) {
        float s = 0.0f;
#pragma unroll
        for (int g = 0; g < NG; ++g) s += counts<NG>(a, g) ? squares(z[g]) : 0.0f;
        factor *= rsqrtf(fmaf(team_sum(s, t, nt, slots, which), rH, p.eps));
      }
      const uint64_t first = (uint64_t)row * (uint64_t)H;
      if (!ALIGNED && drops) keep_bytes(p.drop, call, first, H, t, nt, bytes);
      const uint32_t group = p.G ? (uint32_t)row / (uint32_t)p.rows_per_gate : 0;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if constexpr (AHEAD) x[g] = get_x(g);
        Keep<ALIGNED, NG> keep = {};
        if (drops) keep = keep8<ALIGNED, NG>(p.drop, call, first, g, a, bytes);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[g].v[i] = mul(z[g].v[i], both(factor));
        if (has_out) {
          const Eight w = load8<ALIGNED, NG>(w_out, 0, g, a);
#pragma unroll
          for (int i = 0; i < 4; ++i) z[g].v[i] = mul(z[g].v[i], w.v[i]);
        }
        // (of z as it is: a norm or a weight that is not finite reaches no dropped element)
        if (drops) drop8(z[g], keep);
        const Eight f = p.G ? load8<ALIGNED, NG>(gates, group, g, a) : ones();
#pragma unroll
        for (int i = 0; i < 4; ++i) x[g].v[i] = fma(z[g].v[i], f.v[i], x[g].v[i]);
        store8<ALIGNED, NG>(xo[row], g, a, x[g]);
      }
    } else {
#pragma unroll
      for (int g = 0; g < NG; ++g) x[g] = get_x(g);
    }
    if constexpr (AHEAD) {
      // (the thread's values of this stage are in its registers)
      ahead(row + (long)stages * teams, stage);
      if (++stage == stages) stage = 0;
    }
    if (!to_next) continue;
    float s = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) s += counts<NG>(a, g) ? squares(x[g]) : 0.0f;
    const float r = rsqrtf(fmaf(team_sum(s, t, nt, slots, which), rH, p.eps));
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const Eight w = load8<ALIGNED, NG>(w_next, 0, g, a);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[g].v[i] = mul(mul(x[g].v[i], both(r)), w.v[i]);
      store8<ALIGNED, NG>(n[row], g, a, x[g]);
    }
  }
}

// ------------------------------------------------------------------ backward
// The rows are cut into units, no unit across two gate rows' rows: G * split
// of them, or as many as workers where there is no gate.  A worker (a team)
// takes whole units.  It sums two things over its rows, by column:
//
//   sum_next = sum dn xh,   sum_y = sum dropout(dx) yh  over a unit
//
// Within a unit the gate is one row, so both other gradients follow from
// sum_y: dw_out = sum over units of scale gate sum_y, dgate = scale w_out
// sum_y.  (Without w_out, yh stands for y.)  The sums of a CTA's workers are
// joined in the order of the teams, those of CTAs and units by a second
// kernel in their order.  With more gate rows than workers (`own`) a unit is
// a gate row's rows: its worker writes that row of dgate itself and sums its
// share of dw_out in shared memory; the gate rows are brought ahead with the
// rows.
struct BackwardPlan {
  int workers;   // teams
  int groups;    // rows of the gate, 1 without
  int split;     // units per group
  int own;       // split is 1 and there are several gate rows
  int ctas;      // CTAs: the parts of dw_next and dw_out
};

// A worker's rows, one after the other.
struct Walk {
  int unit, group;
  long row, end;  // the row at hand and the end of its unit
};
__device__ __forceinline__ void walk_unit(Walk& w, const ResidualParams& p, const BackwardPlan& plan) {
  const long per = p.T / plan.groups;
  w.group = w.unit / plan.split;
  const int part = w.unit - w.group * plan.split;
  w.row = w.group * per + per * part / plan.split;
  w.end = w.group * per + per * (part + 1) / plan.split;
}
__device__ __forceinline__ bool walk_on(Walk& w, const ResidualParams& p, const BackwardPlan& plan) {
  if (++w.row < w.end) return true;
  w.unit += plan.workers;
  if (w.unit >= plan.groups * plan.split) return false;
  walk_unit(w, p, plan);
  return true;
}

// Bytes of a row of f32 in shared memory, and of a team's shared memory beside its stages: two such rows (its share of
// dw_out; what is joined at the end), and the keep bytes.
__host__ __device__ __forceinline__ size_t row_f32(int H) { return (size_t)(H + 3) / 4 * 16; }
__host__ __device__ __forceinline__ size_t backward_beside(int H, bool bytes, bool own, bool several) {
  return (own ? row_f32(H) : 0) + (several ? row_f32(H) : 0) + (bytes ? ((H + 14) / 8 + 16) / 16 * 16 : 0);
}

template <typename S, typename B, bool ALIGNED, int NG, bool AHEAD, int PARTS>
__global__ void __launch_bounds__(NG == 1 ? 256 : 512, NG == 1 ? 3 : 1)
    residual_backward_kernel(const ResidualParams p, const BackwardPlan plan, int stages) {
  extern __shared__ uint4 shared[];
  __shared__ Slots slots;
  const int t = threadIdx.x, nt = blockDim.x, H = p.H;
  const int worker = blockIdx.x * blockDim.y + threadIdx.y;
  constexpr bool kAsk = PARTS == kAnything;
  const bool has_dxo = !kAsk || p.dxo, to_x = !kAsk || p.dx, to_y = !kAsk || p.dy;
  const bool has_dn = kAsk ? p.dn != nullptr : PARTS & kNext, has_out = kAsk ? p.w_out != nullptr : PARTS & kOut;
  const bool has_y = !kAsk && (PARTS & kOut) ? true : p.y != nullptr, drops = kAsk ? p.drop.below != 0 : PARTS & kDrop;
  const Place a = place<NG>(t, nt, H);
  const float rH = 1.0f / (float)H;
  const auto dxos = rows_in<S>(p.dxo, p.lddxo, p.T, H), xs = rows_in<S>(p.x, p.ldx, p.T, H);
  const auto dns = rows_in<B>(p.dn, p.lddn, p.T, H), ys = rows_in<B>(p.y, p.ldy, p.T, H);
  const auto gates = rows_in<B>(p.gate, H, p.G, H), w_out = rows_in<B>(p.w_out, H, 1, H),
             w_next = rows_in<B>(p.w_next, H, 1, H);
  const auto dx = rows_out<S>(p.dx, p.lddx);
  const auto dy = rows_out<B>(p.dy, p.lddy);
  const uint64_t call = drops ? drop_call(p.drop) : 0;
  // a stage's planes: dxo, x, dn, y
  constexpr int kS = NG * vectors8<S, ALIGNED>(), kB = NG * vectors8<B, ALIGNED>();
  const int stage_planes = 2 * (kS + kB) + (plan.own ? kB : 0);  // (and the gate row)
  const int team_planes = AHEAD ? stages * stage_planes * nt : 0;
  uint4* mine = shared + threadIdx.y * team_planes + t;
  const bool several = blockDim.y > 1;
  const size_t beside_bytes = backward_beside(H, !ALIGNED && drops, plan.own, several);
  uint8_t* all_beside = reinterpret_cast<uint8_t*>(shared + blockDim.y * team_planes);
  uint8_t* beside = all_beside + threadIdx.y * beside_bytes;
  float* share = reinterpret_cast<float*>(beside);  // whole vectors of its own: a thread's eight are its alone
  const size_t join_at = plan.own ? row_f32(H) : 0;
  uint8_t* bytes = beside + join_at + (several ? row_f32(H) : 0);
  Eight sum_next[NG], sum_y[NG];
  // the weights of the thread's columns: of the norm before the next block, and what stands between dx and t', the
  // gate and w_out (`scale` and dropout's factor come in at the end)
  Eight wn[NG], f[NG];
  auto unit_weights = [&](int group, const uint4* held) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f[g] = held ? held8<ALIGNED, NG>(held, gates, group, g, a) : p.G ? load8<ALIGNED, NG>(gates, group, g, a) : ones();
      if (has_out) {
        const Eight w = load8<ALIGNED, NG>(w_out, 0, g, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[g].v[i] = mul(f[g].v[i], w.v[i]);
      }
    }
  };
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    wn[g] = has_dn ? load8<ALIGNED, NG>(w_next, 0, g, a) : zeros();
    sum_next[g] = sum_y[g] = zeros();
    if (plan.own) store8<ALIGNED, NG>(share, g, a, zeros());
  }

  // (a worker without a unit: no rows, sums of zero)
  Walk at = {worker, 0, 0, 0};
  if (worker < plan.workers && worker < plan.groups * plan.split) walk_unit(at, p, plan);
  bool more = at.row < at.end;
  if (more && !(AHEAD && plan.own)) unit_weights(at.group, nullptr);
  Walk next = at;
  bool more_next = more, fresh = true, fresh_next = true;  // (the first row of a unit)
  auto ahead = [&](int stage) {
    if (more_next) {
      uint4* m = mine + stage * stage_planes * nt;
      if (has_dxo) row_ahead<ALIGNED, NG>(m, dxos, next.row, a);
      if (has_dn) {
        row_ahead<ALIGNED, NG>(m + kS * nt, xs, next.row, a);
        row_ahead<ALIGNED, NG>(m + 2 * kS * nt, dns, next.row, a);
      }
      if (has_y) row_ahead<ALIGNED, NG>(m + (2 * kS + kB) * nt, ys, next.row, a);
      if (plan.own && fresh_next) row_ahead<ALIGNED, NG>(m + 2 * (kS + kB) * nt, gates, next.group, a);
      const int unit = next.unit;
      more_next = walk_on(next, p, plan);
      fresh_next = next.unit != unit;
    }
    copies_commit();
  };
  if constexpr (AHEAD)
    for (int i = 0; i < stages; ++i) ahead(i);
  int stage = 0, which = 0;
  while (more) {
    // A row's values are read again where they are used again (from shared memory, or the second time from L1):
    // what stays in registers over the barrier is the columns' sums.
    const long row = at.row;
    uint4* m = mine + stage * stage_planes * nt;
    auto get = [&](int plane, const auto& rows, int g) {
      if constexpr (AHEAD && !ALIGNED) return placed8<NG>(m + plane * nt, rows, row, g, a);
      else if constexpr (AHEAD) return held8<true, NG>(m + plane * nt, rows, row, g, a);
      else return load8<ALIGNED, NG>(rows, row, g, a);
    };
    auto get_again = [&](int plane, const auto& rows, int g, bool seen) {
      if constexpr (AHEAD && !ALIGNED) return seen ? again8(m + plane * nt, rows, g, a) : held8<false, NG>(m + plane * nt, rows, row, g, a);
      else if constexpr (AHEAD) return held8<true, NG>(m + plane * nt, rows, row, g, a);
      else return load8<ALIGNED, NG>(rows, row, g, a);
    };
    constexpr int kDxo = 0, kX = kS, kDn = 2 * kS, kY = 2 * kS + kB;
    const bool norm_y = has_out && has_y;  // (y, and dx' with it, are in the sums)
    const uint64_t first = (uint64_t)row * (uint64_t)H;
    if constexpr (AHEAD) {
      copies_wait(stages - 1);
      if (plan.own && fresh) unit_weights(at.group, m + 2 * (kS + kB) * nt);
    }
    if (!ALIGNED && drops && to_y) keep_bytes(p.drop, call, first, H, t, nt, bytes);
    Keep<ALIGNED, NG> keep[NG];
    // Sums of y^2, x'^2, t x' and, with f as above and y, of dx' f y, t f y, x' f y: as dx is linear in the first
    // norm's two factors, sum t' y follows from those three, and all of a row's sums are made at once.
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float u[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      Eight fy = zeros();
      if (drops && to_y) keep[g] = keep8<ALIGNED, NG>(p.drop, call, first, g, a, bytes);
      if (norm_y) {
        const Eight y = get(kY, ys, g);
        u[0] = squares(y);
#pragma unroll
        for (int i = 0; i < 4; ++i) fy.v[i] = mul(f[g].v[i], y.v[i]);
        if (drops) drop8(fy, keep[g]);
      }
      if (has_dxo && norm_y) {
        Eight d = get(kDxo, dxos, g);
        if (drops) drop8(d, keep[g]);  // (a dropped gradient may be anything too)
        u[3] = product(d, fy);
      }
      if (has_dn) {
        const Eight x = get(kX, xs, g);
        Eight v = get(kDn, dns, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.v[i] = mul(v.v[i], wn[g].v[i]);
        u[1] = squares(x);
        u[2] = product(v, x);
        u[4] = product(v, fy);
        u[5] = product(x, fy);
      }
#pragma unroll
      for (int i = 0; i < 6; ++i) s[i] += counts<NG>(a, g) ? u[i] : 0.0f;
    }
    if (has_dn || has_out) team_sum8(s, t, nt, slots, which);
    const float ry = has_out ? rsqrtf(fmaf(s[0], rH, p.eps)) : 1.0f, r = rsqrtf(fmaf(s[1], rH, p.eps));
    const float mean = s[2] * rH * r * r;  // mean(t xh) r / r
    const float mean_y = (s[3] + r * (s[4] - mean * s[5])) * rH * ry * ry;  // mean(t' yh) ry / ry
    const float factor = (drops ? p.scale * p.drop.scale : p.scale) * ry;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      Eight d = has_dxo ? get_again(kDxo, dxos, g, norm_y) : zeros();
      if (has_dn) {
        const Eight x = get_again(kX, xs, g, true), v = get_again(kDn, dns, g, true);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum_next[g].v[i] = fma(v.v[i], mul(x.v[i], both(r)), sum_next[g].v[i]);
          d.v[i] = fma(both(r), fma(both(-mean), x.v[i], mul(v.v[i], wn[g].v[i])), d.v[i]);
        }
      }
      Eight y = zeros();
      if (has_y) y = get_again(kY, ys, g, norm_y);
      if (to_x) store8<ALIGNED, NG>(dx[row], g, a, d);
      if (!to_y) continue;
      // the branch
      if (drops) drop8(d, keep[g]);
      if (has_y) {
        Eight u = y;
        if (drops) drop8(u, keep[g]);  // (a dropped y may be anything, an infinity too)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum_y[g].v[i] = fma(d.v[i], mul(u.v[i], both(ry)), sum_y[g].v[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d.v[i] = mul(d.v[i], f[g].v[i]);
        if (has_out) d.v[i] = fma(both(-mean_y), y.v[i], d.v[i]);
        d.v[i] = mul(d.v[i], both(factor));
      }
      store8<ALIGNED, NG>(dy[row], g, a, d);
    }
    const int unit = at.unit, group = at.group;
    more = walk_on(at, p, plan);
    const bool ends = !more || at.unit != unit;
    if (ends && plan.own) {
      // the unit ends: its row of dgate, its share of dw_out
      const float scale = drops ? p.scale * p.drop.scale : p.scale;
      const bool held = AHEAD && fresh;  // (a unit of one row: its gate is still there)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        Eight v = sum_y[g];
#pragma unroll
        for (int i = 0; i < 4; ++i) v.v[i] = mul(v.v[i], both(scale));
        if (p.dw_out) {
          const Eight gate = held ? held8<ALIGNED, NG>(m + 2 * (kS + kB) * nt, gates, group, g, a)
                                  : load8<ALIGNED, NG>(gates, group, g, a);
          Eight sh = shared8<NG>(share, g, a);
#pragma unroll
          for (int i = 0; i < 4; ++i) sh.v[i] = fma(v.v[i], gate.v[i], sh.v[i]);
          store8<ALIGNED, NG>(share, g, a, sh);
        }
        if (p.dgate) {
          if (has_out) {
            const Eight w = load8<ALIGNED, NG>(w_out, 0, g, a);
#pragma unroll
            for (int i = 0; i < 4; ++i) v.v[i] = mul(v.v[i], w.v[i]);
          }
          store8<ALIGNED, NG>(static_cast<B*>(p.dgate) + (long)group * H, g, a, v);
        }
        sum_y[g] = zeros();
      }
      if (!AHEAD && more) unit_weights(at.group, nullptr);
    }
    fresh = ends;
    if constexpr (AHEAD) {
      ahead(stage);
      if (++stage == stages) stage = 0;
    }
  }

  // (the kernel that joins the sums may start, and waits for this one's end; started with the first rows it cost the
  // others' time: 8,192 rows of 7,168, 129 -> 134 us)
  griddep_launch_dependents();
  // What is left (a worker has one unit at most unless it wrote them itself): its sums into the parts, those of a CTA's
  // teams as one where they are of the same columns' whole.
  const long cta = blockIdx.x;
  auto join = [&](float* part, auto&& value) {
    if (several) {
      float* rows = reinterpret_cast<float*>(all_beside + join_at);
      const size_t apart = beside_bytes / 4;
      __syncthreads();
#pragma unroll
      for (int g = 0; g < NG; ++g) store8<ALIGNED, NG>(rows + threadIdx.y * apart, g, a, value(g));
      __syncthreads();
      for (int c = threadIdx.y * nt + t; c < H; c += blockDim.y * nt) {
        float v = 0.0f;
        for (int i = 0; i < (int)blockDim.y; ++i) v += rows[i * apart + c];
        part[c] = v;
      }
    } else {
#pragma unroll
      for (int g = 0; g < NG; ++g) store8<ALIGNED, NG>(part, g, a, value(g));
    }
  };
  if (p.dw_next) join(p.part + cta * H, [&](int g) { return sum_next[g]; });
  if (p.dw_out) {
    // (by the gate: f without w_out)
    const bool gated = p.G && !plan.own && worker < plan.groups * plan.split;
    join(p.part + (plan.ctas + cta) * H, [&](int g) {
      if (plan.own) return shared8<NG>(share, g, a);
      Eight v = sum_y[g];
      if (gated) {
        const Eight gate = load8<ALIGNED, NG>(gates, worker / plan.split, g, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.v[i] = mul(v.v[i], gate.v[i]);
      }
      return v;
    });
  }
  if (p.dgate && !plan.own) {
    float* part = p.part + 2l * plan.ctas * H;
    if (plan.groups == 1) {
      join(part + cta * H, [&](int g) { return sum_y[g]; });
    } else if (worker < plan.groups * plan.split) {
#pragma unroll
      for (int g = 0; g < NG; ++g) store8<ALIGNED, NG>(part + (long)worker * H, g, a, sum_y[g]);
    }
  }
}

// Joins the parts: 32 columns a CTA, 16 threads a column, each over every 16th
// part and then in order.  Row 0 of the grid is dw_next, row 1 dw_out, then the rows of dgate.
constexpr int kJoinRows = 16;
template <typename B>
__global__ void __launch_bounds__(32 * kJoinRows) residual_join_kernel(const ResidualParams p, const BackwardPlan plan) {
  __shared__ float sums[kJoinRows][33];
  const int c = blockIdx.x * 32 + threadIdx.x, what = blockIdx.y;
  griddep_wait();
  if ((what == 0 && !p.dw_next) || (what == 1 && !p.dw_out)) return;
  const int n = what < 2 || plan.groups == 1 ? plan.ctas : plan.split;
  const float* part = p.part + ((what < 2 ? (long)what : 2l) * plan.ctas + (what < 2 ? 0l : (long)(what - 2) * n)) * p.H;
  float s = 0.0f;
  if (c < p.H) {
#pragma unroll 8
    for (int i = threadIdx.y; i < n; i += kJoinRows) s += part[(long)i * p.H + c];
  }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= p.H) return;
#pragma unroll
  for (int i = 1; i < kJoinRows; ++i) s += sums[i][threadIdx.x];
  const float scale = p.drop.below ? p.scale * p.drop.scale : p.scale;
  if (what == 0) {
    p.dw_next[c] = s;
  } else if (what == 1) {
    p.dw_out[c] = plan.own ? s : s * scale;
  } else {
    s *= scale;
    if (p.w_out) s *= to_f32(static_cast<const B*>(p.w_out)[c]);
    static_cast<B*>(p.dgate)[(long)(what - 2) * p.H + c] = from_f32<B>(s);
  }
}

// ------------------------------------------------------------------ launches
// Shared memory of the rows ahead, over all of an SM's CTAs: enough for what HBM has on its way, and the rest left to
// L1 for the weights (which the backward pass has in registers).
constexpr size_t kAheadBytes = 176 * 1024, kAheadBytesBackward = 200 * 1024;
constexpr size_t kMostSmem = 227 * 1024 - sizeof(Slots);
constexpr int kMaxStages = 4;

inline int team_threads(int H, int ng) { return ((H + 8 * ng - 1) / (8 * ng) + 31) / 32 * 32; }
inline int groups_forward(int H) { return H <= 4096 ? 1 : H <= 8192 ? 2 : 4; }
// A warp holds rows of up to 512 columns, which need no barrier. Of longer ones at any alignment the shifts, not the
// registers, are what counts, and more threads hide them (8,192 rows of 515 bf16, dropout: two groups 81 us, one 56; of
// 1,003 84 and 69; of 2,043 without dropout 108 and 118; aligned, 4,096 of 2,048: 29 and 35).
inline int groups_backward(int H, bool aligned) {
  return H <= 256 || (!aligned && H > 512 && H <= 1536) ? 1 : H <= 8192 ? 2 : 4;
}
// CTAs that an SM holds (registers).
inline int ctas_forward(int threads, int ng) { return std::max(1, (ng <= 2 ? 1024 : 512) / threads); }
inline int ctas_backward(int threads, int ng) { return std::max(1, (ng == 1 ? 768 : 512) / threads); }

// How many rows ahead a CTA's share of the memory holds (0: not two at least).
inline int stages_ahead(size_t room, size_t stage, size_t beside) {
  const int stages = room > beside ? std::min<int>(kMaxStages, (int)((room - beside) / stage)) : 0;
  return stages >= 2 ? stages : 0;
}

// All the teams that the SMs hold; where there are few rows, four of them at least for a team, so that the parts stay few
// beside the rows, but teams for four on every SM (64 rows of 7,168 bf16: 16.4 us with four rows each, 9.1 with one).
inline BackwardPlan backward_plan(int T, int G, int teams, int rows) {
  BackwardPlan b;
  b.workers = std::max(1, std::min(teams, std::max((T + 3) / 4, std::min(T, 4 * device_sm_count()))));
  b.groups = std::max(1, G);
  b.split = std::max(1, std::min(b.workers / b.groups, T / b.groups));
  b.own = b.split == 1 && b.groups > 1;
  b.ctas = (b.workers + rows - 1) / rows;
  return b;
}

template <auto kernel, typename... A>
cudaError_t start(dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem((const void*)kernel, kMostSmem, allowed);
  if (e != cudaSuccess) return e;
  kernel<<<grid, block, smem, st>>>(args...);
  return cudaGetLastError();
}

template <typename S, typename B, bool ALIGNED, int NG>
cudaError_t forward(const ResidualParams& p, cudaStream_t st) {
  const int nt = team_threads(p.H, NG), rows = nt == 32 ? kTeamRows : 1, sms = device_sm_count();
  const dim3 block(nt, rows);
  const size_t beside = !ALIGNED && p.drop.below ? (size_t)rows * ((p.H + 14) / 8 + 1) : 0;
  const size_t stage = (size_t)rows * nt * NG * (vectors8<S, ALIGNED>() + vectors8<B, ALIGNED>()) * 16;
  const int ctas = ctas_forward(nt * rows, NG), grid = (p.T + rows - 1) / rows;
  // (a team's only row needs no stage; rows so long that fewer CTAs would hold two are better off with all of them:
  // 8,192 rows of 7,168 f32 of both kinds, 161 us, ahead on half the CTAs 272)
  const int stages = grid > ctas * sms ? stages_ahead(kAheadBytes / ctas, stage, beside) : 0;
  auto run = [&](auto parts) {
    constexpr int kParts = decltype(parts)::value;
    if (stages == 0)
      return start<residual_forward_kernel<S, B, ALIGNED, NG, false, kParts>>(dim3(grid), block, beside, st, p, 0);
    return start<residual_forward_kernel<S, B, ALIGNED, NG, true, kParts>>(dim3(ctas * sms), block, stages * stage + beside,
                 st, p, stages);
  };
  if constexpr (NG <= 2) {
    if (p.y) {
      const int parts = (p.n ? kNext : 0) | (p.w_out ? kOut : 0) | (p.drop.below ? kDrop : 0);
      switch (parts) {
        case kNext: return run(std::integral_constant<int, kNext>());
        case kOut: return run(std::integral_constant<int, kOut>());
        case kNext | kOut: return run(std::integral_constant<int, kNext | kOut>());
        case kNext | kDrop: return run(std::integral_constant<int, kNext | kDrop>());
        case kOut | kDrop: return run(std::integral_constant<int, kOut | kDrop>());
        case kNext | kOut | kDrop: return run(std::integral_constant<int, kNext | kOut | kDrop>());
      }
    }
  }
  return run(std::integral_constant<int, kAnything>());
}

template <typename S, typename B, bool ALIGNED, int NG>
cudaError_t backward(const ResidualParams& p, int* launches, cudaStream_t st) {
  const int nt = team_threads(p.H, NG), rows = nt == 32 ? kTeamRows : 1;
  const bool bytes = !ALIGNED && p.drop.below;
  const int most = ctas_backward(nt * rows, NG);
  // as many CTAs an SM as have room for two rows ahead at least, or all of them with none
  BackwardPlan plan;
  size_t beside = 0, stage = 0;
  int stages = 0;
  for (int ctas = most; ctas >= 0 && !stages; --ctas) {
    plan = backward_plan(p.T, p.G, device_sm_count() * (ctas ? ctas : most) * rows, rows);
    beside = rows * backward_beside(p.H, bytes, plan.own, rows > 1);
    stage = (size_t)rows * nt * NG * 16 * (2 * vectors8<S, ALIGNED>() + (plan.own ? 3 : 2) * vectors8<B, ALIGNED>());
    if (ctas) stages = stages_ahead(kAheadBytesBackward / ctas, stage, beside);
    // (two rows that need all of it: 8,192 of 4,099 f32 of both kinds 426 us, with none ahead 517; where three fit, a fourth
    // for which L1 is given up costs: 8,192 of 7,168 bf16, dropout, 186 and 210)
    if (ctas == 1 && !stages) stages = stages_ahead(kMostSmem, stage, beside);
  }
  const dim3 grid(plan.ctas), block(nt, rows);
  auto run = [&](auto parts) {
    constexpr int kParts = decltype(parts)::value;
    return start<residual_backward_kernel<S, B, ALIGNED, NG, true, kParts>>(grid, block, stages * stage + beside, st, p, plan,
                 stages);
  };
  cudaError_t e = cudaErrorInvalidValue;
  const int parts = stages && NG <= 2 && p.dxo && p.dx && p.dy && !p.dn == !p.dw_next
                        ? (p.dn ? kNext : 0) | (p.w_out ? kOut : 0) | (p.drop.below ? kDrop : 0)
                        : kAnything;
  if constexpr (NG <= 2) {
    switch (parts) {
      case kNext: e = run(std::integral_constant<int, kNext>()); break;
      case kOut: e = run(std::integral_constant<int, kOut>()); break;
      case kNext | kOut: e = run(std::integral_constant<int, kNext | kOut>()); break;
      case kNext | kDrop: e = run(std::integral_constant<int, kNext | kDrop>()); break;
      case kOut | kDrop: e = run(std::integral_constant<int, kOut | kDrop>()); break;
      case kNext | kOut | kDrop: e = run(std::integral_constant<int, kNext | kOut | kDrop>()); break;
      default: break;
    }
  }
  if (NG > 2 || parts <= 0 || parts == kDrop) {
    e = stages ? run(std::integral_constant<int, kAnything>())
               : start<residual_backward_kernel<S, B, ALIGNED, NG, false, kAnything>>(grid, block, beside, st, p, plan, 0);
  }
  *launches = 1;
  const bool dgate = p.dgate && !plan.own;
  if (e != cudaSuccess || (!p.dw_next && !p.dw_out && !dgate)) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((p.H + 31) / 32, dgate ? 2 + plan.groups : 2);
  cfg.blockDim = dim3(32, kJoinRows);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  ++*launches;
  return cudaLaunchKernelEx(&cfg, residual_join_kernel<B>, p, plan);
}

// The instances, each in a file of its own.
template <typename S, typename B, bool ALIGNED>
cudaError_t forward_rows(const ResidualParams& p, cudaStream_t st) {
  switch (groups_forward(p.H)) {
    case 1: return forward<S, B, ALIGNED, 1>(p, st);
    case 2: return forward<S, B, ALIGNED, 2>(p, st);
    default: return forward<S, B, ALIGNED, 4>(p, st);
  }
}
template <typename S, typename B, bool ALIGNED>
cudaError_t backward_rows(const ResidualParams& p, int* launches, cudaStream_t st) {
  switch (groups_backward(p.H, ALIGNED)) {
    case 1: return backward<S, B, ALIGNED, 1>(p, launches, st);
    case 2: return backward<S, B, ALIGNED, 2>(p, launches, st);
    default: return backward<S, B, ALIGNED, 4>(p, launches, st);
  }
}

}  // namespace residual
}  // namespace mok

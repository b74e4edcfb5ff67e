// The join of a block with its residual stream, forward and backward.
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
#include <algorithm>

#include "residual.cuh"

namespace mok {

namespace {

// ------------------------------------------------------------------ rows in registers
// A row belongs to a team of NT threads (a warp, or a whole CTA), 8 NG
// elements each.  VEC: thread t holds the eight elements from (g NT + t) 8,
// loaded as vectors; otherwise the elements (8 g + e) NT + t, one by one, so
// that neighbouring threads read neighbouring elements at any alignment.
template <bool VEC>
__device__ __forceinline__ int column(int g, int e, int t, int nt) {
  return VEC ? (g * nt + t) * 8 + e : (g * 8 + e) * nt + t;
}

template <typename E>
__device__ __forceinline__ E from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int g, int t, int nt, int H, float (&v)[8]) {
  if constexpr (VEC) {
    const int c = column<true>(g, 0, t, nt);
    unpack8(c < H ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<false>(g, e, t, nt);
      v[e] = c < H ? __bfloat162float(row[c]) : 0.0f;
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void load8(const float* row, int g, int t, int nt, int H, float (&v)[8]) {
  if constexpr (VEC) {
    const int c = column<true>(g, 0, t, nt);
    float4 a = make_float4(0, 0, 0, 0), b = a;
    if (c < H) a = reinterpret_cast<const float4*>(row + c)[0], b = reinterpret_cast<const float4*>(row + c)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<false>(g, e, t, nt);
      v[e] = c < H ? row[c] : 0.0f;
    }
  }
}

template <bool VEC, typename E>
__device__ __forceinline__ void store8(E* row, int g, int t, int nt, int H, const float (&v)[8]) {
  if constexpr (VEC) {
    const int c = column<true>(g, 0, t, nt);
    if (c >= H) return;
    if constexpr (sizeof(E) == 2) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(row + c) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      reinterpret_cast<float4*>(row + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(row + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<false>(g, e, t, nt);
      if (c < H) row[c] = from_f32<E>(v[e]);
    }
  }
}

// ------------------------------------------------------------------ teams
// A team of 32 threads is one of the CTA's warps; a larger one is the CTA.
__device__ __forceinline__ void team_sync(int nt) {
  if (nt > 32) __syncthreads();
  else __syncwarp();
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// N sums over the team, in a fixed order; `slots` holds N * 32 floats of shared memory
// that no one else writes between two of the team's barriers.
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int t, int nt, float* slots) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (nt == 32) return;
  __syncthreads();  // (the slots' last readers are done)
  if ((t & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) slots[i * 32 + (t >> 5)] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum((t & 31) < (nt >> 5) ? slots[i * 32 + (t & 31)] : 0.0f);
}

// Eight elements' keep bits.  VEC: the row's elements from a multiple of eight
// are one of the generator's blocks.  Otherwise a block may straddle rows and
// threads: the team makes the row's blocks together, a byte each, in `bytes`
// (shared, (H + 14) / 8 + 1 of them), and every thread picks its bits.
__device__ __forceinline__ void keep_bytes(const DropParams& d, uint64_t call, uint64_t first, int H, int t, int nt,
                                           uint8_t* bytes) {
  const uint64_t b0 = first >> 3;
  const int n = (int)(((first + H - 1) >> 3) - b0) + 1;
  team_sync(nt);
  for (int i = t; i < n; i += nt) bytes[i] = (uint8_t)drop_keep8(d, b0 + i, call);
  team_sync(nt);
}

template <bool VEC>
__device__ __forceinline__ uint32_t keep8(const DropParams& d, uint64_t call, uint64_t first, int g, int t, int nt, int H,
                                          const uint8_t* bytes) {
  if constexpr (VEC) return drop_keep8(d, (first + column<true>(g, 0, t, nt)) >> 3, call);
  uint32_t keep = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = column<false>(g, e, t, nt);
    const uint32_t at = (uint32_t)(first & 7) + c;
    if (c < H) keep |= ((bytes[at >> 3] >> (at & 7)) & 1u) << e;
  }
  return keep;
}

// (a dropped element is 0 whatever it was)
__device__ __forceinline__ void drop8(float (&v)[8], uint32_t keep, float scale) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (keep >> e) & 1u ? v[e] * scale : 0.0f;
}

template <bool VEC, typename E>
__device__ __forceinline__ void weights8(const void* w, int g, int t, int nt, int H, float (&v)[8]) {
  load8<VEC>(static_cast<const E*>(w), g, t, nt, H, v);
}

// ------------------------------------------------------------------ forward
constexpr int kTeamRows = 8;  // rows, a warp each, in a CTA where a warp holds a row

template <typename S, typename B, bool VEC, int NG>
__global__ void __launch_bounds__(1024) residual_forward_kernel(const ResidualParams p) {
  extern __shared__ uint8_t mask[];
  __shared__ float slots[32];
  const int t = threadIdx.x, nt = blockDim.x, H = p.H;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.T) return;  // (a whole team: a warp of its own, or the whole CTA)
  const float rH = 1.0f / (float)H;
  float x[NG][8];
  const S* xr = static_cast<const S*>(p.x) + row * p.ldx;
#pragma unroll
  for (int g = 0; g < NG; ++g) load8<VEC>(xr, g, t, nt, H, x[g]);
  if (p.y) {
    float z[NG][8];
    const B* yr = static_cast<const B*>(p.y) + row * p.ldy;
#pragma unroll
    for (int g = 0; g < NG; ++g) load8<VEC>(yr, g, t, nt, H, z[g]);
    float ry = 1.0f;
    if (p.w_out) {
      float s[1] = {0.0f};
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] = fmaf(z[g][e], z[g][e], s[0]);
      team_sum(s, t, nt, slots);
      ry = 1.0f / sqrtf(fmaf(s[0], rH, p.eps));
    }
    const uint64_t first = (uint64_t)row * (uint64_t)H;
    uint8_t* bytes = mask + threadIdx.y * ((H + 14) / 8 + 1);
    uint64_t call = 0;
    if (p.drop.below) {
      call = drop_call(p.drop);
      if (!VEC) keep_bytes(p.drop, call, first, H, t, nt, bytes);
    }
    const B* gr = p.G ? static_cast<const B*>(p.gate) + (long)(row / p.rows_per_gate) * H : nullptr;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float w[8];
      if (p.w_out) {
        weights8<VEC, B>(p.w_out, g, t, nt, H, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[g][e] *= ry * w[e];
      }
      if (p.drop.below) drop8(z[g], keep8<VEC>(p.drop, call, first, g, t, nt, H, bytes), p.drop.scale);
      if (gr) {
        load8<VEC>(gr, g, t, nt, H, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[g][e] = fmaf(p.scale * w[e], z[g][e], x[g][e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[g][e] = fmaf(p.scale, z[g][e], x[g][e]);
      }
    }
    S* xo = static_cast<S*>(p.xo) + row * p.ldxo;
#pragma unroll
    for (int g = 0; g < NG; ++g) store8<VEC>(xo, g, t, nt, H, x[g]);
  }
  if (!p.n) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] = fmaf(x[g][e], x[g][e], s[0]);
  team_sum(s, t, nt, slots);
  const float r = 1.0f / sqrtf(fmaf(s[0], rH, p.eps));
  B* n = static_cast<B*>(p.n) + row * p.ldn;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    float w[8];
    weights8<VEC, B>(p.w_next, g, t, nt, H, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= x[g][e] * r;
    store8<VEC>(n, g, t, nt, H, w);
  }
}

// ------------------------------------------------------------------ backward
// The rows are cut into units, no unit across two gate rows' rows: G * split
// of them, or as many as workers where there is no gate.  A worker (a team)
// takes whole units and sums the columns of dw_next and dw_out over all of its
// rows, of dgate over a unit; the sums of workers and units are then joined in
// a fixed order by a second kernel.
struct BackwardPlan {
  int workers;   // teams
  int groups;    // rows of the gate, 1 without
  int split;     // units per group
};

template <typename S, typename B, bool VEC, int NG>
__global__ void __launch_bounds__(1024) residual_backward_kernel(const ResidualParams p, const BackwardPlan plan) {
  extern __shared__ uint8_t mask[];
  __shared__ float slots[3 * 32];
  const int t = threadIdx.x, nt = blockDim.x, H = p.H;
  const int worker = blockIdx.x * blockDim.y + threadIdx.y;
  if (worker >= plan.workers) return;  // (whole teams)
  const float rH = 1.0f / (float)H;
  const bool has_y = p.y != nullptr && (p.w_out || p.G);  // y's values matter
  uint8_t* bytes = mask + threadIdx.y * ((H + 14) / 8 + 1);
  const uint64_t call = p.drop.below ? drop_call(p.drop) : 0;
  const long rows_per_group = p.T / plan.groups;
  float sum_next[NG][8], sum_out[NG][8], sum_gate[NG][8];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum_next[g][e] = sum_out[g][e] = 0.0f;

  for (int unit = worker; unit < plan.groups * plan.split; unit += plan.workers) {
    const int group = unit / plan.split, part = unit % plan.split;
    const long row0 = group * rows_per_group + rows_per_group * part / plan.split;
    const long row1 = group * rows_per_group + rows_per_group * (part + 1) / plan.split;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum_gate[g][e] = 0.0f;
    const B* gr = p.G ? static_cast<const B*>(p.gate) + (long)group * H : nullptr;
    for (long row = row0; row < row1; ++row) {
      const uint64_t first = (uint64_t)row * (uint64_t)H;
      // dx in d, y in y
      float d[NG][8], y[NG][8];
      float s[3] = {0.0f, 0.0f, 0.0f};  // of y^2, x'^2, t x'
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (p.dxo) {
          load8<VEC>(static_cast<const S*>(p.dxo) + row * p.lddxo, g, t, nt, H, d[g]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[g][e] = 0.0f;
        }
        if (has_y) {
          load8<VEC>(static_cast<const B*>(p.y) + row * p.ldy, g, t, nt, H, y[g]);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] = fmaf(y[g][e], y[g][e], s[0]);
        }
      }
      if (p.dn) {
        float x[NG][8], dn[NG][8];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float w[8];
          load8<VEC>(static_cast<const S*>(p.x) + row * p.ldx, g, t, nt, H, x[g]);
          load8<VEC>(static_cast<const B*>(p.dn) + row * p.lddn, g, t, nt, H, dn[g]);
          weights8<VEC, B>(p.w_next, g, t, nt, H, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s[1] = fmaf(x[g][e], x[g][e], s[1]);
            s[2] = fmaf(dn[g][e] * w[e], x[g][e], s[2]);
          }
        }
        team_sum(s, t, nt, slots);
        const float r = 1.0f / sqrtf(fmaf(s[1], rH, p.eps));
        const float m = s[2] * rH * r * r;  // mean(t xh) r / r
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float w[8];
          weights8<VEC, B>(p.w_next, g, t, nt, H, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            sum_next[g][e] = fmaf(dn[g][e], x[g][e] * r, sum_next[g][e]);
            d[g][e] = fmaf(r, fmaf(dn[g][e], w[e], -m * x[g][e]), d[g][e]);
          }
        }
      } else if (p.w_out) {
        team_sum(s, t, nt, slots);
      }
      if (p.dx) {
#pragma unroll
        for (int g = 0; g < NG; ++g) store8<VEC>(static_cast<S*>(p.dx) + row * p.lddx, g, t, nt, H, d[g]);
      }
      if (!p.dy) continue;
      // the branch: d becomes dz
      const float ry = p.w_out ? 1.0f / sqrtf(fmaf(s[0], rH, p.eps)) : 1.0f;
      if (!VEC && p.drop.below) keep_bytes(p.drop, call, first, H, t, nt, bytes);
      float q[1] = {0.0f};  // of t' y
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float w[8], v[8];
        if (p.w_out) weights8<VEC, B>(p.w_out, g, t, nt, H, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[g][e] *= p.scale;
        uint32_t keep = 0xffu;
        if (p.drop.below) {
          keep = keep8<VEC>(p.drop, call, first, g, t, nt, H, bytes);
          drop8(d[g], keep, p.drop.scale);
        }
        if (gr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // (a dropped y may be anything, an infinity too)
            const float z = !((keep >> e) & 1u) ? 0.0f : p.w_out ? y[g][e] * (ry * w[e]) : y[g][e];
            sum_gate[g][e] = fmaf(d[g][e], z, sum_gate[g][e]);
          }
          load8<VEC>(gr, g, t, nt, H, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) d[g][e] *= v[e];
        }
        if (p.w_out) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            sum_out[g][e] = fmaf(d[g][e], y[g][e] * ry, sum_out[g][e]);
            d[g][e] *= w[e];
            q[0] = fmaf(d[g][e], y[g][e], q[0]);
          }
        }
      }
      if (p.w_out) {
        team_sum(q, t, nt, slots);
        const float m = q[0] * rH * ry * ry;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int e = 0; e < 8; ++e) d[g][e] = ry * fmaf(-m, y[g][e], d[g][e]);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) store8<VEC>(static_cast<B*>(p.dy) + row * p.lddy, g, t, nt, H, d[g]);
    }
    if (p.G) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (plan.split == 1)
          store8<VEC>(static_cast<B*>(p.dgate) + (long)group * H, g, t, nt, H, sum_gate[g]);
        else
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int c = column<VEC>(g, e, t, nt);
            if (c < H) p.part[(2l * plan.workers + unit) * H + c] = sum_gate[g][e];
          }
      }
    }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<VEC>(g, e, t, nt);
      if (c < H) {
        if (p.dw_next) p.part[(long)worker * H + c] = sum_next[g][e];
        if (p.dw_out) p.part[((long)plan.workers + worker) * H + c] = sum_out[g][e];
      }
    }
}

// Joins the column sums: 32 columns a CTA, 16 threads a column, each over
// every 16th part and then in order.
constexpr int kJoinRows = 16;
template <typename B>
__global__ void __launch_bounds__(32 * kJoinRows) residual_join_kernel(const ResidualParams p, const BackwardPlan plan) {
  __shared__ float sums[kJoinRows][33];
  const int c = blockIdx.x * 32 + threadIdx.x, what = blockIdx.y;  // 0 dw_next, 1 dw_out, 2 + g dgate
  if ((what == 0 && !p.dw_next) || (what == 1 && !p.dw_out)) return;
  const int n = what < 2 ? plan.workers : plan.split;
  const float* part = p.part + (what < 2 ? (long)what * plan.workers : 2l * plan.workers + (long)(what - 2) * plan.split) * p.H;
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
  if (what == 0) p.dw_next[c] = s;
  else if (what == 1) p.dw_out[c] = s;
  else static_cast<B*>(p.dgate)[(long)(what - 2) * p.H + c] = from_f32<B>(s);
}

// ------------------------------------------------------------------ launches
template <typename E>
bool vectors(const void* ptr, long ld) {
  return !ptr || (reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && ld % (16 / (int)sizeof(E)) == 0);
}

// Whether every row of every tensor is made of whole 16-byte vectors.
template <typename S, typename B>
bool all_vectors(const ResidualParams& p) {
  return p.H % 8 == 0 && vectors<B>(p.w_out, 0) && vectors<B>(p.gate, 0) && vectors<B>(p.w_next, 0) &&
         vectors<S>(p.x, p.ldx) && vectors<B>(p.y, p.ldy) && vectors<S>(p.xo, p.ldxo) && vectors<B>(p.n, p.ldn) &&
         vectors<S>(p.dxo, p.lddxo) && vectors<B>(p.dn, p.lddn) && vectors<S>(p.dx, p.lddx) &&
         vectors<B>(p.dy, p.lddy) && vectors<B>(p.dgate, 0);
}

int groups_per_thread(int H) { return H <= 8192 ? 1 : 2; }
int team_threads(int H) {
  const int per = 8 * groups_per_thread(H);
  return ((H + per - 1) / per + 31) / 32 * 32;
}

BackwardPlan backward_plan(int T, int H, int G, int sms) {
  BackwardPlan b;
  const int nt = team_threads(H);
  // at most 2,048 threads an SM, and four rows at least for a worker, so that the
  // parts stay few beside the rows
  const int most = nt == 32 ? sms * 32 : sms * std::max(1, 1024 / nt);
  b.workers = std::max(1, std::min(most, (T + 3) / 4));
  b.groups = std::max(1, G);
  b.split = std::max(1, std::min(b.workers / b.groups, T / b.groups));
  return b;
}

template <typename S, typename B>
cudaError_t forward(const ResidualParams& p, cudaStream_t st) {
  const int nt = team_threads(p.H), rows = nt == 32 ? kTeamRows : 1;
  const dim3 grid((p.T + rows - 1) / rows), block(nt, rows);
  const bool vec = all_vectors<S, B>(p);
  const size_t smem = !vec && p.drop.below ? (size_t)rows * ((p.H + 14) / 8 + 1) : 0;
  const bool one = groups_per_thread(p.H) == 1;
  auto k = vec ? (one ? residual_forward_kernel<S, B, true, 1> : residual_forward_kernel<S, B, true, 2>)
               : (one ? residual_forward_kernel<S, B, false, 1> : residual_forward_kernel<S, B, false, 2>);
  k<<<grid, block, smem, st>>>(p);
  return cudaGetLastError();
}

template <typename S, typename B>
cudaError_t backward(const ResidualParams& p, int* launches, cudaStream_t st) {
  const BackwardPlan plan = backward_plan(p.T, p.H, p.G, device_sm_count());
  const int nt = team_threads(p.H), rows = nt == 32 ? kTeamRows : 1;
  const dim3 grid((plan.workers + rows - 1) / rows), block(nt, rows);
  const bool vec = all_vectors<S, B>(p);
  const size_t smem = !vec && p.drop.below ? (size_t)rows * ((p.H + 14) / 8 + 1) : 0;
  const bool one = groups_per_thread(p.H) == 1;
  auto k = vec ? (one ? residual_backward_kernel<S, B, true, 1> : residual_backward_kernel<S, B, true, 2>)
               : (one ? residual_backward_kernel<S, B, false, 1> : residual_backward_kernel<S, B, false, 2>);
  k<<<grid, block, smem, st>>>(p, plan);
  cudaError_t e = cudaGetLastError();
  *launches = 1;
  const int joins = p.G && plan.split > 1 ? 2 + plan.groups : 2;
  if (e != cudaSuccess || (joins == 2 && !p.dw_next && !p.dw_out)) return e;
  residual_join_kernel<B><<<dim3((p.H + 31) / 32, joins), dim3(32, kJoinRows), 0, st>>>(p, plan);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace

size_t residual_part_floats(int T, int H) {
  // (any gate: units are no more than workers where their sums are parts)
  return 3 * (size_t)backward_plan(T, H, 0, device_sm_count()).workers * H;
}

cudaError_t launch_residual_forward(mok_dtype stream, mok_dtype branch, const ResidualParams& p, int* launches,
                                    cudaStream_t st) {
  *launches = 1;
  if (stream == MOK_TYPE_BF16) return forward<__nv_bfloat16, __nv_bfloat16>(p, st);
  return branch == MOK_TYPE_BF16 ? forward<float, __nv_bfloat16>(p, st) : forward<float, float>(p, st);
}

cudaError_t launch_residual_backward(mok_dtype stream, mok_dtype branch, const ResidualParams& p, int* launches,
                                     cudaStream_t st) {
  if (stream == MOK_TYPE_BF16) return backward<__nv_bfloat16, __nv_bfloat16>(p, launches, st);
  return branch == MOK_TYPE_BF16 ? backward<float, __nv_bfloat16>(p, launches, st)
                                 : backward<float, float>(p, launches, st);
}

}  // namespace mok

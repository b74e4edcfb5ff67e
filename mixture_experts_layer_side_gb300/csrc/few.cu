// The layer for a few tokens (T <= MOK_FEW_MAX_TOKENS): routed SwiGLU experts
// and combine, with or without the router, in one launch.
//
//   h = x_t W1_e,  u = x_t W3_e,  a = silu(h) * u,  y = a W2_e,  e = idx[t, j]
//   out_t = sum_j s[t, j] y_(t, j)
//
// What bounds it is the read of the chosen experts' weights: a row or two of
// tokens per expert is a few operations for each weight.  The design streams
// weights without a pause:
//
//  * The weight is the MMA's A operand (128 output columns by K, straight
//    from its row-major layout) and the tokens its B operand (N = 16 to 64 of
//    them), so the tensor core takes weights from shared memory as TMA brings
//    them and no thread touches one.
//  * One CTA per SM.  A "unit" is up to unit_rows rows of one expert; a tile
//    is 2 x 128 output columns of a unit (first GEMM: 128 of h and the same
//    of u; second: 256 of y); a block is 64 (MXFP8: 128) of a tile's K.  All
//    blocks of a GEMM, tiles in order, are cut into equal runs whatever the
//    number of experts: no SM waits for a last wave.  A tile that a cut splits
//    leaves f32 sums in the workspace; the last of its CTAs to arrive (first
//    GEMM) or the combine (second) adds them in the order of K.
//  * A run belongs to a group of CTAs that take neighbouring column tiles of
//    the same K, so that the 128 or 256 bytes that one CTA reads of a weight
//    row lie beside what its neighbours read at the same time.
//  * The second GEMM needs all of a.  The units are split in two halves, A
//    and B, and the order is a(A), a(B), y(A), y(B): while the last sums of
//    one half are joined, the weights of the next part stream in.
//  * Every CTA sorts the routing by expert for itself (at most 4,096 ids), so
//    no launch or barrier stands between the routing and the first weight.
//
// Measured, of the rate of a copy (6.69 TB/s), on the weights of the experts
// chosen: H 7168, I 2048, top-8: bf16 24 tokens 426 us (all of it), 4 tokens
// 234 us (97%), 1 token with the router 120 us (88%); MXFP8 8 tokens 393 us (all
// of it), 128 tokens 446 us (81%, the joins of experts with many rows).  H
// 2048, I 768, top-8 of 64: bf16 1 token 29 us (39%: the start, the join
// between the GEMMs and the combine stand beside 11 us of weights), 128 tokens
// 114 us (61%: the joins of experts with many rows), MXFP8 84 (43%), with the
// router 92 (50%).
//
// Arrivals are counted in the workspace and every CTA has to be resident: the
// launch is cooperative.  All waits are bounded (MOK_ERR_TIMEOUT).  The
// counters are zero again when a call ends.
#include <string.h>

#include "few.cuh"
#include "mx.cuh"
#include "tc.cuh"
#include "topk.cuh"

namespace mok {

namespace {

// Stages of 32 KB of weights in flight on an SM.  bf16: four; a fifth only
// delays the loads that others wait for (4 tokens, H 7168, I 2048: 233 us;
// three 239, five 237, six 247).  MXFP8 needs six (8 tokens: 395 us; four 402,
// three 420), but four where a CTA has few blocks of the first GEMM (128
// tokens, H 2048, I 768, E 64: 83.5 us; three 84.3, five 85.4, as many as fit 85.5).
constexpr int kStages = 4;
constexpr int kMaxFewStages = 6;
constexpr int kLongRun = 64;
constexpr int kATile = 128 * 128;      // one A operand: 128 output columns x 128 bytes of K
constexpr int kSfBytes = 1024 + 1024 + 512;  // MXFP8, per stage: raw and tiled A scales (two tiles), B scales
constexpr int kProducers = 64;         // threads that bring the tokens' operand
constexpr int kEpilogue = 256;         // two warps for each quarter of the accumulator's rows
constexpr int kLogitWarps = 8;
constexpr int kLogitTokens = 8;        // tokens side by side in the router's logits; a single one has a form of
                                       // its own (H 2048, I 768: 33.7 us, as one of eight 34.5)

// header words
constexpr int kWordPrepared = kHdrCounters;      // CTAs done with the logits' parts and x's quantisation
constexpr int kWordRouted = kHdrCounters + 1;    // tokens routed
constexpr int kWordHidden = kHdrCounters + 2;    // [2] tiles of a finished, each half
constexpr int kWordSummed = kHdrCounters + 4;    // CTAs whose sums of y are stored
constexpr int kWordLeft = kHdrCounters + 5;      // CTAs that ended
// Two halves only where a half is long beside the joining it hides, in blocks a
// CTA of the first GEMM: 128 tokens, H 2048, I 768, E 64, bf16 (77 blocks) 114
// us, in one 123; 1 token (10 blocks) 37 us in halves, in one 30.
constexpr int kHalvesFrom = 32;
// Blocks: a shorter run would not fill the stages (1 token, H 2048, I 768: 29.9
// us; runs of 3 or more 30.3, of 12 or more 31.8).
constexpr int kMinRun = 6;

// The routing sorted by expert, in shared memory.
struct Schedule {
  uint16_t* offset;   // [E] first sorted row of each expert
  uint16_t* unit0;    // [E] its first unit
  uint16_t* perm;     // [T*k] sorted row -> flat index
  uint16_t* token;    // [T*k] sorted row -> token
  uint16_t* unit_of;  // [T*k] flat index -> unit (kNoUnit: an id out of range)
  uint16_t* unit_e;   // [max_units] expert, first sorted row and rows of each unit
  uint16_t* unit_r;
  uint8_t* row_of;    // [T*k] flat index -> row of its unit
  uint8_t* unit_n;
};
constexpr int kNoUnit = 0xFFFF;

__host__ __device__ constexpr size_t schedule_bytes(int E, int R, int units) {
  return (size_t)E * 4 + (size_t)R * 7 + (size_t)units * 5 + 16;
}

// (a call, so that its instructions are fetched once)
__device__ __noinline__ int quotient(int a, int b) { return (int)((unsigned)a / (unsigned)b); }

// One GEMM of one half of the units, its blocks cut into runs whose lengths
// differ by one at most.
struct Cut {
  int group, group_shift;  // CTAs side by side on neighbouring column tiles
  int supers, tiles;  // groups of column tiles, and column tiles, of a unit
  int kb;             // blocks along K
  int unit0, units;
  int blocks;         // of one CTA of a group
  int runs, each, rest;  // blocks = runs * each + rest
  __device__ bool takes(int c) const { return c < runs * group; }
  __device__ int begin(int run) const { return each * run + quotient(rest * run, runs); }
  // the run that holds block b
  __device__ int owner(int b) const {
    int o = (int)((float)b * (float)runs / (float)blocks);
    o = min(o, runs - 1);
    while (begin(o) > b) --o;
    while (begin(o + 1) <= b) ++o;
    return o;
  }
};

__device__ __forceinline__ Cut make_cut(const FewShape& f, int unit0, int units, int ctas) {
  Cut c;
  c.group = 1 << f.group_shift;
  c.group_shift = f.group_shift;
  c.supers = f.supers;
  c.tiles = f.supers << f.group_shift;
  c.kb = f.kb;
  c.unit0 = unit0;
  c.units = units;
  c.blocks = units * c.supers * c.kb;
  c.runs = 0;
  c.each = c.rest = 0;
  if (units) {
    c.runs = max(1, min(quotient(c.blocks + kMinRun - 1, kMinRun), ctas >> f.group_shift));
    c.each = quotient(c.blocks, c.runs);
    c.rest = c.blocks - c.each * c.runs;
  }
  return c;
}

// A run's share of one tile.
struct Seg {
  int unit, n;    // unit and column tile
  int k0, k1;     // blocks
  int super;      // index of the tile's group
};

// A CTA's run of a cut: its first share, and the blocks from there on.  (Made
// once per CTA; the roles step through it without a division.)
struct Run {
  Seg seg;
  int left;
};

__device__ __forceinline__ Run run_of(const Cut& c, int cta) {
  Run r;
  r.left = 0;
  if (!c.takes(cta)) return r;
  const int run = cta >> c.group_shift, b = c.begin(run);
  r.left = c.begin(run + 1) - b;
  Seg& s = r.seg;
  s.super = quotient(b, c.kb);
  s.k0 = b - s.super * c.kb;
  s.k1 = min(c.kb, s.k0 + r.left);
  const int u = quotient(s.super, c.supers);
  s.unit = c.unit0 + u;
  s.n = ((s.super - u * c.supers) << c.group_shift) + cta - (run << c.group_shift);
  return r;
}

// The next share.
__device__ __forceinline__ void step(Run& r, const Cut& c) {
  Seg& s = r.seg;
  r.left -= s.k1 - s.k0;
  ++s.super;
  s.n += c.group;
  if (s.n >= c.tiles) {
    s.n -= c.tiles;
    ++s.unit;
  }
  s.k0 = 0;
  s.k1 = min(c.kb, r.left);
}

// The runs that a tile is split over.
__device__ __forceinline__ void seg_runs(const Cut& c, int super, int& first, int& last) {
  const int b = super * c.kb;
  first = c.owner(b);
  last = c.owner(b + c.kb - 1);
}

struct Ctl {
  uint64_t full_a[kMaxFewStages], full_b[kMaxFewStages], scales[kMaxFewStages], empty[kMaxFewStages];
  uint64_t tfull[2], tempty[2], drained;
  uint32_t tmem;
  int abort, go;
  int failed;  // a wait of this CTA gave up
  int units;
  int last;
  int warp_sum[16];
  Cut cuts[4];  // in order: a of each half of the units, y of each half
  Run runs[4];  // this CTA's
};

__device__ __forceinline__ bool vote_all(int bar, int threads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "r"(bar), "r"(threads)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ int atom_add_acq_rel(int32_t* p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

__device__ __forceinline__ uint32_t* word(const FewParams& p, int i) { return reinterpret_cast<uint32_t*>(p.hdr + i); }

// ---------------------------------------------------------------- router
// This CTA's part of the logits: TOK tokens by h_rows rows of Wr.  A lane
// takes 8 neighbouring experts, as many lanes as a row needs (32 at most), the
// rest of the warp and the other warps other rows; the lanes' and the warps'
// sums are added in a fixed order.
template <int TOK>
__device__ __forceinline__ void router_logits(const FewParams& p, uint8_t* smem, int nthreads) {
  const int groups = (p.T + TOK - 1) / TOK;
  const int warps = kLogitWarps, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x / groups, t0 = (blockIdx.x % groups) * TOK;
  if (part >= p.h_parts) return;
  const int nt = min(TOK, p.T - t0);
  const int h0 = part * p.h_rows, rows = min(p.h_rows, p.H - h0);
  float* xs = reinterpret_cast<float*>(smem);                 // [h_rows][TOK]
  float* red = xs + (size_t)p.h_rows * TOK;                   // [warps][TOK][256]
  // (h0 and rows are multiples of 8)
  for (int i = threadIdx.x; i < rows / 8 * TOK; i += nthreads) {
    const int t = i % TOK, h = i / TOK * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t < nt) v = __ldg(reinterpret_cast<const uint4*>(p.x + (long)(t0 + t) * p.H + h0 + h));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      xs[(h + 2 * m) * TOK + t] = __uint_as_float(w[m] << 16);
      xs[(h + 2 * m + 1) * TOK + t] = __uint_as_float(w[m] & 0xffff0000u);
    }
  }
  __syncthreads();
  int across = 1;  // lanes along a row
  while (across < 32 && across * 8 < p.E) across <<= 1;
  const int down = 32 / across;
  const bool vec = p.E % 8 == 0 && (reinterpret_cast<uintptr_t>(p.Wr) & 15) == 0;
  for (int e0 = 0; e0 < p.E; e0 += 256) {
    const int e = e0 + (lane & (across - 1)) * 8;
    float acc[TOK][8];
#pragma unroll
    for (int t = 0; t < TOK; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[t][i] = 0.0f;
    // eight rows a warp in flight
    constexpr int kAhead = 8;
    for (int hb = warp * down + lane / across; warp < warps && hb - lane / across < rows; hb += warps * down * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int h = hb + i * warps * down;
        const __nv_bfloat16* wr = p.Wr + (long)(h0 + h) * p.E + e;
        v[i] = make_uint4(0, 0, 0, 0);
        if (h < rows && e < p.E) {
          if (vec) {
            v[i] = __ldg(reinterpret_cast<const uint4*>(wr));
          } else {
            uint32_t w[4];
            for (int m = 0; m < 4; ++m) {
              const uint32_t lo = e + 2 * m < p.E ? __bfloat16_as_ushort(wr[2 * m]) : 0;
              const uint32_t hi = e + 2 * m + 1 < p.E ? __bfloat16_as_ushort(wr[2 * m + 1]) : 0;
              w[m] = lo | hi << 16;
            }
            v[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int h = hb + i * warps * down;
        if (h >= rows) break;  // (an infinite x times 0 is NaN)
        const uint32_t vv[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
          const float x = xs[h * TOK + t];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            acc[t][2 * m] = fmaf(x, __uint_as_float(vv[m] << 16), acc[t][2 * m]);
            acc[t][2 * m + 1] = fmaf(x, __uint_as_float(vv[m] & 0xffff0000u), acc[t][2 * m + 1]);
          }
        }
      }
    }
    for (int o = across; o < 32; o <<= 1)
#pragma unroll
      for (int t = 0; t < TOK; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[t][i] += __shfl_xor_sync(0xffffffffu, acc[t][i], o);
    if (lane < across && warp < warps)
#pragma unroll
      for (int t = 0; t < TOK; ++t) {
        float4* r = reinterpret_cast<float4*>(red + (warp * TOK + t) * 256 + lane * 8);
        r[0] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
        r[1] = make_float4(acc[t][4], acc[t][5], acc[t][6], acc[t][7]);
      }
    __syncthreads();
    const int ne = min(256, p.E - e0);
    for (int i = threadIdx.x; i < nt * 256; i += nthreads) {
      const int t = i >> 8, c = i & 255;
      if (c >= ne) continue;
      float s = 0.0f;
      for (int w = 0; w < warps; ++w) s += red[(w * TOK + t) * 256 + c];
      p.logits[((long)part * p.T + t0 + t) * p.E + e0 + c] = s;
    }
    __syncthreads();
  }
}

// Selection and scores of one token from the parts of its logits: groups of
// threads take shares of the parts, so that the loads are in flight together.
// (smem: first the bias, which the caller brings while the parts are awaited.)
__device__ void router_select(const FewParams& p, int t, float* smem, int nthreads) {
  float* bias = smem;                 // [E]
  float* row = bias + p.E;            // [E]
  float* red = row + p.E;             // [shares][E]
  const int w = p.E % 4 == 0 ? 4 : 1; // experts a load brings
  const int cols = (p.E + w - 1) / w;
  const int shares = max(1, min(16, nthreads / cols));
  const int per = (p.h_parts + shares - 1) / shares;
  const int share = threadIdx.x / cols, c0 = threadIdx.x - share * cols;
  if (share < shares)
    for (int c = c0; c < cols; c += shares > 1 ? cols : nthreads) {
      const int i0 = share * per, i1 = min(p.h_parts, i0 + per);
      const float* from = p.logits + (long)t * p.E + c * w;
      const long step = (long)p.T * p.E;
      float* to = red + share * p.E + c * w;
      if (w == 4) {
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int i = i0; i < i1; ++i) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(from + i * step));
          s.x += v.x;
          s.y += v.y;
          s.z += v.z;
          s.w += v.w;
        }
        to[0] = s.x;
        to[1] = s.y;
        to[2] = s.z;
        to[3] = s.w;
      } else {
        float s = 0.0f;
#pragma unroll 8
        for (int i = i0; i < i1; ++i) s += __ldcg(from + i * step);
        to[0] = s;
      }
    }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += nthreads) {
    float s = red[e];
#pragma unroll 4
    for (int i = 1; i < shares; ++i) s += red[i * p.E + e];
    row[e] = s;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int e;
    float s;
    const float* b = p.bias ? bias : nullptr;
    if (p.E <= 256)
      topk_softmax_warp<8>(row, b, p.E, p.k, lane, e, s);
    else
      topk_softmax_warp<kMaxRouterExperts / 32>(row, b, p.E, p.k, lane, e, s);
    if (lane < p.k) {
      p.idx_out[(long)t * p.k + lane] = e;
      p.scores_out[(long)t * p.k + lane] = s;
    }
    __syncwarp();
    if (lane == 0) red_release_gpu_add(word(p, kWordRouted), 1u);
  }
  __syncthreads();
}

// MXFP8: x quantised along H, one thread per block of 32.
__device__ void quantize_x(const FewParams& p, int nthreads) {
  const int n = p.T * (p.H / 32);
  for (int b = blockIdx.x * nthreads + threadIdx.x; b < n; b += gridDim.x * nthreads) {
    const uint4* s = reinterpret_cast<const uint4*>(p.x + (long)b * 32);
    float v[32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = s[i];
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + 2 * j] = __uint_as_float(ww[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(ww[j] & 0xffff0000u);
      }
    }
    uint32_t codes[8];
    p.xsf[b] = mx_quant32(v, codes);
    uint4* d = reinterpret_cast<uint4*>(p.xq + (long)b * 32);
    d[0] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
    d[1] = make_uint4(codes[4], codes[5], codes[6], codes[7]);
  }
}

// ---------------------------------------------------------------- schedule
// At most 32 rows, by one warp: lane f's row goes after those of lower experts
// and of lower f.  False where an expert has more rows than a unit takes.  (1
// token, H 2048, I 768: 28 us, with the sort below 31.)
__device__ __forceinline__ bool build_few(const FewParams& p, const Schedule& s, Ctl* ctl, int id, int lane) {
  const int R = p.T * p.k;
  if (p.Wr) id = lane < R ? __ldcg(p.idx + lane) : -1;
  const bool in = lane < R && id >= 0 && id < p.E;
  const uint32_t valid = __ballot_sync(0xffffffffu, in);
  const uint32_t same = __match_any_sync(0xffffffffu, in ? id : -1);
  const int rows = __popc(same), ahead = __popc(same & ((1u << lane) - 1u));
  if (__any_sync(0xffffffffu, in && rows > p.unit_rows)) return false;
  const bool first = in && ahead == 0;
  const uint32_t firsts = __ballot_sync(0xffffffffu, first);
  int before = 0, unit = 0;
#pragma unroll 4
  for (int j = 0; j < 32; ++j) {
    const int e = __shfl_sync(0xffffffffu, id, j);
    const bool lower = e < id;
    before += lower && ((valid >> j) & 1u);
    unit += lower && ((firsts >> j) & 1u);
  }
  if (in) {
    s.perm[before + ahead] = (uint16_t)lane;
    s.token[before + ahead] = (uint16_t)(lane / p.k);
    s.row_of[lane] = (uint8_t)ahead;
  }
  if (lane < R) s.unit_of[lane] = (uint16_t)(in ? unit : kNoUnit);
  if (first) {
    s.unit_e[unit] = (uint16_t)id;
    s.unit_r[unit] = (uint16_t)before;
    s.unit_n[unit] = (uint8_t)rows;
  }
  if (lane == 0) ctl->units = __popc(firsts);
  if (blockIdx.x == 0 && lane < R && !in) atomicOr(p.hdr + kHdrError, MOK_ERRBIT_BAD_INDEX);
  __syncwarp();
  return true;
}

// Rows grouped by expert in ascending flat index, and cut into units: a
// counting sort whose warps own contiguous ranges of the flat indices, so
// that (warp, place) is their order.  `scratch`: of each flat index its expert
// and its place among the warp's rows of that expert, and a count per warp
// and expert.
__device__ void build_units(const FewParams& p, const Schedule& s, uint8_t* scratch, Ctl* ctl, int nthreads) {
  const int R = p.T * p.k, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_shift = max(5, 32 - __clz((R - 1) / (nthreads / 32)));  // flat indices a warp, a power of two
  const int per = 1 << per_shift, W = (R + per - 1) >> per_shift;       // warps that have some
  const int shift = __ffs(p.unit_rows) - 1;
  uint16_t* ids = reinterpret_cast<uint16_t*>(scratch);
  uint16_t* place = ids + R;
  uint32_t* hist = reinterpret_cast<uint32_t*>(scratch + (((size_t)R * 4 + 15) & ~15));  // [W][E]
  bool bad = false;
  for (int f0 = threadIdx.x; f0 < R; f0 += 4 * nthreads) {
    int e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = f0 + i * nthreads < R ? __ldcg(p.idx + f0 + i * nthreads) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int f = f0 + i * nthreads;
      if (f >= R) break;
      const bool in = e[i] >= 0 && e[i] < p.E;
      bad |= !in;
      ids[f] = (uint16_t)(in ? e[i] : kNoUnit);
    }
  }
  for (int i = threadIdx.x; i < W * p.E; i += nthreads) hist[i] = 0;
  if (bad && blockIdx.x == 0) atomicOr(p.hdr + kHdrError, MOK_ERRBIT_BAD_INDEX);
  __syncthreads();
  const int f0 = warp << per_shift, f1 = min(R, f0 + per);
  uint32_t* mine = hist + warp * p.E;
  for (int f = f0 + lane; f - lane < f1; f += 32) {
    const int e = f < f1 ? ids[f] : kNoUnit;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int ahead = __popc(same & ((1u << lane) - 1u));
    const uint32_t so_far = e != kNoUnit ? mine[e] : 0;
    __syncwarp();
    if (e != kNoUnit) {
      place[f] = (uint16_t)(so_far + ahead);
      if (ahead == 0) mine[e] = so_far + __popc(same);
    }
    __syncwarp();
  }
  __syncthreads();
  // thread i: experts [i * each, (i + 1) * each); rows and units scanned in one word
  const int each = (p.E + nthreads - 1) / nthreads;
  const int e0 = threadIdx.x * each, e1 = min(p.E, e0 + each);
  uint32_t sum = 0;
  for (int e = e0; e < e1; ++e) {
    uint32_t rows = 0;
#pragma unroll 4
    for (int w = 0; w < W; ++w) {
      const uint32_t v = hist[w * p.E + e];
      hist[w * p.E + e] = rows;
      rows += v;
    }
    s.offset[e] = (uint16_t)rows;  // the count, for now
    sum += rows | (((rows + p.unit_rows - 1) >> shift) << 16);
  }
  uint32_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) ctl->warp_sum[warp] = (int)incl;
  __syncthreads();
  uint32_t at = incl - sum;
  for (int w = 0; w < warp; ++w) at += (uint32_t)ctl->warp_sum[w];
  for (int e = e0; e < e1; ++e) {
    const int rows = s.offset[e], off = at & 0xFFFF, u0 = at >> 16;
    const int units = (rows + p.unit_rows - 1) >> shift;
    s.offset[e] = (uint16_t)off;
    s.unit0[e] = (uint16_t)u0;
    for (int i = 0; i < units; ++i) {
      s.unit_e[u0 + i] = (uint16_t)e;
      s.unit_r[u0 + i] = (uint16_t)(off + i * p.unit_rows);
      s.unit_n[u0 + i] = (uint8_t)min(p.unit_rows, rows - i * p.unit_rows);
    }
    at += (uint32_t)rows | ((uint32_t)units << 16);
  }
  if (threadIdx.x == nthreads - 1) ctl->units = (int)(at >> 16);
  __syncthreads();
#pragma unroll 2
  for (int f = threadIdx.x; f < R; f += nthreads) {
    const int e = ids[f];
    s.unit_of[f] = (uint16_t)kNoUnit;
    if (e == kNoUnit) continue;
    const int n = (int)hist[(f >> per_shift) * p.E + e] + place[f];  // among the expert's rows
    const int to = s.offset[e] + n;
    s.perm[to] = (uint16_t)f;
    s.token[to] = (uint16_t)(f / p.k);
    s.unit_of[f] = (uint16_t)(s.unit0[e] + (n >> shift));
    s.row_of[f] = (uint8_t)(n & (p.unit_rows - 1));
  }
  __syncthreads();
}

// ---------------------------------------------------------------- epilogue
// Four columns of each of two accumulators, this lane's row.
__device__ __forceinline__ void tmem_ld4x2(uint32_t a0, uint32_t a1, float (&v0)[4], float (&v1)[4]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a0));
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(a1));
  tmem_wait_ld();
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v0[i] = __uint_as_float(r[i]);
    v1[i] = __uint_as_float(r[4 + i]);
  }
}

__device__ __forceinline__ float silu_mul(float h, float u) { return h / (1.0f + __expf(-h)) * u; }

// a of 4 rows in column `col` (a lane's): bf16 and what its rounding left, or
// codes and a scale per 32 columns.  Two bf16 hold 16 bits of a, off by 2^-18 of
// it at most: y is off by 2.5e-6 of itself (H 7168, I 2048), where out is
// rounded to 2^-9, and a third part would take TMEM that 64 rows do not leave.
template <bool MX>
__device__ __forceinline__ void store_hidden(const FewParams& p, int row, int n, int col, int lane, const float (&h)[4],
                                             const float (&u)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = silu_mul(h[i], u[i]);
    const long at = (long)(row + i) * p.I + col;
    if constexpr (MX) {
      const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(a))));
      const int X = mx_block_exponent(amax);
      const uint8_t code = (uint8_t)mx_cvt_e4m3x2(a * mx_exp2_int(-X), 0.0f);
      if (i < n) {
        static_cast<uint8_t*>(p.a)[at] = code;
        if (lane == 0) p.asf[at / 32] = (uint8_t)(X + 127);
      }
    } else {
      __nv_bfloat16* hi = static_cast<__nv_bfloat16*>(p.a) + at;
      const float back = bf16_round(a);
      if (i < n) {
        hi[0] = __float2bfloat16(back);
        hi[(long)p.T * p.k * p.I] = __float2bfloat16(isinf(back) ? 0.0f : a - back);
      }
    }
  }
}

// a of four columns of a row, from the sums of its h and u.
template <bool MX>
__device__ __forceinline__ void store_hidden4(const FewParams& p, int row, int col, int lane, bool in, float4 h,
                                              float4 u) {
  const long at = (long)row * p.I + col;
  const float a[4] = {silu_mul(h.x, u.x), silu_mul(h.y, u.y), silu_mul(h.z, u.z), silu_mul(h.w, u.w)};
  if constexpr (MX) {
    // eight lanes hold a block
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(fabsf(a[i])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int X = mx_block_exponent(__uint_as_float(top));
    const float inv = mx_exp2_int(-X);
    const uint32_t codes =
        mx_cvt_e4m3x2(a[0] * inv, a[1] * inv) | (uint32_t)mx_cvt_e4m3x2(a[2] * inv, a[3] * inv) << 16;
    if (in) {
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.a) + at) = codes;
      if ((lane & 7) == 0) p.asf[at / 32] = (uint8_t)(X + 127);
    }
  } else {
    __nv_bfloat16* hi = static_cast<__nv_bfloat16*>(p.a) + at;
    float back[4], left[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      back[i] = bf16_round(a[i]);
      left[i] = isinf(back[i]) ? 0.0f : a[i] - back[i];
    }
    if (in) {
      *reinterpret_cast<uint2*>(hi) = make_uint2(pack_bf16x2(back[0], back[1]), pack_bf16x2(back[2], back[3]));
      *reinterpret_cast<uint2*>(hi + (long)p.T * p.k * p.I) =
          make_uint2(pack_bf16x2(left[0], left[1]), pack_bf16x2(left[2], left[3]));
    }
  }
}

// The parts of a tile of a that is split along K, added in the order of K (the
// tile ends the first run, and begins the others), and a of the sums.  A warp
// takes every eighth row, ROWS of them at a time, a lane four columns; the
// loads of PARTS parts of each are in flight together.
template <bool MX, int ROWS, int PARTS>
__device__ __forceinline__ void join_hidden(const FewParams& p, const Cut& cut, const Seg& s, int rank, int half,
                                            int first, int last, int r0, int n, int warp, int lane) {
  const int slot_floats = 2 * p.unit_rows * 128;
  const int col = s.n * 128 + lane * 4;
  const float* base = p.part + lane * 4;
#pragma unroll 1
  for (int row = warp; row < n; row += 8 * ROWS) {
    float4 h[ROWS], u[ROWS];
#pragma unroll
    for (int m = 0; m < ROWS; ++m) h[m] = u[m] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int o0 = first; o0 <= last; o0 += PARTS) {
      float4 vh[ROWS][PARTS], vu[ROWS][PARTS];
#pragma unroll
      for (int o = 0; o < PARTS; ++o) {
        const int slot = 4 * ((o0 + o) * cut.group + rank) + 2 * half + (o0 + o == first ? 1 : 0);
        const float* from = base + (long)slot * slot_floats + row * 128;
#pragma unroll
        for (int m = 0; m < ROWS; ++m) {
          vh[m][o] = vu[m][o] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (o0 + o <= last && row + 8 * m < n) {
            vh[m][o] = __ldcg(reinterpret_cast<const float4*>(from + m * 1024));
            vu[m][o] = __ldcg(reinterpret_cast<const float4*>(from + m * 1024 + p.unit_rows * 128));
          }
        }
      }
#pragma unroll
      for (int m = 0; m < ROWS; ++m)
#pragma unroll
        for (int o = 0; o < PARTS; ++o) {
          h[m].x += vh[m][o].x, h[m].y += vh[m][o].y, h[m].z += vh[m][o].z, h[m].w += vh[m][o].w;
          u[m].x += vu[m][o].x, u[m].y += vu[m][o].y, u[m].z += vu[m][o].z, u[m].w += vu[m][o].w;
        }
    }
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
      store_hidden4<MX>(p, r0 + row + 8 * m, col, lane, row + 8 * m < n, h[m], u[m]);
  }
}

// The runs of every tile of y, for the combine: first | last << 16,
// [units][supers] of each half in turn.
__device__ void list_runs(const Cut* cuts, uint32_t* table, int nthreads) {
  const int n0 = cuts[0].units * cuts[0].supers, n = n0 + cuts[1].units * cuts[1].supers;
  for (int i = threadIdx.x; i < n; i += nthreads) {
    const Cut& c = cuts[i >= n0];
    int first, last;
    seg_runs(c, i - (i >= n0 ? n0 : 0), first, last);
    table[i] = (uint32_t)first | (uint32_t)last << 16;
  }
}

// The combine: 4 columns of a token to LANES threads.  Each brings y of
// EACH experts at a time -- from y's buffer or, where its tile was split along
// K, as the sum of the parts -- all their loads in flight together; the
// lanes' values are added up in the order of j.
template <int LANES, int EACH>
__device__ __forceinline__ void combine(const FewParams& p, const Schedule& s, const Cut* cuts, const uint32_t* table,
                                        int nthreads) {
  static_assert(LANES == 1 || EACH == 1, "several lanes bring one expert each");
  const int vecs = p.H / 4;
  const int slot_floats = 2 * p.unit_rows * 128;
  const int sub = threadIdx.x & (LANES - 1);
  const int items = p.T * vecs, stride = gridDim.x * nthreads / LANES;
  const int group = cuts[0].group, supers = cuts[0].supers;
  const int ahead = (threadIdx.x & 31) / LANES;  // items of the warp before this one: its lanes stay together
#pragma unroll 1
  for (int i = (blockIdx.x * nthreads + threadIdx.x) / LANES; i - ahead < items; i += stride) {
    const bool in = i < items;
    const int t = in ? i / vecs : 0, col = (in ? i - t * vecs : 0) * 4;
    const int n = col >> 8, sup = n / group, rank = n - sup * group;
    const float* part_at = p.part + ((col >> 7) & 1) * p.unit_rows * 128 + (col & 127);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int j0 = 0; j0 < p.k; j0 += LANES * EACH) {
      const float4 *from[EACH], *next[EACH];
      int more[EACH];  // parts past the first; -1: nothing there
#pragma unroll
      for (int m = 0; m < EACH; ++m) {
        const int j = j0 + sub + m, f = t * p.k + j;
        const int unit = in && j < p.k ? s.unit_of[f] : kNoUnit;
        more[m] = -1;
        from[m] = next[m] = reinterpret_cast<const float4*>(p.y);
        if (unit != kNoUnit) {
          const int half = unit >= cuts[1].unit0;
          int first, last;
          if (table) {
            const uint32_t runs = table[unit * supers + sup];
            first = runs & 0xFFFF;
            last = runs >> 16;
          } else {
            seg_runs(cuts[half], (unit - cuts[half].unit0) * supers + sup, first, last);
          }
          more[m] = last - first;
          const float* at = part_at + s.row_of[f] * 128;
          from[m] = reinterpret_cast<const float4*>(
              more[m] ? at + (long)((first * group + rank) * 4 + half * 2 + 1) * slot_floats : p.y + (long)f * p.H + col);
          next[m] = reinterpret_cast<const float4*>(at + (long)(((first + 1) * group + rank) * 4 + half * 2) * slot_floats);
        }
      }
      float w[EACH];
      float4 y[EACH], z[EACH];
#pragma unroll
      for (int m = 0; m < EACH; ++m) {
        const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        w[m] = more[m] >= 0 ? p.scores[t * p.k + j0 + sub + m] : 0.0f;
        y[m] = more[m] >= 0 ? __ldcg(from[m]) : none;
        z[m] = more[m] > 0 ? __ldcg(next[m]) : none;
      }
#pragma unroll
      for (int m = 0; m < EACH; ++m) {
        y[m].x += z[m].x, y[m].y += z[m].y, y[m].z += z[m].z, y[m].w += z[m].w;
#pragma unroll 1
        for (int o = 1; o < more[m]; ++o) {
          const float4 v = __ldcg(next[m] + o * group * slot_floats);  // 4 slots a CTA, 4 floats a vector
          y[m].x += v.x, y[m].y += v.y, y[m].z += v.z, y[m].w += v.w;
        }
      }
#pragma unroll
      for (int l = 0; l < LANES * EACH; ++l) {
        float wl = w[EACH > 1 ? l : 0];
        float4 v = y[EACH > 1 ? l : 0];
        bool on = more[EACH > 1 ? l : 0] >= 0;
        if (LANES > 1) {
          wl = __shfl_sync(0xffffffffu, wl, l, LANES);
          v.x = __shfl_sync(0xffffffffu, v.x, l, LANES);
          v.y = __shfl_sync(0xffffffffu, v.y, l, LANES);
          v.z = __shfl_sync(0xffffffffu, v.z, l, LANES);
          v.w = __shfl_sync(0xffffffffu, v.w, l, LANES);
          on = __shfl_sync(0xffffffffu, (int)on, l, LANES) != 0;
        }
        if (on) {
          acc.x = fmaf(wl, v.x, acc.x);
          acc.y = fmaf(wl, v.y, acc.y);
          acc.z = fmaf(wl, v.z, acc.z);
          acc.w = fmaf(wl, v.w, acc.w);
        }
      }
    }
    if (sub == 0 && in)
      *reinterpret_cast<uint2*>(p.out + (long)t * p.H + col) =
          make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
  }
}

template <bool MX>
__global__ void __launch_bounds__(MX ? 448 : 384, 1) few_kernel(const __grid_constant__ FewMaps maps, FewParams p) {
  constexpr int kThreads = MX ? 448 : 384;  // warps: weights, MMA, 2 tokens, 8 epilogue, MXFP8: 2 scales
  constexpr int kEl = MX ? 128 : 64;  // K per block
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  const int b_bytes = p.unit_rows * 128;
  const int stage_bytes = 2 * kATile + (MX ? 1 : 2) * b_bytes;
  uint8_t* sf_smem = smem + (size_t)p.stages * stage_bytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + p.area);
  Schedule sched;
  const int R = p.T * p.k;
  sched.offset = reinterpret_cast<uint16_t*>(ctl + 1);
  sched.unit0 = sched.offset + p.E;
  sched.perm = sched.unit0 + p.E;
  sched.token = sched.perm + R;
  sched.unit_of = sched.token + R;
  sched.unit_e = sched.unit_of + R;
  sched.unit_r = sched.unit_e + p.max_units;
  sched.row_of = reinterpret_cast<uint8_t*>(sched.unit_r + p.max_units);
  sched.unit_n = sched.row_of + R;

  const int d_cols = (MX ? 1 : 2) * p.unit_rows;  // TMEM columns of one accumulator: at most 4 x 64 (MXFP8), 4 x 128
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  WaitCtx wc{&ctl->abort, p.hdr + kHdrAbort, p.hdr + kHdrError};

  // what the routing and the first tiles need soon, on its way from memory meanwhile
  const int early_id = !p.Wr && warp == 0 && lane < R ? __ldg(p.idx + lane) : -1;
  // a call that timed out left the abort word set: this one's results cannot be trusted either
  const int stale = c == 0 && threadIdx.x == 0 ? __ldcg(p.hdr + kHdrAbort) : 0;
  {
    const char* a = reinterpret_cast<const char*>(p.x);
    const long bytes = (long)p.T * p.H * 2, at = ((long)blockIdx.x * kThreads + threadIdx.x) * 128;
    if (at < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(a + at));
    if (!p.Wr && R > 32 && threadIdx.x * 32 < R) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.idx + threadIdx.x * 32));
    if (blockIdx.x == 0 && p.bias && threadIdx.x * 32 < p.E)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.bias + threadIdx.x * 32));
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&ctl->full_a[i], 1);
      mbar_init(&ctl->full_b[i], kProducers);
      mbar_init(&ctl->scales[i], 2);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->tfull[i], 1);
      mbar_init(&ctl->tempty[i], kEpilogue);
    }
    mbar_init(&ctl->drained, 1);
    ctl->abort = 0;
    ctl->failed = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
    if (lane < 3) tma_prefetch_desc(&maps.w[lane]);
    if (MX && lane < 3) tma_prefetch_desc(&maps.sf[lane]);
  }
  __syncthreads();

  // ---- routing and the quantised x
  if (MX) quantize_x(p, kThreads);
  if (p.Wr) {
    if (p.logit_tokens == 1)
      router_logits<1>(p, smem, kThreads);
    else
      router_logits<kLogitTokens>(p, smem, kThreads);
  }
  bool ok = true;
  if (MX || p.Wr) {
    __syncthreads();
    if (threadIdx.x == 0) red_release_gpu_add(word(p, kWordPrepared), 1u);
  }
  if (p.Wr) {
    if (blockIdx.x < p.T) {
      if (p.bias)
        for (int e = threadIdx.x; e < p.E; e += kThreads) reinterpret_cast<float*>(smem)[e] = p.bias[e];
      if (threadIdx.x == 0) ctl->go = wait_flag_geq(word(p, kWordPrepared), gridDim.x, wc) ? 1 : 0;
      __syncthreads();
      if (ctl->go)
        for (int t = blockIdx.x; t < p.T; t += gridDim.x)
          router_select(p, t, reinterpret_cast<float*>(smem), kThreads);
    }
    __syncthreads();
    if (threadIdx.x == 0) ctl->go = wait_flag_geq(word(p, kWordRouted), p.T, wc) ? 1 : 0;
    __syncthreads();
    ok = ctl->go != 0;
  }
  bool made = false;  // (uniform in warp 0, which alone knows)
  if (ok && R <= 32 && warp == 0) made = build_few(p, sched, ctl, early_id, lane);
  if (ok && R <= 32) made = __syncthreads_or(made);
  if (ok && !made) build_units(p, sched, smem, ctl, kThreads);
  // the stages' first loads (async proxy) come after these threads' use of the same shared memory
  fence_proxy_async_shared();
  if (ok && threadIdx.x < 4) {
    const int i = threadIdx.x, units = ctl->units;
    const int blocks = units * (p.I / 128) * (p.H / kEl);
    const int half = blocks >= kHalvesFrom * (int)gridDim.x ? (units + 1) / 2 : units;
    const int u0 = i & 1 ? half : 0, nu = i & 1 ? units - half : half;
    const Cut cut = make_cut(p.gemm[i >> 1], u0, nu, gridDim.x);
    ctl->cuts[i] = cut;
    ctl->runs[i] = run_of(cut, c);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  const int units = ok ? ctl->units : 0;

  // From here a wait that gives up ends its role.  What the threads of a role
  // do next is decided by all of them together: between the answers of two
  // threads to the same wait the abort word may change, and a barrier or a
  // warp-wide instruction that some have left never completes.
  int issued = 0;  // thread 0: blocks of weights asked for
  if (!ok && threadIdx.x == 0) ctl->failed = 1;
  if (units == 0) {
    // nothing routed: zeros (or a call that gave up)
    for (long i = (long)c * kThreads + threadIdx.x; i < (long)p.T * p.H; i += (long)gridDim.x * kThreads)
      p.out[i] = __float2bfloat16(0.0f);
  } else if (warp == 0) {
    // ---------------------------------------------------------------- weights
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      bool fine = true;
      for (int ph = 0; ph < 4; ++ph) {
        const Cut& cut = ctl->cuts[ph];
        const int g = ph >> 1;
        for (Run r = ctl->runs[ph]; r.left > 0 && fine; step(r, cut)) {
          const Seg s = r.seg;
          const int e = sched.unit_e[s.unit];
          const int col = g == 0 ? s.n * 128 : s.n * 256;
          const bool second = g == 0 || col + 128 < p.H;
          const CUtensorMap* m0 = &maps.w[g == 0 ? 0 : 2];
          const CUtensorMap* m1 = &maps.w[g == 0 ? 1 : 2];
          const int col1 = g == 0 ? col : col + 128;
          const uint32_t bytes = (second ? 2 : 1) * (kATile + (MX ? 512 : 0));
          for (int kb = s.k0; kb < s.k1; ++kb) {
            if (!mbar_wait(&ctl->empty[stage], phase ^ 1, wc)) {
              fine = false;
              break;
            }
            uint8_t* a = smem + (size_t)stage * stage_bytes;
            uint64_t* bar = &ctl->full_a[stage];
            mbar_arrive_expect_tx(bar, bytes);
            if constexpr (MX) {
              uint8_t* sf = sf_smem + stage * kSfBytes;
              tma_load_3d(a, m0, bar, col, kb * kEl, e);
              tma_load_3d(sf, &maps.sf[g == 0 ? 0 : 2], bar, col, kb * 4, e);
              if (second) {
                tma_load_3d(a + kATile, m1, bar, col1, kb * kEl, e);
                tma_load_3d(sf + 512, &maps.sf[g == 0 ? 1 : 2], bar, col1, kb * 4, e);
              }
            } else {
              tma_load_3d(a, m0, bar, col, kb * kEl, e);
              tma_load_3d(a + kATile / 2, m0, bar, col + 64, kb * kEl, e);
              if (second) {
                tma_load_3d(a + kATile, m1, bar, col1, kb * kEl, e);
                tma_load_3d(a + kATile + kATile / 2, m1, bar, col1 + 64, kb * kEl, e);
              }
            }
            ++issued;
            if (++stage == (uint32_t)p.stages) { stage = 0; phase ^= 1; }
          }
        }
      }
      if (!fine) ctl->failed = 1;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, count = 0;
      bool fine = true;
      for (int ph = 0; ph < 4; ++ph) {
        const Cut& cut = ctl->cuts[ph];
        const int g = ph >> 1;
        for (Run r = ctl->runs[ph]; r.left > 0 && fine; step(r, cut)) {
          const Seg s = r.seg;
          const int n = (sched.unit_n[s.unit] + 15) & ~15;
          const bool second = g == 0 || s.n * 256 + 128 < p.H;
          const uint32_t buf = count & 1;
          fine = mbar_wait(&ctl->tempty[buf], ((count >> 1) & 1) ^ 1, wc);
          if (!fine) break;
          tc_fence_after();
          const uint32_t d0 = tmem + buf * 2 * d_cols, d1 = d0 + d_cols;
          for (int kb = s.k0; kb < s.k1; ++kb) {
            fine = mbar_wait(&ctl->full_a[stage], phase, wc) && mbar_wait(&ctl->full_b[stage], phase, wc) &&
                   (!MX || mbar_wait(&ctl->scales[stage], phase, wc));
            if (!fine) break;
            tc_fence_after();
            // the tokens' operand was written with cp.async: order it before the tensor core's (async-proxy) reads
            fence_proxy_async_shared();
            const uint32_t a0 = smem_u32(smem + (size_t)stage * stage_bytes), b0 = a0 + 2 * kATile;
            if constexpr (MX) {
              const uint32_t sf = smem_u32(sf_smem + stage * kSfBytes);
              const uint32_t t = tmem + 256 + stage * 16;  // scales: two A tiles, B
              uint64_t ad = sdesc_sw128(a0, 16384, 1024), bd = sdesc_sw128(b0, 16, 1024);
              tmem_cp_32x128b_warpx4(t, sdesc_plain(sf + 1024, 16, 128));
              if (second) tmem_cp_32x128b_warpx4(t + 4, sdesc_plain(sf + 1536, 16, 128));
              tmem_cp_32x128b_warpx4(t + 8, sdesc_plain(sf + 2048, 16, 128));
#pragma unroll 1
              for (int k32 = 0; k32 < 4; ++k32) {
                const uint32_t idesc = idesc_mxf8(128, n, 1, 0, k32, k32);
                const uint32_t acc = kb > s.k0 || k32 > 0;
                mma_mxf8(d0, ad, bd, idesc, t, t + 8, acc);
                if (second) mma_mxf8(d1, ad + kATile / 16, bd, idesc, t + 4, t + 8, acc);
                ad += 4096 / 16;
                bd += 32 / 16;
              }
            } else {
              // second GEMM: a's bf16 and, as more columns, what its rounding
              // left (a matrix instruction of so few columns takes as long as
              // one of twice as many: it waits for its A operand)
              const uint32_t idesc = idesc_bf16(128, g == 0 ? n : 2 * n, 1, 0);
              uint64_t ad = sdesc_sw128(a0, 8192, 1024), bd = sdesc_sw128(b0, 16, 1024);
#pragma unroll
              for (int k16 = 0; k16 < 4; ++k16) {
                const uint32_t acc = kb > s.k0 || k16 > 0;
                mma_bf16(d0, ad, bd, idesc, acc);
                if (second) mma_bf16(d1, ad + kATile / 16, bd, idesc, acc);
                ad += 2048 / 16;
                bd += 32 / 16;
              }
            }
            mma_commit(&ctl->empty[stage]);
            if (++stage == (uint32_t)p.stages) { stage = 0; phase ^= 1; }
          }
          if (!fine) break;
          mma_commit(&ctl->tfull[buf]);
          ++count;
        }
      }
      if (!fine) {
        // no MMA may still run when the CTA leaves
        ctl->failed = 1;
        mma_commit(&ctl->drained);
        mbar_drain(&ctl->drained, 0, 1000000000ull);
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------------- tokens' operand
    const int tid = threadIdx.x - 64;
    const int ch = tid & 7;  // this thread's 16-byte piece of a row's 128 bytes
    uint32_t stage = 0, phase = 0;
    bool fine = true;
    for (int ph = 0; ph < 4; ++ph) {
      const Cut& cut = ctl->cuts[ph];
      const int g = ph >> 1;
      if (ctl->runs[ph].left == 0) continue;
      // x is ready at once (MXFP8: once every CTA has quantised its share),
      // a when every tile of this half of it is finished
      if (g == 1 || (MX && !p.Wr)) {
        // (a thread whose waits gave up votes too)
        bool go = fine;
        if (tid == 0 && fine)
          go = g == 0 ? wait_flag_geq(word(p, kWordPrepared), gridDim.x, wc)
                      : wait_flag_geq(word(p, kWordHidden + (ph & 1)), cut.units * (p.I / 128), wc);
        fine = vote_all(2, kProducers, go);
      }
      const int K = g == 0 ? p.H : p.I;
      const uint8_t* src = g == 0 ? (MX ? p.xq : reinterpret_cast<const uint8_t*>(p.x)) : static_cast<uint8_t*>(p.a);
      const uint8_t* sfs = g == 0 ? p.xsf : p.asf;
      const long lo = (long)p.T * p.k * p.I * 2;  // a's second part
      for (Run run = ctl->runs[ph]; run.left > 0 && fine; step(run, cut)) {
        const Seg s = run.seg;
        const int n = sched.unit_n[s.unit], r0 = sched.unit_r[s.unit];
        const int n16 = (n + 15) & ~15;
        const long row_bytes = (long)K * (MX ? 1 : 2);
        const int sf_row = MX && tid < n ? (g == 0 ? sched.token[r0 + tid] : r0 + tid) : 0;
        for (int kb = s.k0; kb < s.k1; ++kb) {
          if (!mbar_wait(&ctl->empty[stage], phase ^ 1, wc)) {
            fine = false;
            break;
          }
          const uint32_t dst = smem_u32(smem + (size_t)stage * stage_bytes + 2 * kATile);
          const uint8_t* from = src + (long)kb * 128 + ch * 16;
#pragma unroll 1
          for (int r = tid >> 3; r < n; r += kProducers / 8) {
            const uint8_t* piece = from + (g == 0 ? sched.token[r0 + r] : r0 + r) * row_bytes;
            const uint32_t d = dst + r * 128 + ((ch ^ (r & 7)) << 4);
            cp_async_16(d, piece);
            if (!MX && g == 1) cp_async_16(d + n16 * 128, piece + lo);
          }
          if (MX && tid < n)
            cp_async_4(smem_u32(sf_smem + stage * kSfBytes + 2048 + mx_sf_offset(tid, 0)),
                       sfs + (long)sf_row * (K / 32) + kb * 4, 4);
          cp_async_arrive_noinc(&ctl->full_b[stage]);
          if (++stage == (uint32_t)p.stages) { stage = 0; phase ^= 1; }
        }
      }
    }
    if (!fine) ctl->failed = 1;
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp < 12) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lanes this warp may read
    const int tid = threadIdx.x - 128;
    const int slot_floats = 2 * p.unit_rows * 128;
    uint32_t count = 0;
    bool fine = true;
    for (int ph = 0; ph < 4; ++ph) {
      const Cut& cut = ctl->cuts[ph];
      const int g = ph >> 1, half = ph & 1;
      for (Run r = ctl->runs[ph]; r.left > 0 && fine; step(r, cut)) {
        const Seg s = r.seg;
        const int n = sched.unit_n[s.unit], r0 = sched.unit_r[s.unit];
        const bool second = g == 0 || s.n * 256 + 128 < p.H;
        const bool whole = s.k0 == 0 && s.k1 == cut.kb;
        const int n16 = (n + 15) & ~15;
        const int lane_col = q * 32 + lane;
        const uint32_t buf = count & 1;
        fine = vote_all(1, kEpilogue, mbar_wait(&ctl->tfull[buf], (count >> 1) & 1, wc));
        if (!fine) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * 2 * d_cols + ((uint32_t)(q * 32) << 16);
        // four slots a CTA: of each half, the tile that its run ends in (1) or begins in (0)
        float* slot = p.part + (long)(4 * c + 2 * half + (s.k0 == 0 ? 1 : 0)) * slot_floats + lane_col;
#pragma unroll 1
        for (int i0 = ((warp - 4) >> 2) * 4; i0 < n; i0 += 8) {
          float v0[4], v1[4];
          tmem_ld4x2(d + i0, d + d_cols + i0, v0, v1);
          if (!MX && g == 1) {
            // (an infinite weight times a remainder of 0 or of the other sign: the first part says what y is)
            float l0[4], l1[4];
            tmem_ld4x2(d + n16 + i0, d + d_cols + n16 + i0, l0, l1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v0[i] += isfinite(v0[i]) ? l0[i] : 0.0f;
              v1[i] += isfinite(v1[i]) ? l1[i] : 0.0f;
            }
          }
          if (g == 0 && whole) {
            store_hidden<MX>(p, r0 + i0, n - i0, s.n * 128 + lane_col, lane, v0, v1);
            continue;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i0 + i >= n) break;
            // y's row, or the row of this part's slot
            float* to = whole ? p.y + (long)sched.perm[r0 + i0 + i] * p.H + s.n * 256 + lane_col : slot + (i0 + i) * 128;
            __stcg(to, v0[i]);
            if (second) __stcg(to + (whole ? 128 : p.unit_rows * 128), v1[i]);
          }
        }
        tc_fence_before();
        mbar_arrive(&ctl->tempty[buf]);
        ++count;
        if (g == 1) continue;
        if (!whole) {
          int first, last;
          seg_runs(cut, s.super, first, last);
          named_bar_sync(1, kEpilogue);
          if (tid == 0) {
            int32_t* arrivals = p.tile_count + s.unit * (p.I / 128) + s.n;
            const int old = atom_add_acq_rel(arrivals, 1);
            ctl->last = old == last - first;
            if (old == last - first) *arrivals = 0;
          }
          __syncwarp();
          named_bar_sync(1, kEpilogue);
          if (!ctl->last) continue;
          // a row a warp and more parts of it at once, or, where that leaves rows over, two rows (128 tokens, H
          // 2048, I 768, bf16: 113 us, the first form alone 117; 1 token 29.3, the second alone 29.9)
          if (n <= 8)
            join_hidden<MX, 1, 4>(p, cut, s, c & (cut.group - 1), half, first, last, r0, n, warp - 4, lane);
          else
            join_hidden<MX, 2, 3>(p, cut, s, c & (cut.group - 1), half, first, last, r0, n, warp - 4, lane);
        }
        // a finished tile of a
        named_bar_sync(1, kEpilogue);
        if (tid == 0) red_release_gpu_add(word(p, kWordHidden + half), 1u);
        __syncwarp();
      }
    }
    if (fine && units > 0) {
      named_bar_sync(1, kEpilogue);
      if (tid == 0) red_release_gpu_add(word(p, kWordSummed), 1u);
    }
    if (!fine && tid == 0) ctl->failed = 1;
  } else {
    // ---------------------------------------------------------------- MXFP8: weight scales
    // from [4 K blocks][128 columns] as they lie in memory to the layout that
    // the tensor core's scale copy takes; one warp per A tile
    const int i = warp - 12;
    uint32_t stage = 0, phase = 0;
    bool fine = true;
    for (int ph = 0; ph < 4; ++ph) {
      const int blocks = ctl->runs[ph].left;
      for (int b = 0; b < blocks && fine; ++b) {
        fine = __all_sync(0xffffffffu, mbar_wait(&ctl->full_a[stage], phase, wc));
        if (!fine) break;
        const uint8_t* raw = sf_smem + stage * kSfBytes + i * 512;
        uint8_t* tiled = sf_smem + stage * kSfBytes + 1024 + i * 512;
        uint32_t w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = *reinterpret_cast<const uint32_t*>(raw + r * 128 + lane * 4);
        const uint32_t l01 = __byte_perm(w[0], w[1], 0x5140), h01 = __byte_perm(w[0], w[1], 0x7362);
        const uint32_t l23 = __byte_perm(w[2], w[3], 0x5140), h23 = __byte_perm(w[2], w[3], 0x7362);
        const uint32_t o[4] = {__byte_perm(l01, l23, 0x5410), __byte_perm(l01, l23, 0x7632),
                               __byte_perm(h01, h23, 0x5410), __byte_perm(h01, h23, 0x7632)};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint32_t*>(tiled + mx_sf_offset(lane * 4 + j, 0)) = o[j];
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->scales[stage]);
        if (++stage == (uint32_t)p.stages) { stage = 0; phase ^= 1; }
      }
    }
    if (!fine && lane == 0) ctl->failed = 1;
  }

  tc_fence_before();
  // (the non-aligned barrier form, defined for warps that arrive diverged)
  asm volatile("barrier.sync 0;" ::: "memory");
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && ctl->failed) {
    // no copy may still be in flight when the CTA leaves, whichever role gave up
    for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
      mbar_drain(&ctl->full_a[i % p.stages], (uint32_t)((i / p.stages) & 1), 1000000000ull);
  }
  // eight threads an item while there are threads for it (1 token, H 2048, I 768: 26.6 us, of one 30.2; 4 tokens
  // 40.9 and 46.1)
  const bool one = (long)p.T * (p.H / 4) * 8 <= (long)gridDim.x * kThreads;
  if (units > 0 && (long)c * kThreads < (long)p.T * (p.H / 4) * (one ? 8 : 1)) {
    // the stages are free for the table (one that is too long for them is looked up as it goes)
    uint32_t* table = reinterpret_cast<uint32_t*>(smem);
    if ((size_t)units * ctl->cuts[2].supers * 4 <= (size_t)p.stages * stage_bytes)
      list_runs(ctl->cuts + 2, table, kThreads);
    else
      table = nullptr;
    if (threadIdx.x == 0) {
      ctl->go = wait_flag_geq(word(p, kWordSummed), gridDim.x, wc) ? 1 : 0;
      if (!ctl->go) ctl->failed = 1;
    }
    __syncthreads();
    if (ctl->go) {
      if (one)
        combine<8, 1>(p, sched, ctl->cuts + 2, table, kThreads);
      else
        combine<1, 8>(p, sched, ctl->cuts + 2, table, kThreads);
    }
  }
  if (threadIdx.x == 0) {
    // (a wait that only saw another's abort has not recorded it)
    if (stale | ctl->failed) atomicOr(p.hdr + kHdrError, MOK_ERRBIT_TIMEOUT);
    // the last CTA to end leaves the counters as it found them
    __threadfence();
    if (atomicAdd(p.hdr + kWordLeft, 1) == (int)gridDim.x - 1) {
      for (int i = kWordPrepared; i <= kWordLeft; ++i) p.hdr[i] = 0;
    }
  }
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

// Units of any routing of T tokens: a part-filled one per expert at most,
// beside full ones.
int units_bound(int T, int E, int k, int unit_rows) {
  const int R = T * k, experts = E < R ? E : R;
  const int n = experts + R / unit_rows;
  return n < R ? n : R;
}

// Neighbouring column tiles are taken by up to 8 CTAs side by side, so that
// they read up to 2 KB of each weight row together.  H 7168, I 2048: 8 tokens,
// MXFP8, 394 us, each tile apart 570, four together 399; 24 tokens, bf16, 430,
// 444 and 432.
FewShape gemm_shape(int tiles, int kb, int ctas) {
  FewShape f;
  f.group_shift = 3;
  while (f.group_shift > 0 && (tiles % (1 << f.group_shift) || (1 << f.group_shift) > ctas)) --f.group_shift;
  f.supers = tiles >> f.group_shift;
  f.kb = kb;
  return f;
}

// Tokens side by side in a part of the logits, and the parts: at most 64,
// enough SMs to read Wr at once and few enough parts to add up quickly.
void logit_parts(int T, int H, int ctas, int* tokens, int* parts, int* rows) {
  *tokens = T == 1 ? 1 : kLogitTokens;
  int n = ctas / ((T + *tokens - 1) / *tokens);
  if (n > 64) n = 64;
  if (n < 1) n = 1;
  int r = (H + n - 1) / n;
  r = (r + 7) & ~7;
  *rows = r;
  *parts = (H + r - 1) / r;
}

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
  const bool mx = prec == MOK_MXFP8;
  const int ctas = device_sm_count() > 0 ? device_sm_count() : 1;
  L.header = take(kHeaderWords * 4);
  // room for the units of any call of this H, I, E and k
  const size_t units = units_bound(MOK_FEW_MAX_TOKENS, s.E, s.k, 16);
  L.tiles = take(units * (s.I / 128) * 4);
  // (the parts' number falls as tokens are added: room for every call of up to T tokens)
  size_t logits = 0;
  for (int t = 1; t <= s.T; ++t) {
    int tokens, parts, rows;
    logit_parts(t, s.H, ctas, &tokens, &parts, &rows);
    if ((size_t)parts * t > logits) logits = (size_t)parts * t;
  }
  L.logits = take(logits * s.E * 4);
  L.xq = mx ? take((size_t)s.T * s.H) : 0;
  L.xsf = mx ? take((size_t)s.T * (s.H / 32)) : 0;
  L.a = take(R * s.I * (mx ? 1 : 4));
  L.asf = mx ? take(R * (s.I / 32)) : 0;
  L.part = take((size_t)ctas * 4 * 2 * few_unit_rows(s.T) * 128 * 4);
  L.y = take(R * s.H * 4);
  L.total = off;
  return L;
}

cudaError_t launch_few(FewParams p, bool mx, int* launches, cudaStream_t st) {
  *launches = 0;
  const int ctas = device_sm_count();
  FewMaps maps;
  const CUtensorMapDataType type = mx ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int es = mx ? 1 : 2, kel = mx ? 128 : 64;
  auto map = [&](CUtensorMap* m, CUtensorMap* ms, const void* w, const uint8_t* sf, int rows, int cols) {
    const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)p.E};
    const uint64_t str[2] = {(uint64_t)cols * es, (uint64_t)cols * rows * es};
    const uint32_t box[3] = {128u / es, (uint32_t)kel, 1};
    if (!make_tmap(m, type, 3, w, dims, str, box, true)) return false;
    if (!mx) return true;
    const uint64_t sdims[3] = {(uint64_t)cols, (uint64_t)rows / 32, (uint64_t)p.E};
    const uint64_t sstr[2] = {(uint64_t)cols, (uint64_t)cols * (rows / 32)};
    const uint32_t sbox[3] = {128, 4, 1};
    return make_tmap(ms, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, sf, sdims, sstr, sbox, false);
  };
  memset(&maps, 0, sizeof(maps));
  if (!map(&maps.w[0], &maps.sf[0], p.W1, p.sf1, p.H, p.I) || !map(&maps.w[1], &maps.sf[1], p.W3, p.sf3, p.H, p.I) ||
      !map(&maps.w[2], &maps.sf[2], p.W2, p.sf2, p.I, p.H))
    return cudaErrorInvalidValue;
  p.unit_rows = few_unit_rows(p.T);
  p.max_units = units_bound(p.T, p.E, p.k, p.unit_rows);
  p.gemm[0] = gemm_shape(p.I / 128, p.H / kel, ctas);
  p.gemm[1] = gemm_shape((p.H + 255) / 256, p.I / kel, ctas);
  logit_parts(p.T, p.H, ctas, &p.logit_tokens, &p.h_parts, &p.h_rows);
  const size_t stage = 2 * kATile + (size_t)p.unit_rows * (mx ? 128 : 256) + (mx ? kSfBytes : 0);
  const size_t rest = 1024 + sizeof(Ctl) + schedule_bytes(p.E, p.T * p.k, p.max_units);
  constexpr size_t kMost = 227 * 1024;
  // (an expert or more of every routed row)
  const long blocks = (long)p.max_units * (p.I / 128) * (p.H / kel);
  const int most = mx && blocks >= (long)kLongRun * ctas ? kMaxFewStages : kStages;
  int stages = (int)((kMost - rest) / stage);
  if (stages > most) stages = most;
  p.stages = stages;
  // (128 tokens of 32,768: the logits' inputs and sums are longer than four stages)
  size_t area = stages * stage;
  if (p.Wr) {
    const size_t tokens = (size_t)p.logit_tokens * 4;
    const size_t logits = p.h_rows * tokens + kLogitWarps * 256 * tokens;
    if (logits > area) area = logits;
  }
  p.area = (int)area;
  const size_t smem = rest + area;
  if (smem > kMost) return cudaErrorInvalidValue;
  const void* kernel = mx ? (const void*)few_kernel<true> : (const void*)few_kernel<false>;
  static std::atomic<uint64_t> allowed[2];
  cudaError_t e = allow_smem(kernel, kMost, allowed[mx]);
  if (e != cudaSuccess) return e;
  void* args[] = {&maps, &p};
  e = cudaLaunchCooperativeKernel(kernel, dim3(ctas), dim3(mx ? 448 : 384), args, smem, st);
  if (e != cudaSuccess) return e;
  *launches = 1;
  return cudaSuccess;
}

}  // namespace mok

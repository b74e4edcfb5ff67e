// The matrix products of the dense gated feed-forward block,
//
//   h = x W1,  u = x W3,  a = silu(h) * u,  out = a W2
//
// and of its gradients,
//
//   da = dout W2^T,  dh = da u sig(h) (1 + h (1 - sig(h))),  du = da silu(h)
//   dx = dh W1^T + du W3^T,  dW1 = x^T dh,  dW3 = x^T du,  dW2 = a^T dout
//
// one persistent kernel for all of them, bound by the tensor cores: a cluster
// of two CTAs shares a 256 x 256 tile of the result through one
// tcgen05.mma.cta_group::2 (each CTA brings its 128 rows of A and half of B:
// 32 KB a step of 64 along K, six steps in flight), FP32 sums in TMEM, two
// accumulators so that the epilogue of a tile runs beside the next one's
// products.  Operands are read as they lie in memory, either way round, by
// TMA, which also fills in zeros past their ends: no size has to be a multiple
// of a tile, only rows of whole 16 bytes are asked for.  Tiles are handed out
// by their number, and every sum runs along K in one order: results do not
// depend on timing.  Launches of a pass overlap (programmatic dependent
// launch): one that reads what the one before it writes has its barriers and
// TMEM ready when that ends, and one that does not runs beside it.
//
// A product of few tiles leaves most SMs idle, and a tile alone takes in no
// more than six steps of 32 KB a round trip to memory.  Such products run in a
// second form: a cluster of 4, 8 or 16 CTAs has one tile, each pair a part of
// K, and the parts' sums are exchanged through the cluster's shared memory, so
// that every CTA adds and stores a slice of the columns.
//
//   warp 0      TMA (both CTAs)
//   warp 1      TMEM allocation; the leader's issues the MMAs
//   warps 2-9   epilogue: two warps for each quarter of the accumulator's rows,
//               half of the columns each
#include <string.h>

#include <algorithm>
#include <atomic>

#include "ffn.cuh"
#include "ring.cuh"
#include "tc.cuh"

namespace mok {

namespace {

constexpr int kFfnStages = 6;
constexpr int kFfnOperandBytes = 128 * 128;               // A's or B's share of a CTA and stage
constexpr int kFfnStageBytes = 2 * kFfnOperandBytes;
constexpr int kFfnEpilogueWarps = 8;
constexpr int kFfnThreads = 64 + 32 * kFfnEpilogueWarps;
constexpr int kFfnOutStage = 32 * 64 * 2;                 // an epilogue warp's 32 x 64 bf16 on their way out
// M tiles (of 256 rows) taken together: their A and the B of the tiles beside them stay in L2
constexpr int kFfnGroup = 8;
constexpr uint64_t kFfnDrainNs = 20000000ull;             // 20 ms

struct FfnMaps {
  CUtensorMap a[2], b[2];
};

struct FfnCtl {
  uint64_t full[kFfnStages];
  uint64_t empty[kFfnStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint32_t tmem_base;
  int abort;
};

constexpr size_t kFfnSmem =
    1024 + kFfnStages * kFfnStageBytes + kFfnEpilogueWarps * kFfnOutStage + 256;
static_assert(kFfnSmem <= 227 * 1024, "shared memory of an SM");

// Whether an operand's rows run along M or N (and not along K).
__host__ __device__ constexpr bool ffn_a_mn(int mode) { return mode == FFN_DW13 || mode == FFN_DW2; }
__host__ __device__ constexpr bool ffn_b_mn(int mode) { return mode != FFN_DA && mode != FFN_DX; }

// Columns of the result that a tile covers (FFN_GATE: 128 of h and the same of u).
__host__ __device__ constexpr int ffn_tile_n(int mode) { return mode == FFN_GATE ? 128 : 256; }

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

template <int MODE>
__device__ __forceinline__ int n_tiles(const FfnParams& p) {
  const int n = ceil_div(p.N, ffn_tile_n(MODE));
  return MODE == FFN_DW13 ? 2 * n : n;
}

struct FfnTile {
  int m, n;    // tile's place: rows m * 256.., columns n * tile_n..
  int which;   // FFN_DW13: 0 dW1, 1 dW3
};

// Tiles in groups of kFfnGroup along M, along M first within a group.
template <int MODE>
__device__ __forceinline__ FfnTile tile_of(const FfnParams& p, int item) {
  const int mt = ceil_div(p.M, 256), nt = n_tiles<MODE>(p);
  const int group = item / (kFfnGroup * nt), rest = item - group * kFfnGroup * nt;
  const int rows = min(kFfnGroup, mt - group * kFfnGroup);
  FfnTile t;
  t.m = group * kFfnGroup + rest % rows;
  t.n = rest / rows;
  t.which = 0;
  if (MODE == FFN_DW13) {
    const int half = nt / 2;
    t.which = t.n >= half;
    t.n -= t.which * half;
  }
  return t;
}

// This CTA's operands of one step along K.  (A CTA whose rows of the result lie past the last needs no A: whatever its
// rows of the product are, they are not stored.)
template <int MODE>
__device__ __forceinline__ void ffn_loads(const FfnMaps& mp, const FfnTile& t, int kk, int k_half, int rank, bool with_a,
                                          uint8_t* a, uint8_t* b, uint32_t bar) {
  const int row = t.m * 256 + rank * 128;
  const int second = MODE == FFN_DX && kk >= k_half ? 1 : 0;
  const int k = (kk - second * k_half) * 64;
  if (!with_a) {
  } else if constexpr (ffn_a_mn(MODE)) {
    for (int c = 0; c < 2; ++c) tma_load_2d_pair(a + c * 8192, &mp.a[0], bar, row + c * 64, k);
  } else {
    tma_load_2d_pair(a, &mp.a[second], bar, k, row);
  }
  if constexpr (MODE == FFN_GATE) {
    // the leader's half of B are columns of W1, the other's the same columns of W3
    for (int c = 0; c < 2; ++c) tma_load_2d_pair(b + c * 8192, &mp.b[rank], bar, t.n * 128 + c * 64, k);
  } else {
    const int col = t.n * 256 + rank * 128;
    const CUtensorMap* m = &mp.b[MODE == FFN_DW13 ? t.which : second];
    if constexpr (ffn_b_mn(MODE)) {
      for (int c = 0; c < 2; ++c) tma_load_2d_pair(b + c * 8192, m, bar, col + c * 64, k);
    } else {
      tma_load_2d_pair(b, m, bar, k, col);
    }
  }
}

// ------------------------------------------------------------------ epilogue
__device__ __forceinline__ float ffn_sigmoid(float h) { return 1.0f / (1.0f + __expf(-h)); }
__device__ __forceinline__ void ffn_gate_gradient(float da, float h, float u, float& dh, float& du) {
  const float s = ffn_sigmoid(h);
  dh = da * u * s * (1.0f + h * (1.0f - s));
  du = da * (h * s);
}

// 32 rows of 128 bytes, a row a lane's 32 words, to memory in whole segments through the warp's staging buffer (16-byte
// pieces swizzled by row): put(row, piece of eight) for each.
template <typename Put>
__device__ __forceinline__ void store_rows(uint8_t* stage, int lane, const uint32_t (&w)[32], Put&& put) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  __syncwarp();
  const int ch = lane & 7;
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const int r = 4 * s + (lane >> 3);
    put(r, *reinterpret_cast<const uint4*>(stage + r * 128 + ((ch ^ (r & 7)) << 4)));
  }
  __syncwarp();
}
// 64 columns of bf16 from row0, col0 on of dst [rows, ld].  ld is a multiple of eight: a piece lies inside or outside.
__device__ __forceinline__ void store_block(uint8_t* stage, int lane, const uint32_t (&w)[32], __nv_bfloat16* dst,
                                            int row0, int rows, int col0, int ld) {
  const int col = col0 + (lane & 7) * 8;
  store_rows(stage, lane, w, [&](int r, const uint4& v) {
    if (row0 + r < rows && col < ld) *reinterpret_cast<uint4*>(dst + (long)(row0 + r) * ld + col) = v;
  });
}

// h and u as they are kept for the backward pass: f32, as an epilogue's lanes have them, [row / 32][column / 4][row % 32]
// fours of columns, so that a warp's 32 rows are 512 bytes in one piece both when they are written and when they are
// read, and nothing has to be turned.  (In bf16 they were two roundings more in every gradient: relative errors of dx,
// dW1 and dW3 of 3.0e-3 where 2.4e-3 come from dh, du and the result themselves.)
__device__ __forceinline__ long kept_at(int row, int col, int N) {
  return ((long)(row >> 5) * (N >> 2) + (col >> 2)) * 32 + (row & 31);
}
__device__ __forceinline__ float4 zero4() { return make_float4(0.0f, 0.0f, 0.0f, 0.0f); }

// The 32 rows from row0 and this warp's half of a tile's columns.  `acc`: the accumulator's
// address for these rows; `ready` waits for it.
template <int MODE, typename Ready>
__device__ __forceinline__ bool ffn_epilogue(const FfnParams& p, const FfnTile& t, uint32_t acc, int row0, int half,
                                             int lane, uint8_t* stage, Ready&& ready) {
  if constexpr (MODE == FFN_GATE) {
    if (!ready()) return false;
    const int col = t.n * 128 + half * 64;
    const bool keeps = p.h && row0 + lane < p.M;
    uint32_t aw[32];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t h[32], u[32];
      tmem_ld32_issue(acc + half * 64 + c * 32, h);
      tmem_ld32_issue(acc + 128 + half * 64 + c * 32, u);
      tmem_wait_ld();
      tmem_regs_ready(h);
      tmem_regs_ready(u);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float h0 = __uint_as_float(h[2 * i]), h1 = __uint_as_float(h[2 * i + 1]);
        const float u0 = __uint_as_float(u[2 * i]), u1 = __uint_as_float(u[2 * i + 1]);
        aw[16 * c + i] = pack_bf16x2(h0 * ffn_sigmoid(h0) * u0, h1 * ffn_sigmoid(h1) * u1);
      }
      if (keeps) {
        uint4* hk = reinterpret_cast<uint4*>(p.h) + kept_at(row0 + lane, col + c * 32, p.N);
        uint4* uk = reinterpret_cast<uint4*>(p.u) + kept_at(row0 + lane, col + c * 32, p.N);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (col + c * 32 + i * 4 >= p.N) break;
          __stcs(hk + i * 32, make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]));
          __stcs(uk + i * 32, make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]));
        }
      }
    }
    store_block(stage, lane, aw, p.out[0], row0, p.M, col, p.N);
  } else if constexpr (MODE == FFN_DA) {
    // 32 columns of h and u are on their way while the products still run or the 32 before are worked on
    const int col0 = t.n * 256 + half * 128;
    const bool there = row0 + lane < p.M;
    const float4* hk = reinterpret_cast<const float4*>(p.h) + kept_at(row0 + lane, col0, p.N);
    const float4* uk = reinterpret_cast<const float4*>(p.u) + kept_at(row0 + lane, col0, p.N);
    float4 hv[8], uv[8];
    auto fetch = [&](int i, int c4) {  // the c4-th four from col0
      const bool in = there && col0 + c4 * 4 < p.N;
      hv[i] = in ? __ldcs(hk + c4 * 32) : zero4();
      uv[i] = in ? __ldcs(uk + c4 * 32) : zero4();
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) fetch(i, i);
    if (!ready()) return false;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float da[32];
      uint32_t w[32];  // dh, then du
      tmem_ld32(acc + half * 128 + c * 32, da);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h[4] = {hv[i].x, hv[i].y, hv[i].z, hv[i].w}, u[4] = {uv[i].x, uv[i].y, uv[i].z, uv[i].w};
        if (c < 3) fetch(i, c * 8 + 8 + i);
        float dh[4], du[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ffn_gate_gradient(da[4 * i + k], h[k], u[k], dh[k], du[k]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          w[2 * i + k] = pack_bf16x2(dh[2 * k], dh[2 * k + 1]);
          w[16 + 2 * i + k] = pack_bf16x2(du[2 * k], du[2 * k + 1]);
        }
      }
      const int col = col0 + c * 32 + (lane & 3) * 8;
      __nv_bfloat16* dst = p.out[(lane & 7) >> 2];
      store_rows(stage, lane, w, [&](int r, const uint4& v) {
        if (row0 + r < p.M && col < p.N) *reinterpret_cast<uint4*>(dst + (long)(row0 + r) * p.N + col) = v;
      });
    }
  } else {
    if (!ready()) return false;
#pragma unroll 1
    for (int g = 0; g < 2; ++g) {
      const int col = t.n * 256 + half * 128 + g * 64;
      uint32_t ra[32], rb[32], w[32];
      tmem_ld32_issue(acc + half * 128 + g * 64, ra);
      tmem_ld32_issue(acc + half * 128 + g * 64 + 32, rb);
      tmem_wait_ld();
      tmem_regs_ready(ra);
      tmem_regs_ready(rb);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        w[i] = pack_bf16x2(__uint_as_float(ra[2 * i]), __uint_as_float(ra[2 * i + 1]));
        w[16 + i] = pack_bf16x2(__uint_as_float(rb[2 * i]), __uint_as_float(rb[2 * i + 1]));
      }
      store_block(stage, lane, w, MODE == FFN_DW13 && t.which ? p.out[1] : p.out[0], row0, p.M, col, p.N);
    }
  }
  return true;
}

// A launch's place in the stream (all threads), and from here on the next one may start where there is room: what that may
// read without waiting stands.
__device__ __forceinline__ void launch_in_turn(const FfnParams& p) {
  if (p.after == FFN_READS_IT) griddep_wait();
  griddep_launch_dependents();
}

// Bytes of a step that both CTAs of a pair bring: their halves of B, and A where they have rows of the result.
__device__ __forceinline__ uint32_t step_bytes(const FfnParams& p, const FfnTile& t, uint32_t a_bytes = kFfnOperandBytes) {
  return 2 * kFfnOperandBytes + a_bytes * (t.m * 256 + 128 < p.M ? 2u : 1u);
}

// ------------------------------------------------------------------ kernel
template <int MODE>
__global__ void __launch_bounds__(kFfnThreads, 1) ffn_kernel(const __grid_constant__ FfnMaps maps, const FfnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = base;
  uint8_t* sB = sA + kFfnStages * kFfnOperandBytes;
  uint8_t* sOut = sB + kFfnStages * kFfnOperandBytes;
  FfnCtl* ctl = reinterpret_cast<FfnCtl*>(sOut + kFfnEpilogueWarps * kFfnOutStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{&ctl->abort, &p.hdr[kHdrAbort], &p.hdr[kHdrError]};
  const int rank = (int)cluster_ctarank();
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int items = ceil_div(p.M, 256) * n_tiles<MODE>(p);
  const int k_half = ceil_div(p.K, 64), k_iters = MODE == FFN_DX ? 2 * k_half : k_half;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kFfnStages; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->tfull[i], 1);
      mbar_init(&ctl->tempty[i], 2 * kFfnEpilogueWarps);
    }
    ctl->abort = 0;
    ctl->tmem_base = 0;
    fence_mbar_init();
    // a call that timed out left the abort word set: this one's results cannot be trusted either
    if (blockIdx.x == 0 && *reinterpret_cast<volatile int*>(&p.hdr[kHdrAbort])) atomicOr(&p.hdr[kHdrError], MOK_ERRBIT_TIMEOUT);
  }
  if (warp == 0 && lane < 2) {
    tma_prefetch_desc(&maps.a[lane]);
    tma_prefetch_desc(&maps.b[lane]);
  }
  if (warp == 1) {
    tmem_alloc_pair(&ctl->tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers stand before either signals the other's
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  launch_in_turn(p);

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int item = first; ok && item < items; item += step) {
        const FfnTile t = tile_of<MODE>(p, item);
        const bool with_a = t.m * 256 + rank * 128 < p.M;
        for (int kk = 0; kk < k_iters; ++kk) {
          if (!mbar_wait(&ctl->empty[stage], phase ^ 1, wc)) { ok = false; break; }
          // (the leader's barrier counts both CTAs' bytes)
          if (rank == 0) mbar_arrive_expect_tx(&ctl->full[stage], step_bytes(p, t, p.a_rows * 128));
          ffn_loads<MODE>(maps, t, kk, k_half, rank, with_a, sA + stage * kFfnOperandBytes, sB + stage * kFfnOperandBytes,
                          mapa_shared(&ctl->full[stage], 0));
          if (++stage == kFfnStages) { stage = 0; phase ^= 1; }
        }
      }
      // no copy may be in flight, nor an MMA read these stages, when the CTA leaves: each stage's last
      // fill is released by the MMAs that read it (after a timeout for a limited time)
      const uint64_t t0 = globaltimer();
      for (int j = 0; j < kFfnStages; ++j) {
        const uint64_t spent = globaltimer() - t0;
        if (spent < kFfnDrainNs) mbar_drain(&ctl->empty[stage], phase ^ 1, kFfnDrainNs - spent);
        if (++stage == kFfnStages) { stage = 0; phase ^= 1; }
      }
    }
  } else if (warp == 1) {
    // (one thread alone waits and issues: lanes that each waited could find a wait given up at different times, and part)
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, tcount = 0;
      constexpr uint32_t idesc = idesc_bf16(256, 256, ffn_a_mn(MODE) ? 1 : 0, ffn_b_mn(MODE) ? 1 : 0);
      bool ok = rank == 0;
      for (int item = first; ok && item < items; item += step, ++tcount) {
        const uint32_t buf = tcount & 1, tph = (tcount >> 1) & 1;
        if (!mbar_wait_cluster(&ctl->tempty[buf], tph ^ 1, wc)) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * 256;
        for (int kk = 0; kk < k_iters; ++kk) {
          if (!mbar_wait(&ctl->full[stage], phase, wc)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + stage * kFfnOperandBytes), b0 = smem_u32(sB + stage * kFfnOperandBytes);
#pragma unroll
          for (int k16 = 0; k16 < 4; ++k16) {
            const uint64_t ad = ffn_a_mn(MODE) ? sdesc_sw128(a0 + k16 * 2048, 8192, 1024) : sdesc_sw128(a0 + k16 * 32, 16, 1024);
            const uint64_t bd = ffn_b_mn(MODE) ? sdesc_sw128(b0 + k16 * 2048, 8192, 1024) : sdesc_sw128(b0 + k16 * 32, 16, 1024);
            mma_bf16_pair(d, ad, bd, idesc, (kk | k16) != 0 ? 1u : 0u);
          }
          mma_commit_pair(&ctl->empty[stage]);
          if (++stage == kFfnStages) { stage = 0; phase ^= 1; }
        }
        if (ok) mma_commit_pair(&ctl->tfull[buf]);
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;  // TMEM lanes that this warp may read; columns it takes
    uint8_t* stage_out = sOut + (warp - 2) * kFfnOutStage;
    uint32_t tcount = 0;
    for (int item = first; item < items; item += step, ++tcount) {
      const FfnTile t = tile_of<MODE>(p, item);
      const uint32_t buf = tcount & 1, tph = (tcount >> 1) & 1;
      auto ready = [&]() {
        // (what the warp loads from TMEM it loads together: it goes on together or not at all)
        if (!__all_sync(0xffffffffu, mbar_wait(&ctl->tfull[buf], tph, wc))) return false;
        tc_fence_after();
        return true;
      };
      if (!ffn_epilogue<MODE>(p, t, tmem + ((uint32_t)(q * 32) << 16) + buf * 256, t.m * 256 + rank * 128 + q * 32, half,
                              lane, stage_out, ready))
        break;
      tc_fence_before();
      __syncwarp();
      // (the leader's MMA warp waits for both CTAs' epilogues)
      if (lane == 0) mbar_arrive_cluster(mapa_shared(&ctl->tempty[buf], 0));
    }
  }

  tc_fence_before();
  // (the non-aligned barrier form, defined for warps that arrive diverged)
  asm volatile("barrier.sync 0;" ::: "memory");
  __syncwarp();  // (the cluster's barrier is of the aligned form)
  // neither CTA leaves (nor frees TMEM) while the other may still signal its barriers or run MMAs on its memory
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
  // (what comes after this launch comes after the one before it too)
  if (p.after == FFN_BESIDE_IT) griddep_wait();
}

// ------------------------------------------------------------------ kernel, few tiles
// S pairs of CTAs share a tile: pair i sums the i-th part of K.  Nothing in it loops over tiles, and every thread comes
// to every cluster barrier, whether a wait gave up or not.
//
// After the sums: each warp of the epilogue sends its 32 rows x 128 columns to the CTAs of its rank that add them, as
// fours of columns by rows, [part][column / 4 of the slice][row]; these then add the parts in the order of K.  FFN_GATE:
// a slice is as many columns of h and the same of u.
//
// A product with no more than 128 rows brings as much of A as it has: its stages are shorter, and more of them are on
// their way (1 token, H 7168, I 2048: ten of 18 KB in place of six of 32).
constexpr int kFfnMostStages = 10;
struct FfnFewCtl {
  uint64_t full[kFfnMostStages];
  uint64_t empty[kFfnMostStages];
  uint64_t done;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(FfnFewCtl) <= 256 && sizeof(FfnCtl) <= 256, "the control block's place");

template <int MODE>
__device__ __forceinline__ void few_store4(const FfnParams& p, const FfnTile& t, int row, int col, const float4& v,
                                           const float4& w, const float4& hv, const float4& uv) {
  // col: within the tile's columns; (rows and sizes are in whole fours)  FFN_GATE: v, w are h and u; FFN_DA: hv, uv
  const float x[4] = {v.x, v.y, v.z, v.w}, y[4] = {w.x, w.y, w.z, w.w};
  const int c = t.n * ffn_tile_n(MODE) + col;
  const long at = (long)row * p.N + c;
  auto put = [&](__nv_bfloat16* dst, const float (&f)[4]) {
    *reinterpret_cast<uint2*>(dst + at) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  };
  if constexpr (MODE == FFN_GATE) {
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = x[i] * ffn_sigmoid(x[i]) * y[i];
    put(p.out[0], a);
    if (p.h) {
      __stcs(reinterpret_cast<float4*>(p.h) + kept_at(row, c, p.N), v);
      __stcs(reinterpret_cast<float4*>(p.u) + kept_at(row, c, p.N), w);
    }
  } else if constexpr (MODE == FFN_DA) {
    const float h[4] = {hv.x, hv.y, hv.z, hv.w}, u[4] = {uv.x, uv.y, uv.z, uv.w};
    float dh[4], du[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ffn_gate_gradient(x[i], h[i], u[i], dh[i], du[i]);
    put(p.out[0], dh);
    put(p.out[1], du);
  } else {
    put(MODE == FFN_DW13 && t.which ? p.out[1] : p.out[0], x);
  }
}

template <int MODE, int S>
__global__ void __launch_bounds__(kFfnThreads, 1) ffn_few_kernel(const __grid_constant__ FfnMaps maps, const FfnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t a_slot = p.a_rows * 128, slot = a_slot + kFfnOperandBytes;
  const int stages = min(kFfnMostStages, (int)(kFfnStages * kFfnStageBytes / slot));
  // (B first: an MMA reads 128 rows of A, past what is there, rows whose sums no one wants)
  uint8_t* sB = base;
  uint8_t* sA = sB + stages * kFfnOperandBytes;
  FfnFewCtl* ctl = reinterpret_cast<FfnFewCtl*>(base + kFfnStages * kFfnStageBytes + kFfnEpilogueWarps * kFfnOutStage);
  // where the parts of this CTA's slice arrive: the stages' place, once their last MMAs are done
  float4* sums = reinterpret_cast<float4*>(base);
  constexpr int kSlice4 = 64 / S;  // fours of columns in a slice, of 64 of the tile
  static_assert(S * kSlice4 * 128 * 16 <= kFfnStages * kFfnStageBytes, "a slice's parts where the stages were");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{&ctl->abort, &p.hdr[kHdrAbort], &p.hdr[kHdrError]};
  const int cta = (int)cluster_ctarank(), rank = cta & 1, part = cta >> 1;
  const FfnTile t = tile_of<MODE>(p, blockIdx.x / (2 * S));
  const int k_half = ceil_div(p.K, 64), k_iters = MODE == FFN_DX ? 2 * k_half : k_half;
  const int k0 = k_iters * part / S, steps = k_iters * (part + 1) / S - k0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    mbar_init(&ctl->done, 1);
    ctl->abort = 0;
    ctl->tmem_base = 0;
    fence_mbar_init();
    if (blockIdx.x == 0 && *reinterpret_cast<volatile int*>(&p.hdr[kHdrAbort])) atomicOr(&p.hdr[kHdrError], MOK_ERRBIT_TIMEOUT);
  }
  if (warp == 0 && lane < 2) {
    tma_prefetch_desc(&maps.a[lane]);
    tma_prefetch_desc(&maps.b[lane]);
  }
  if (warp == 1) {
    tmem_alloc_pair(&ctl->tmem_base, 256);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // all barriers stand before any CTA signals another's
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  launch_in_turn(p);

  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      const bool with_a = t.m * 256 + rank * 128 < p.M;
      uint32_t stage = 0, phase = 0;
      int i = 0;
      for (; i < steps; ++i) {
        if (!mbar_wait(&ctl->empty[stage], phase ^ 1, wc)) { ok = false; break; }
        if (rank == 0) mbar_arrive_expect_tx(&ctl->full[stage], step_bytes(p, t, a_slot));
        ffn_loads<MODE>(maps, t, k0 + i, k_half, rank, with_a, sA + stage * a_slot, sB + stage * kFfnOperandBytes,
                        mapa_shared(&ctl->full[stage], (uint32_t)(cta & ~1)));
        if ((int)++stage == stages) { stage = 0; phase ^= 1; }
      }
      // Whoever gives up, no copy is in flight when the stages serve for the sums, nor when the CTA leaves: the leader,
      // whose barriers count both CTAs' bytes, waits for each stage's last fill (the MMAs did for those before, and wait for
      // these meanwhile).  Where the two CTAs gave up at different steps, not all that was asked for is counted: a fill that
      // is short of the other's bytes, or the other's fills that were never armed here.  Those land within the limit.
      if (rank == 0) {
        const uint64_t t0 = globaltimer();
        for (int f = last_fills_from(i, stages); f < i; ++f) {
          if (mbar_try_wait(&ctl->full[f % stages], fill_parity(f, stages))) continue;
          const uint64_t spent = globaltimer() - t0;
          if (spent < kFfnDrainNs) mbar_drain(&ctl->full[f % stages], fill_parity(f, stages), kFfnDrainNs - spent);
        }
        while (!ok && globaltimer() - t0 < kFfnDrainNs) __nanosleep(10000);
      }
    }
  } else if (warp == 1 && rank == 0) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16(256, 256, ffn_a_mn(MODE) ? 1 : 0, ffn_b_mn(MODE) ? 1 : 0);
      uint32_t stage = 0, phase = 0;
      for (int i = 0; i < steps; ++i) {
        if (!mbar_wait(&ctl->full[stage], phase, wc)) { ok = false; break; }
        tc_fence_after();
        const uint32_t a0 = smem_u32(sA + stage * a_slot), b0 = smem_u32(sB + stage * kFfnOperandBytes);
#pragma unroll
        for (int k16 = 0; k16 < 4; ++k16) {
          const uint64_t ad = ffn_a_mn(MODE) ? sdesc_sw128(a0 + k16 * 2048, 8192, 1024) : sdesc_sw128(a0 + k16 * 32, 16, 1024);
          const uint64_t bd = ffn_b_mn(MODE) ? sdesc_sw128(b0 + k16 * 2048, 8192, 1024) : sdesc_sw128(b0 + k16 * 32, 16, 1024);
          mma_bf16_pair(tmem, ad, bd, idesc, (i | k16) != 0 ? 1u : 0u);
        }
        mma_commit_pair(&ctl->empty[stage], 3u << (cta & ~1));
        if ((int)++stage == stages) { stage = 0; phase ^= 1; }
      }
      mma_commit_pair(&ctl->done, 3u << (cta & ~1));
    }
  }
  __syncwarp();
  // every MMA of the pair is done: the sums stand, the stages are free
  const int q = warp & 3, half = (warp - 2) >> 2;  // epilogue warps: TMEM lanes that this warp may read; columns it takes
  // (a warp comes to the cluster's barrier, and to its loads from TMEM, in one piece and of one mind)
  const bool summed = __all_sync(0xffffffffu, mbar_wait(&ctl->done, 0, wc));
  if (!summed) {
    // the leader commits `done` whether its own waits gave up or not: no MMA is under way past here either
    mbar_drain(&ctl->done, 0, kWaitLimitNs);
    __syncwarp();
  }
  tc_fence_after();
  cluster_sync();
  const int row0 = t.m * 256 + rank * 128;
  // what this thread adds and stores at last: eight rows x four fours a warp at a time (whole sectors out, no two lanes on
  // a bank), kAtOnce of them together.  FFN_DA: the first ones' h and u are on their way from here on
  constexpr int kPer = MODE == FFN_GATE ? kSlice4 / 2 : kSlice4, kAcross = (kPer + 3) / 4;  // fours of results in a slice
  constexpr int kAtOnce = 4;
  const int rows = min(128, p.M - row0), blocks = (rows + 7) / 8 * kAcross;
  auto place = [&](int i, int& row, int& c) {
    row = i / kAcross * 8 + (lane & 7);
    c = i % kAcross * 4 + (lane >> 3);
    return i < blocks && row < rows && c < kPer && t.n * ffn_tile_n(MODE) + (part * kPer + c) * 4 < p.N;
  };
  float4 hv[kAtOnce], uv[kAtOnce];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      hv[j] = uv[j] = zero4();
      if constexpr (MODE == FFN_DA) {
        int row, c;
        if (!place(i0 + j * kFfnEpilogueWarps, row, c)) continue;
        const long at = kept_at(row0 + row, t.n * 256 + (part * kPer + c) * 4, p.N);
        hv[j] = __ldcs(reinterpret_cast<const float4*>(p.h) + at);
        uv[j] = __ldcs(reinterpret_cast<const float4*>(p.u) + at);
      }
    }
  };
  if (warp >= 2) fetch(warp - 2);
  if (warp >= 2 && summed && row0 + q * 32 < p.M) {
    const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      // 32 columns, in the tile's order of fours: 0 to 63 (FFN_GATE: h and then u)
      const int col = half * 128 + i * 32;
      float v[32];
      tmem_ld32(acc + col, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c4 = col / 4 + j;
        // whose slice: FFN_GATE has half of a slice of h and half of u
        int owner, in_slice;
        if (MODE == FFN_GATE) {
          owner = (c4 & 31) / (kSlice4 / 2);
          in_slice = (c4 >> 5) * (kSlice4 / 2) + (c4 & 31) % (kSlice4 / 2);
        } else {
          owner = c4 / kSlice4;
          in_slice = c4 % kSlice4;
        }
        const uint32_t to = mapa_shared(sums + (part * kSlice4 + in_slice) * 128 + q * 32 + lane, (uint32_t)(2 * owner + rank));
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v[4 * j]), "f"(v[4 * j + 1]),
                     "f"(v[4 * j + 2]), "f"(v[4 * j + 3])
                     : "memory");
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 256);
  if (warp >= 2 && summed) {
    auto add = [&](int at, int row) {
      float4 s = sums[at * 128 + row];
#pragma unroll
      for (int j = 1; j < S; ++j) {
        const float4 w = sums[(j * kSlice4 + at) * 128 + row];
        s.x += w.x, s.y += w.y, s.z += w.z, s.w += w.w;
      }
      return s;
    };
#pragma unroll 1
    for (int i = warp - 2; i < blocks; i += kAtOnce * kFfnEpilogueWarps) {
      if (i >= kAtOnce * kFfnEpilogueWarps) fetch(i);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        int row, c;
        if (!place(i + j * kFfnEpilogueWarps, row, c)) continue;
        const float4 v = add(c, row), w = MODE == FFN_GATE ? add(kPer + c, row) : v;
        few_store4<MODE>(p, t, row0 + row, (part * kPer + c) * 4, v, w, hv[j], uv[j]);
      }
    }
  }
  if (p.after == FFN_BESIDE_IT) griddep_wait();
}

// ------------------------------------------------------------------ launches
// Steps along K that a pair's part has at least.
constexpr int kFfnPartSteps = 2;

// Rows along K: boxes of 128 rows x 64 of K; along M or N: 64 of K x 64.
bool operand_map(CUtensorMap* m, const FfnOperand& o, bool mn, int rows = 128) {
  const uint64_t dims[2] = {(uint64_t)o.cols, (uint64_t)o.rows};
  const uint64_t str[1] = {(uint64_t)o.cols * 2};
  const uint32_t box[2] = {64, mn ? 64u : (uint32_t)rows};
  return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, o.p, dims, str, box, true);
}

// What the device holds of a kernel's clusters at once, asked for once per device (`held`: a number per device, the
// kernel's own), and its shared memory allowed.
cudaError_t clusters_held(const void* kernel, const cudaLaunchConfig_t& cfg, std::atomic<int>* held, int* clusters) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  *clusters = dev < 64 ? held[dev].load(std::memory_order_relaxed) : 0;
  if (*clusters) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFfnSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(clusters, kernel, &cfg);
  if (e != cudaSuccess) return e;
  if (*clusters < 1) *clusters = -1;  // (none: known from here on)
  if (dev < 64) held[dev].store(*clusters, std::memory_order_relaxed);
  return cudaSuccess;
}

struct FfnLaunch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
};
void prepare(FfnLaunch* l, const FfnParams& p, int cluster, unsigned grid, cudaStream_t st) {
  l->cfg = {};
  l->attr[0].id = cudaLaunchAttributeClusterDimension;
  l->attr[0].val.clusterDim.x = (unsigned)cluster;
  l->attr[0].val.clusterDim.y = 1;
  l->attr[0].val.clusterDim.z = 1;
  l->attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  l->attr[1].val.programmaticStreamSerializationAllowed = 1;
  l->cfg.gridDim = dim3(grid);
  l->cfg.blockDim = dim3(kFfnThreads);
  l->cfg.dynamicSmemBytes = kFfnSmem;
  l->cfg.stream = st;
  l->cfg.attrs = l->attr;
  l->cfg.numAttrs = p.after == FFN_AFTER_ALL ? 1 : 2;
}

// The tile of a cluster of 2 S CTAs, if the device holds as many as there are tiles (*done: whether it was launched).
template <int MODE, int S>
cudaError_t launch_few_tiles(const FfnMaps& maps, const FfnParams& p, int tiles, int k_iters, bool* done, cudaStream_t st) {
  *done = false;
  if (tiles * 2 * S > p.sms || k_iters < S * kFfnPartSteps) return cudaSuccess;
  static std::atomic<int> held[64];
  FfnLaunch l;
  prepare(&l, p, 2 * S, 2u * S * (unsigned)tiles, st);
  int clusters = 0;
  const cudaError_t e = clusters_held((const void*)ffn_few_kernel<MODE, S>, l.cfg, held, &clusters);
  if (e != cudaSuccess) return e;
  if (clusters < tiles) return cudaSuccess;
  *done = true;
  return cudaLaunchKernelEx(&l.cfg, ffn_few_kernel<MODE, S>, maps, p);
}

int tiles_of(int mode, int M, int N) { return ceil_div(M, 256) * ceil_div(N, ffn_tile_n(mode)) * (mode == FFN_DW13 ? 2 : 1); }
int steps_of(int mode, int K) { return ceil_div(K, 64) * (mode == FFN_DX ? 2 : 1); }

template <int MODE>
cudaError_t launch_mode(const FfnMaps& maps, const FfnParams& p, cudaStream_t st) {
  const int tiles = tiles_of(MODE, p.M, p.N), k_iters = steps_of(MODE, p.K);
  bool done;
  cudaError_t e = launch_few_tiles<MODE, 8>(maps, p, tiles, k_iters, &done, st);
  if (e == cudaSuccess && !done) e = launch_few_tiles<MODE, 4>(maps, p, tiles, k_iters, &done, st);
  if (e == cudaSuccess && !done) e = launch_few_tiles<MODE, 2>(maps, p, tiles, k_iters, &done, st);
  if (e != cudaSuccess || done) return e;
  static std::atomic<int> held[64];
  FfnLaunch l;
  prepare(&l, p, 2, (unsigned)device_sm_count() & ~1u, st);
  int clusters = 0;
  e = clusters_held((const void*)ffn_kernel<MODE>, l.cfg, held, &clusters);
  if (e != cudaSuccess) return e;
  if (clusters < 1) return cudaErrorNotSupported;
  l.cfg.gridDim = dim3(2u * (unsigned)std::min(tiles, clusters));
  return cudaLaunchKernelEx(&l.cfg, ffn_kernel<MODE>, maps, p);
}

}  // namespace

void ffn_share_sms(const FfnSize (&two)[2], int (&sms)[2]) {
  const int all = device_sm_count();
  int tiles[2], steps[2], S[2] = {1, 1};
  for (int i = 0; i < 2; ++i) {
    tiles[i] = tiles_of(two[i].mode, two[i].M, two[i].N);
    steps[i] = steps_of(two[i].mode, two[i].K);
    sms[i] = all;
  }
  if ((long)tiles[0] + tiles[1] > all / 2) return;
  // the longer parts are halved as long as there is room
  bool open[2] = {true, true};
  while (open[0] || open[1]) {
    const int i = open[0] && (!open[1] || steps[0] / S[0] >= steps[1] / S[1]) ? 0 : 1;
    if (S[i] < 8 && steps[i] >= 2 * S[i] * kFfnPartSteps && 2 * (tiles[0] * S[0] + tiles[1] * S[1] + tiles[i] * S[i]) <= all)
      S[i] *= 2;
    else
      open[i] = false;
  }
  for (int i = 0; i < 2; ++i) sms[i] = 2 * S[i] * tiles[i];
}

cudaError_t launch_ffn(FfnMode mode, const FfnOperand (&a)[2], const FfnOperand (&b)[2], FfnParams p,
                       cudaStream_t st) {
  FfnMaps maps;
  memset(&maps, 0, sizeof(maps));
  // A's rows of a CTA: all of the result's where they are few (in whole eights, as the operand is laid out by)
  if (p.sms == 0) p.sms = device_sm_count();
  p.a_rows = ffn_a_mn(mode) ? 128 : std::min(128, ceil_div(p.M, 8) * 8);
  for (int i = 0; i < 2; ++i) {
    if (!a[i].p) maps.a[i] = maps.a[0];
    else if (!operand_map(&maps.a[i], a[i], ffn_a_mn(mode), p.a_rows)) return cudaErrorInvalidValue;
    if (!b[i].p) maps.b[i] = maps.b[0];
    else if (!operand_map(&maps.b[i], b[i], ffn_b_mn(mode))) return cudaErrorInvalidValue;
  }
  switch (mode) {
    case FFN_GATE: return launch_mode<FFN_GATE>(maps, p, st);
    case FFN_OUT: return launch_mode<FFN_OUT>(maps, p, st);
    case FFN_DA: return launch_mode<FFN_DA>(maps, p, st);
    case FFN_DX: return launch_mode<FFN_DX>(maps, p, st);
    case FFN_DW13: return launch_mode<FFN_DW13>(maps, p, st);
    case FFN_DW2: return launch_mode<FFN_DW2>(maps, p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace mok

// The dense products of the backward pass, bf16 in, fp32 accumulation, bf16
// out, on CTA pairs (tcgen05 kind::f16, cta_group::2).
//
//     D[r, c] = 1 / scale[r] * sum_t A[r, t] * B[t, c]      (scale optional)
//
//   input gradient    dx[m, k] = sum_r dz[m, r] * What[r, k]
//                     A = dz, contraction index contiguous (K-major);
//                     B = What, the expanded weight, c contiguous
//   weight gradient   dw[r, k] = sum_m dz[m, r] * xhat[m, k]
//                     A = dz again, now r contiguous (MN-major);
//                     B = xhat, the expanded 8-bit checkpoint, c contiguous
//
// Neither operand is ever transposed in memory: the MMA reads either major-
// ness from shared memory, so dz is written once and used both ways, and What
// and xhat keep the layout of the weight and the activation.
//
// A tile is 256 x BN (BN 256 or 128) and takes the contraction in stages of
// 64: CTA r of the pair holds rows [128 r, 128 r + 128) of A and columns
// [r BN/2, (r + 1) BN/2) of B, so each SM loads half of both.  K-major
// operands are 128-byte rows of 64 t; MN-major ones 128-byte rows of 64 r (or
// c) per t, as boxes of 64 x 64, both with the 128-byte swizzle.  Two fp32
// accumulators of BN columns in tensor memory: the epilogue of a tile runs
// under the MMAs of the next.
//
// Roles as in sparse_linear_pair.cuh: warps 0-3 produce (TMA), warp 4 of rank
// 0 issues the MMAs, warps 5-12 are the epilogue (two per tensor-memory lane
// quadrant, each taking every other 32-column chunk).
//
// One launch does both products: their tiles are one list of work items for
// the resident CTA pairs (GgWalk), the product with the longer items first and
// the other's filling up what that leaves uneven.  Of 128 + 256 items of 64
// and 32 stages (m = 2048, n = k = 4096) the busiest of 74 pairs gets 224
// stages where two launches take 256.
//
// Few tiles and a long contraction: it is cut into `splits` equal runs of
// stages, every run a work item of its own that writes fp32 partial sums, and
// the join kernel adds the runs in order (no atomics: the same bits every
// time) and rounds.
//
// The prologue kernel expands the operands (and copies or sums dy where that
// is needed), all in one launch of independent blocks.
//
// Rows and columns past the operands' ends are filled with zeros by TMA and
// never stored.  Every wait is bounded (device_common.cuh).
//
// Both products of m = 8192, r = 28672, k = 4096: 2.57 ms, 1.50 PFLOP/s, the
// tensor pipe 98 % busy; of m = 2048, r = k = 4096: 88 us, 1.56 PFLOP/s.  The
// epilogue's last tile is exposed, so its stores count at small sizes: whole
// 32-byte sectors took m = 777, r = 1003, k = 1536 from 17.9 to 15.1 us.  TMA
// fills rows that do not exist more slowly than it loads real ones, so the boxes
// are no higher than the tokens or the contraction: m = 1, r = 16544, k = 1408
// 68 to 41 us.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "device_common.cuh"
#include "sparse24_pack.cuh"

namespace sfp8 {

constexpr int kGgTileM = 256;
constexpr int kGgStageK = 64;
constexpr int kGgLoadWarps = 4;
constexpr int kGgMmaWarp = kGgLoadWarps;
constexpr int kGgEpiWarp0 = kGgMmaWarp + 1;
constexpr int kGgEpiWarps = 8;
constexpr int kGgThreads = 32 * (kGgLoadWarps + 1 + kGgEpiWarps);
constexpr int kGgMaxStages = 12;
constexpr int kGgSmemBudget = 225 * 1024;
constexpr int kGgChunk = 128;     // bytes of a swizzled row: 64 bf16

template <int BN>
struct GgCfg {
  static_assert(BN == 256 || BN == 128, "tile widths");
  static constexpr int kABytes = 128 * kGgStageK * 2;        // 16 KB per CTA
  static constexpr int kBBytes = (BN / 2) * kGgStageK * 2;   // 16 or 8 KB per CTA
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages =
      kGgSmemBudget / kStageBytes < kGgMaxStages ? kGgSmemBudget / kStageBytes : kGgMaxStages;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + 1024;
};

// One of the two products.
struct GgProblem {
  __nv_bfloat16* d;       // [rows][cols]
  float* partial;         // [splits][rows][cols] fp32 (splits > 1)
  const float* row_scale; // [rows], divided out of D's rows; or null
  int rows, cols;         // of D; cols a multiple of 128
  int m_tiles, n_tiles;
  int stages_total;       // ceil(contraction / 64)
  int splits;
  int items;              // m_tiles * n_tiles * splits
  int band;               // row tiles per band of the tile order
  int pair_rows;          // != 0: D's row r is stored at row (r & 1) * pair_rows + r / 2
  int a_mn;               // A is MN-major
  int a_rows;             // rows of a K-major A's boxes: 128, or fewer tokens rounded up to 8
  int t_rows;             // rows of the boxes that run along the contraction: 64, or a
                          // shorter contraction rounded up to 16
  int by_sector;          // D is 32-byte aligned
  uint32_t idesc;
};

struct GgParams {
  GgProblem prob[2];
  int pairs;              // gridDim.x / 2
  int lag_rounds;         // items of product 1 that each less loaded pair takes first
};

struct GgMaps {
  CUtensorMap a[2], b[2];
};

// Instruction descriptor of kind::f16 with bf16 operands and fp32
// accumulation: bits 4-5 D = f32 (1), 7-9 / 10-12 A / B = bf16 (1), bit 15 /
// 16 A / B MN-major, 17-22 N >> 3, 24-28 M >> 4.
__host__ __device__ constexpr uint32_t make_idesc_bf16(bool a_mn, bool b_mn, uint32_t mma_m,
                                                       uint32_t mma_n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (((mma_n >> 3) & 0x3Fu) << 17) | (((mma_m >> 4) & 0x1Fu) << 24);
}

__device__ __forceinline__ void mma_bf16_pair_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 bytes at a 32-byte aligned address: a whole sector in one store.
__device__ __forceinline__ void store_sector(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 2-D form of tma_load_3d_pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* desc, int x, int y,
                                                 uint32_t bar_cluster, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx"
      "::bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(desc), "r"(x), "r"(y), "r"(bar_cluster), "l"(policy)
      : "memory");
}

// The work items of one pair, in order: product 0's items pair, pair + P, ...;
// then, if that gave this pair one item less than others, lag_rounds items of
// product 1; then an even share of product 1's other items.  All roles walk
// it identically.
struct GgWalk {
  int pair, pairs, i, lag, lag_pairs, lag_items, phase;
  __device__ GgWalk(const GgParams& p, int pr) : pair(pr), pairs(p.pairs), i(pr), phase(0) {
    const int q = p.prob[0].items % pairs;
    lag_pairs = q == 0 ? 0 : pairs - q;
    lag = pr - q;                       // its place among the less loaded pairs
    const int most = lag_pairs * p.lag_rounds;
    lag_items = most < p.prob[1].items ? most : p.prob[1].items;
  }
  // The next item: its product and its index there.
  __device__ bool next(const GgParams& p, int& which, int& index) {
    if (phase == 0) {
      if (i < p.prob[0].items) {
        which = 0;
        index = i;
        i += pairs;
        return true;
      }
      phase = lag_pairs > 0 && lag >= 0 ? 1 : 2;
      i = phase == 1 ? lag : lag_items + pair;
    }
    if (phase == 1) {
      if (i < lag_items) {
        which = 1;
        index = i;
        i += lag_pairs;
        return true;
      }
      phase = 2;
      i = lag_items + pair;
    }
    if (i < p.prob[1].items) {
      which = 1;
      index = i;
      i += pairs;
      return true;
    }
    return false;
  }
};

// Item of a product -> (row tile, column tile, split).  Items run in bands of
// `band` row tiles, the split outermost and the row tile fastest, so that the
// items in flight at a time form a block of D about as tall as wide and share
// the operand stages they read through L2.
__device__ __forceinline__ void gg_item(const GgProblem& p, int i, int& mt, int& nt, int& sp) {
  const uint32_t tiles = static_cast<uint32_t>(p.m_tiles * p.n_tiles);
  const uint32_t s = p.splits == 1 ? 0 : static_cast<uint32_t>(i) / tiles;
  const uint32_t t = static_cast<uint32_t>(i) - s * tiles;
  const uint32_t per_band = static_cast<uint32_t>(p.band * p.n_tiles);
  const uint32_t b = t / per_band;
  const uint32_t r = t - b * per_band;
  const uint32_t m0 = b * static_cast<uint32_t>(p.band);
  const uint32_t left = static_cast<uint32_t>(p.m_tiles) - m0;
  const uint32_t bsize = left < static_cast<uint32_t>(p.band) ? left : p.band;
  const uint32_t n = r / bsize;
  sp = static_cast<int>(s);
  nt = static_cast<int>(n);
  mt = static_cast<int>(m0 + (r - n * bsize));
}

// The product stays below 2^31: at most 2^25 stages and 32 splits.
__device__ __forceinline__ int gg_first_stage(const GgProblem& p, int sp) {
  if (p.splits == 1) return sp == 0 ? 0 : p.stages_total;
  return static_cast<int>(static_cast<uint32_t>(p.stages_total) * static_cast<uint32_t>(sp) /
                          static_cast<uint32_t>(p.splits));
}

template <int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGgThreads, 1)
    grad_gemm_kernel(const __grid_constant__ GgMaps maps, const __grid_constant__ GgParams p) {
  using Cfg = GgCfg<BN>;
  constexpr int S = Cfg::kStages;
  constexpr int SB = Cfg::kStageBytes;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* stage_base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(stage_base + S * SB);
  uint64_t* full_bar = bars;                          // [S], used on rank 0
  uint64_t* empty_bar = bars + kGgMaxStages;          // [S]
  uint64_t* accf_bar = bars + 2 * kGgMaxStages;       // [2]
  uint64_t* acce_bar = bars + 2 * kGgMaxStages + 2;   // [2], rank 0
  uint64_t* drain_bar = bars + 2 * kGgMaxStages + 4;  // rank 0
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kGgMaxStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * kGgMaxStages + 6);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x / 2;
  grid_dependents_launch();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&accf_bar[b]), 1);
      mbar_init(smem_u32(&acce_bar[b]), 2 * kGgEpiWarps);
    }
    mbar_init(smem_u32(drain_bar), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    for (int w = 0; w < 2; ++w) {
      if (p.prob[w].items == 0) continue;
      tma_prefetch_desc(&maps.a[w]);
      tma_prefetch_desc(&maps.b[w]);
    }
  }
  if (warp == kGgMmaWarp) {
    tmem_alloc_pair(smem_u32(tmem_slot), 2 * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // Both operands were written by the kernels before this one.
  grid_dependency_wait();

  if (warp < kGgLoadWarps) {
    // ------------------------------------------------------------ producers
    constexpr int P = kGgLoadWarps < S ? kGgLoadWarps : S;
    if (lane == 0 && warp < P) {
      const uint64_t pol = l2_policy_evict_normal();
      long long i = 0;
      bool ok = true;
      GgWalk walk(p, pair);
      int which, index;
      while (ok && walk.next(p, which, index)) {
        const GgProblem& pr = p.prob[which];
        int mt, nt, sp;
        gg_item(pr, index, mt, nt, sp);
        const int s1 = gg_first_stage(pr, sp + 1);
        const int tile0 = mt * kGgTileM;
        const int m0 = tile0 + static_cast<int>(rank) * 128;
        const int n0 = nt * BN + static_cast<int>(rank) * (BN / 2);
        const CUtensorMap* ta = &maps.a[which];
        const CUtensorMap* tb = &maps.b[which];
        // boxes of this CTA's A (a K-major one past the last row is left out:
        // what D's rows there become is not stored); the pair's bytes a stage
        const bool a_mn = pr.a_mn != 0;
        const bool load_a = a_mn || m0 < pr.rows;
        const uint32_t t_bytes = pr.t_rows * kGgChunk;
        const uint32_t stage_bytes =
            BN / 64 * t_bytes +
            (a_mn ? 4 * t_bytes : (tile0 + 128 < pr.rows ? 2u : 1u) * pr.a_rows * kGgChunk);
        for (int u = gg_first_stage(pr, sp); u < s1; ++u, ++i) {
          if (i % P != warp) continue;
          const int stage = static_cast<int>(i % S);
          if (i >= S &&
              !mbar_wait(smem_u32(&empty_bar[stage]),
                         static_cast<uint32_t>((i / S) & 1) ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full_bar[stage]), stage_bytes);
          const uint32_t full = map_to_cta(smem_u32(&full_bar[stage]), 0);
          const uint32_t a_dst = smem_u32(stage_base + stage * SB);
          const uint32_t b_dst = a_dst + Cfg::kABytes;
          const int t0 = u * kGgStageK;
          if (a_mn) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load_2d_pair(a_dst + h * kGgStageK * kGgChunk, ta, m0 + 64 * h, t0, full, pol);
          } else if (load_a) {
            tma_load_2d_pair(a_dst, ta, t0, m0, full, pol);
          }
#pragma unroll
          for (int h = 0; h < BN / 128; ++h)
            tma_load_2d_pair(b_dst + h * kGgStageK * kGgChunk, tb, n0 + 64 * h, t0, full, pol);
        }
      }
      if (!ok && rank == 0) {
        // Let the stages this lane armed complete before the pair exits.
        const long long issued = i;
        for (long long t = issued > S ? issued - S : 0; t < issued; ++t) {
          if (t % P != warp) continue;
          volatile int no_abort = 0;
          mbar_wait(smem_u32(&full_bar[t % S]), static_cast<uint32_t>((t / S) & 1), &no_abort);
        }
      }
    }
  } else if (warp == kGgMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      bool ready = false;   // the next stage's barrier already seen complete
      GgWalk walk(p, pair);
      int which, index;
      while (ok && walk.next(p, which, index)) {
        const GgProblem& pr = p.prob[which];
        const int sp = pr.splits == 1 ? 0 : index / (pr.m_tiles * pr.n_tiles);
        const int count = gg_first_stage(pr, sp + 1) - gg_first_stage(pr, sp);
        const uint32_t idesc = pr.idesc;
        const int steps = pr.t_rows / 16;
        // K-major: 8-row groups 1024 bytes apart, 16 t = 32 bytes on.
        // MN-major: 64-wide chunks kGgStageK rows apart (leading offset),
        // groups of 8 t 1024 bytes apart, 16 t = two groups on.
        const uint32_t a_lbo = pr.a_mn ? kGgStageK * kGgChunk : 16;
        const uint32_t a_step = pr.a_mn ? 2048 : 32;
        if (!mbar_wait_cluster_warp(smem_u32(&acce_bar[acc]), acc_phase ^ 1u, abort_flag)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        // One stage's products: all four 16-wide steps along the contraction, or `steps`.
        auto take_stage = [&](auto whole, bool first) {
          if (!ready && !mbar_wait_warp(smem_u32(&full_bar[stage]), phase, abort_flag)) return false;
          tc_fence_after();
          const int next_stage = stage + 1 == S ? 0 : stage + 1;
          const uint32_t next_phase = stage + 1 == S ? phase ^ 1u : phase;
          const uint32_t a_addr = smem_u32(stage_base + stage * SB);
          const uint32_t b_addr = a_addr + Cfg::kABytes;
          const int n = decltype(whole)::value ? kGgStageK / 16 : steps;
#pragma unroll
          for (int j = 0; j < n; ++j) {
            const uint64_t adesc = smem_desc(a_addr + j * a_step, a_lbo, 1024, kSwizzle128);
            const uint64_t bdesc =
                smem_desc(b_addr + j * 2048, kGgStageK * kGgChunk, 1024, kSwizzle128);
            mma_bf16_pair_w(d_tmem, adesc, bdesc, idesc, (!first || j > 0) ? 1u : 0u);
            if (j == 0) ready = mbar_test_warp(smem_u32(&full_bar[next_stage]), next_phase);
          }
          tc_commit_pair_mc_w(smem_u32(&empty_bar[stage]), 0x3);
          stage = next_stage;
          phase = next_phase;
          return true;
        };
        if (steps == kGgStageK / 16) {
          for (int u = 0; ok && u < count; ++u) ok = take_stage(std::true_type{}, u == 0);
        } else {
          ok = take_stage(std::false_type{}, true);   // a contraction below one stage
        }
        if (!ok) break;
        tc_commit_pair_mc_w(smem_u32(&accf_bar[acc]), 0x3);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      tc_commit_pair_mc_w(smem_u32(drain_bar), 0x1);
      volatile int no_abort = 0;
      mbar_wait_warp(smem_u32(drain_bar), 0, &no_abort);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int e = warp - kGgEpiWarp0;
    const int q = warp % 4;      // tensor-memory lane quadrant
    const int half = e / 4;      // 32-column chunks half, half + 2, ...
    uint32_t acce_leader[2];
    for (int b = 0; b < 2; ++b) acce_leader[b] = map_to_cta(smem_u32(&acce_bar[b]), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    GgWalk walk(p, pair);
    int which, index;
    while (walk.next(p, which, index)) {
      const GgProblem& pr = p.prob[which];
      int mt, nt, sp;
      gg_item(pr, index, mt, nt, sp);
      const int r = mt * kGgTileM + static_cast<int>(rank) * 128 + q * 32 + lane;
      const float rs =
          pr.row_scale != nullptr && r < pr.rows ? 1.0f / __ldg(pr.row_scale + r) : 1.0f;
      int ok = 1;
      if (lane == 0) ok = mbar_wait(smem_u32(&accf_bar[acc]), acc_phase, abort_flag) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_row =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);
      long long out_row = r;
      if (pr.pair_rows != 0) out_row = (r & 1) ? pr.pair_rows + (r >> 1) : (r >> 1);
#pragma unroll 1
      for (int c = half; c < BN / 32; c += 2) {
        uint32_t v[2][16];
        tmem_ld_32x32b_x16(t_row + c * 32, v[0]);
        tmem_ld_32x32b_x16(t_row + c * 32 + 16, v[1]);
        tmem_ld_wait();
        const int c0 = nt * BN + c * 32;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col = c0 + 16 * h;
          if (r >= pr.rows || col >= pr.cols) continue;
          if (pr.splits > 1) {
            float* dst = pr.partial +
                         (static_cast<long long>(sp) * pr.rows + r) * pr.cols + col;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = v[h][8 * j + i];
              store_sector(dst + 8 * j, w);
            }
          } else {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(
                  __uint_as_float(v[h][2 * j]) * rs, __uint_as_float(v[h][2 * j + 1]) * rs);
              w[j] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            __nv_bfloat16* dst = pr.d + out_row * pr.cols + col;
            if (pr.by_sector) {
              store_sector(dst, w);
            } else {
              *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acce_leader[acc]);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == kGgMmaWarp) tmem_dealloc_pair(tmem_base, 2 * BN);
}

// ------------------------------------------------------------------ join

struct JoinParams {
  GgProblem prob[2];      // those with splits > 1 are joined
  int blocks[2];          // blocks of each
  const float* sums;      // [runs][cols] column sums, or null
  __nv_bfloat16* dbias;
  int runs, cols;
  int pair_rows;          // as in GgProblem, for the columns
};

// D = the sum of the splits' partial sums, in split order, scaled and rounded
// once (one thread per 8 columns; D's columns are a multiple of 128); then, in
// blocks of their own, the bias gradient: 32 columns a block, each of 8 row
// lanes adding every eighth run, the lanes added in order.
__global__ void __launch_bounds__(256) backward_join_kernel(const __grid_constant__ JoinParams p) {
  grid_dependents_launch();
  grid_dependency_wait();
  int block = blockIdx.x;
  for (int w = 0; w < 2; ++w) {
    if (block >= p.blocks[w]) {
      block -= p.blocks[w];
      continue;
    }
    const GgProblem& pr = p.prob[w];
    const long long plane = static_cast<long long>(pr.rows) * pr.cols;
    // 16 rows x 128 columns a block and step
    const int chunks = pr.cols / 128;
    const int units = (pr.rows + 15) / 16 * chunks;
    for (int u = block; u < units; u += p.blocks[w]) {
      const long long r = static_cast<long long>(u / chunks) * 16 + threadIdx.x / 16;
      const int c = u % chunks * 128 + threadIdx.x % 16 * 8;
      if (r >= pr.rows) continue;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      const float* src = pr.partial + r * pr.cols + c;
#pragma unroll 4
      for (int sp = 0; sp < pr.splits; ++sp) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(src + sp * plane));
        const float4 b = __ldcs(reinterpret_cast<const float4*>(src + sp * plane + 4));
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
      }
      const float rs = pr.row_scale != nullptr ? 1.0f / pr.row_scale[r] : 1.0f;
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * j] * rs, v[2 * j + 1] * rs);
        o[j] = *reinterpret_cast<const uint32_t*>(&b2);
      }
      long long row = r;
      if (pr.pair_rows != 0) row = (r & 1) ? pr.pair_rows + (r >> 1) : (r >> 1);
      *reinterpret_cast<uint4*>(pr.d + row * pr.cols + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    return;
  }
  __shared__ float lanes[8][32];
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  const long long c = static_cast<long long>(block) * 32 + tx;
  float s = 0.0f;
  if (c < p.cols) {
#pragma unroll 8
    for (int y = ty; y < p.runs; y += 8) s += p.sums[static_cast<long long>(y) * p.cols + c];
  }
  lanes[ty][tx] = s;
  __syncthreads();
  if (ty != 0 || c >= p.cols) return;
  for (int j = 1; j < 8; ++j) s += lanes[j][tx];
  long long at = c;
  if (p.pair_rows != 0) at = (c & 1) ? p.pair_rows + (c >> 1) : (c >> 1);
  p.dbias[at] = __float2bfloat16_rn(s);
}

// ------------------------------------------------------------------ prologue

// What the gradient products read, made in one launch; each part has blocks of
// its own (0: not needed).
struct PrologueParams {
  int blocks[4];
  // 0: the expanded weight
  const uint8_t* packed;
  const float* s_w;             // or null
  int w_fmt;
  long long rows, k;
  __nv_bfloat16* what;
  // 1: the expanded checkpoint
  const uint8_t* a_q;
  const float* s_a;             // or null
  int a_fmt;
  long long m;
  __nv_bfloat16* xhat;
  // 2: dy [m][ld_dy] copied to rows of ld_copy
  const __nv_bfloat16* dy;
  long long ld_dy;
  __nv_bfloat16* copy;
  long long ld_copy;
  int copy_shift;               // log2 of the threads that copy a row
  // 3: column sums of dy over runs of rows
  float* sums;                  // [runs][rows]
  int runs, sums_by_16;         // sums_by_16: dy's rows may be read 16 bytes at a time
};

// Two FP8 codes -> two floats (exact), first from the low byte.
__device__ __forceinline__ float2 fp8_pair_to_float(uint32_t codes, int fmt) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(codes), fmt == SFP8_E5M2 ? __NV_E5M2 : __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b2 = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b2);
}

// Rows of the pieces that the expanding blocks take: half a packed tile, so
// that medium sizes spread evenly over the device.
constexpr int kExpandRows = 64;

// What[r, k] = bf16(dec(W_q[r, k]) * s_w[r]), dense, half a 128 x 128 tile of
// the packed weight at a time: every thread takes pieces of 16 k (8 kept codes,
// 4 index nibbles), neighbouring threads neighbouring words of the tile and
// neighbouring 32-byte sectors of a row.  With s_w the one rounding (half a
// bf16 step) is that of the operand; without it (null: the scales are in dz)
// the codes are exact in bf16.
__device__ __forceinline__ void expand_weight(const PrologueParams& p, int block) {
  const int ktiles = static_cast<int>(p.k / 128);
  const int units = static_cast<int>((p.rows + kExpandRows - 1) / kExpandRows) * ktiles;
  for (int u = block; u < units; u += p.blocks[0]) {
    const int half = u / ktiles, kt = u - half * ktiles;   // 64-row group, k tile
    const uint8_t* tile = p.packed + (static_cast<long long>(half / 2) * ktiles + kt) * 10240;
    const long long tile0 = half / 2 * 128ll;
    __nv_bfloat16* out = p.what + tile0 * p.k + kt * 128ll;
#pragma unroll
    for (int i = 0; i < kExpandRows / 32; ++i) {
      const int item = i * 256 + threadIdx.x;
      const int r = half % 2 * kExpandRows + item / 8, j = item % 8;   // piece of 16 k
      if (tile0 + r >= p.rows) continue;
      const uint2 vals = __ldg(reinterpret_cast<const uint2*>(
          tile + 64 * r + (((j / 2) ^ (r >> 1 & 3)) * 16) + (j % 2) * 8));
      const uint32_t meta = __ldg(reinterpret_cast<const uint16_t*>(tile + 8192 + 16 * r + 2 * j));
      const float s = p.s_w != nullptr ? __ldg(p.s_w + tile0 + r) : 1.0f;
      uint32_t w[8];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float2 f = fp8_pair_to_float(((g < 2 ? vals.x : vals.y) >> (16 * (g % 2))) & 0xFFFFu,
                                           p.w_fmt);
        const uint32_t bits = bf16_pair(f.x * s, f.y * s);
        const uint32_t nib = (meta >> (4 * g)) & 0xFu;
        // the group's four bf16 as one 64-bit word
        const unsigned long long word =
            (static_cast<unsigned long long>(bits & 0xFFFFu) << (16 * (nib & 3u))) |
            (static_cast<unsigned long long>(bits >> 16) << (16 * (nib >> 2)));
        w[2 * g] = static_cast<uint32_t>(word);
        w[2 * g + 1] = static_cast<uint32_t>(word >> 32);
      }
      store_sector(out + r * p.k + 16 * j, w);
    }
  }
}

// xhat[m, k] = bf16(dec(A_q[m, k]) * s_a[m]), or with s_a null the codes' own
// values, 64 x 128 at a time as above.
__device__ __forceinline__ void expand_rows(const PrologueParams& p, int block) {
  const int ktiles = static_cast<int>(p.k / 128);
  const int units = static_cast<int>((p.m + kExpandRows - 1) / kExpandRows) * ktiles;
  for (int u = block; u < units; u += p.blocks[1]) {
    const int mt = u / ktiles;
    const long long row0 = static_cast<long long>(mt) * kExpandRows;
    const long long at = row0 * p.k + (u - mt * ktiles) * 128ll;
#pragma unroll
    for (int i = 0; i < kExpandRows / 32; ++i) {
      const int item = i * 256 + threadIdx.x;
      const int r = item / 8, j = item % 8;
      if (row0 + r >= p.m) continue;
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.a_q + at + r * p.k + 16 * j));
      const float s = p.s_a != nullptr ? __ldg(p.s_a + row0 + r) : 1.0f;
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
      uint32_t w[8];
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const float2 f = fp8_pair_to_float((in[h / 2] >> (16 * (h % 2))) & 0xFFFFu, p.a_fmt);
        w[h] = bf16_pair(f.x * s, f.y * s);
      }
      store_sector(p.xhat + at + r * p.k + 16 * j, w);
    }
  }
}

// dy to rows of ld_copy elements (a multiple of 8), for a dy whose base or
// row stride TMA cannot take; zeros past its columns.  8 elements a thread, a
// row (or 2048 columns of one) by 1 << copy_shift threads.
__device__ __forceinline__ void copy_dy(const PrologueParams& p, int block) {
  const int width = 1 << p.copy_shift, per_step = 256 >> p.copy_shift;
  const int tx = threadIdx.x & (width - 1), ty = threadIdx.x >> p.copy_shift;
  for (long long r = static_cast<long long>(block) * per_step + ty; r < p.m;
       r += static_cast<long long>(p.blocks[2]) * per_step) {
    const unsigned short* src = reinterpret_cast<const unsigned short*>(p.dy) + r * p.ld_dy;
    for (long long c = tx * 8; c < p.ld_copy; c += width * 8) {
      uint32_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + j < p.rows ? __ldg(src + c + j) : 0u;
      *reinterpret_cast<uint4*>(p.copy + r * p.ld_copy + c) =
          make_uint4(v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16),
                     v[6] | (v[7] << 16));
    }
  }
}

// Column sums of dy, in fp32: block (x, y) adds the rows of its run y for 256
// columns, 8 row lanes of 32 threads with 8 columns each.
constexpr int kColSumCols = 256;
__device__ __forceinline__ void sum_columns(const PrologueParams& p, int block,
                                            float (*lanes)[kColSumCols]) {
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  const long long c0 = static_cast<long long>(block / p.runs) * kColSumCols;
  const int run = block % p.runs;
  const long long r0 = p.m * run / p.runs, r1 = p.m * (run + 1) / p.runs;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  // 16-byte reads: 8 neighbouring columns; else every 32nd
  const bool vec = p.sums_by_16 && c0 + 8 * tx + 8 <= p.rows;
  if (vec) {
    const __nv_bfloat16* src = p.dy + c0 + 8 * tx;
#pragma unroll 4
    for (long long r = r0 + ty; r < r1; r += 8) {
      float f[8];
      InputTraits<__nv_bfloat16>::to_float(
          __ldg(reinterpret_cast<const uint4*>(src + r * p.ld_dy)), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += f[j];
    }
  } else {
    const int step = p.sums_by_16 ? 1 : 32;
    const long long first = c0 + (p.sums_by_16 ? 8 * tx : tx);
    for (long long r = r0 + ty; r < r1; r += 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (first + j * step < p.rows)
          s[j] += __bfloat162float(p.dy[r * p.ld_dy + first + j * step]);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) lanes[ty][p.sums_by_16 ? 8 * tx + j : tx + 32 * j] = s[j];
  __syncthreads();
  const long long c = c0 + threadIdx.x;
  if (c < p.rows) {
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) t += lanes[j][threadIdx.x];
    p.sums[run * p.rows + c] = t;
  }
}

__global__ void __launch_bounds__(256)
    backward_prologue_kernel(const __grid_constant__ PrologueParams p) {
  // only a launch that sums columns asks for the shared memory: without it,
  // the gradient GEMM's blocks can be resident before this grid has drained
  extern __shared__ __align__(16) float column_lanes[];
  grid_dependents_launch();
  grid_dependency_wait();
  int block = blockIdx.x;
  int part = 0;
  while (block >= p.blocks[part]) block -= p.blocks[part++];
  if (part == 0) expand_weight(p, block);
  else if (part == 1) expand_rows(p, block);
  else if (part == 2) copy_dy(p, block);
  else sum_columns(p, block, reinterpret_cast<float(*)[kColSumCols]>(column_lanes));
}

}  // namespace sfp8

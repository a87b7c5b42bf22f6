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
// Few tiles and a long contraction: it is cut into `splits` equal runs of
// stages, every run a work item of its own that writes fp32 partial sums, and
// a second kernel adds the runs in order (no atomics: the same bits every
// time) and rounds.
//
// Rows and columns past the operands' ends are filled with zeros by TMA and
// never stored.  Every wait is bounded (device_common.cuh).
#pragma once

#include <cuda_bf16.h>

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

struct GgParams {
  __nv_bfloat16* d;       // [rows][ld_d]
  float* partial;         // [splits][rows][cols] fp32 (splits > 1)
  long long ld_d;
  int rows, cols;         // of D; cols a multiple of 16
  int m_tiles, n_tiles;
  int stages_total;       // ceil(contraction / 64)
  int splits;
  int items;              // m_tiles * n_tiles * splits
  int pairs;              // gridDim.x / 2
  int band;               // row tiles per band of the tile order
  const float* row_scale; // [rows], divided out of D's rows; or null
  int pair_rows;          // != 0: D's row r is stored at row (r & 1) * pair_rows + r / 2
  uint32_t idesc;
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

// 2-D form of tma_load_3d_pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* desc, int x, int y,
                                                 uint32_t bar_cluster, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx"
      "::bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(desc), "r"(x), "r"(y), "r"(bar_cluster), "l"(policy)
      : "memory");
}

// Work item -> (row tile, column tile, split).  Items run in bands of
// p.band row tiles, the split outermost and the row tile fastest, so that
// the items in flight at a time form a block of D about as tall as wide and
// share the operand stages they read through L2.
__device__ __forceinline__ void gg_item(const GgParams& p, int i, int& mt, int& nt, int& sp) {
  const int tiles = p.m_tiles * p.n_tiles;
  sp = i / tiles;
  const int t = i - sp * tiles;
  const int per_band = p.band * p.n_tiles;
  const int b = t / per_band;
  const int r = t - b * per_band;
  const int m0 = b * p.band;
  const int bsize = p.m_tiles - m0 < p.band ? p.m_tiles - m0 : p.band;
  nt = r / bsize;
  mt = m0 + (r - nt * bsize);
}

__device__ __forceinline__ int gg_first_stage(const GgParams& p, int sp) {
  return static_cast<int>(static_cast<long long>(p.stages_total) * sp / p.splits);
}

template <int BN, bool A_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGgThreads, 1)
    grad_gemm_kernel(const __grid_constant__ CUtensorMap tm_a,
                     const __grid_constant__ CUtensorMap tm_b, const GgParams p) {
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
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
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
      for (int it = pair; ok && it < p.items; it += p.pairs) {
        int mt, nt, sp;
        gg_item(p, it, mt, nt, sp);
        const int s1 = gg_first_stage(p, sp + 1);
        for (int u = gg_first_stage(p, sp); u < s1; ++u, ++i) {
          if (i % P != warp) continue;
          const int stage = static_cast<int>(i % S);
          if (i >= S &&
              !mbar_wait(smem_u32(&empty_bar[stage]),
                         static_cast<uint32_t>((i / S) & 1) ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full_bar[stage]), 2 * SB);
          const uint32_t full = map_to_cta(smem_u32(&full_bar[stage]), 0);
          const uint32_t a_dst = smem_u32(stage_base + stage * SB);
          const uint32_t b_dst = a_dst + Cfg::kABytes;
          const int m0 = mt * kGgTileM + static_cast<int>(rank) * 128;
          const int n0 = nt * BN + static_cast<int>(rank) * (BN / 2);
          const int t0 = u * kGgStageK;
          if (A_MN) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load_2d_pair(a_dst + h * kGgStageK * kGgChunk, &tm_a, m0 + 64 * h, t0, full, pol);
          } else {
            tma_load_2d_pair(a_dst, &tm_a, t0, m0, full, pol);
          }
#pragma unroll
          for (int h = 0; h < BN / 128; ++h)
            tma_load_2d_pair(b_dst + h * kGgStageK * kGgChunk, &tm_b, n0 + 64 * h, t0, full, pol);
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
      for (int it = pair; ok && it < p.items; it += p.pairs) {
        int mt, nt, sp;
        gg_item(p, it, mt, nt, sp);
        const int count = gg_first_stage(p, sp + 1) - gg_first_stage(p, sp);
        if (!mbar_wait_cluster_warp(smem_u32(&acce_bar[acc]), acc_phase ^ 1u, abort_flag)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int u = 0; u < count; ++u) {
          if (!ready && !mbar_wait_warp(smem_u32(&full_bar[stage]), phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int next_stage = stage + 1 == S ? 0 : stage + 1;
          const uint32_t next_phase = stage + 1 == S ? phase ^ 1u : phase;
          const uint32_t a_addr = smem_u32(stage_base + stage * SB);
          const uint32_t b_addr = a_addr + Cfg::kABytes;
#pragma unroll
          for (int j = 0; j < kGgStageK / 16; ++j) {
            // K-major: 8-row groups 1024 bytes apart, 16 t = 32 bytes on.
            // MN-major: 64-wide chunks kGgStageK rows apart (leading offset),
            // groups of 8 t 1024 bytes apart, 16 t = two groups on.
            const uint64_t adesc =
                A_MN ? smem_desc(a_addr + j * 2048, kGgStageK * kGgChunk, 1024, kSwizzle128)
                     : smem_desc(a_addr + j * 32, 16, 1024, kSwizzle128);
            const uint64_t bdesc =
                smem_desc(b_addr + j * 2048, kGgStageK * kGgChunk, 1024, kSwizzle128);
            mma_bf16_pair_w(d_tmem, adesc, bdesc, p.idesc, (u > 0 || j > 0) ? 1u : 0u);
            if (j == 0) ready = mbar_test_warp(smem_u32(&full_bar[next_stage]), next_phase);
          }
          tc_commit_pair_mc_w(smem_u32(&empty_bar[stage]), 0x3);
          stage = next_stage;
          phase = next_phase;
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
    for (int it = pair; it < p.items; it += p.pairs) {
      int mt, nt, sp;
      gg_item(p, it, mt, nt, sp);
      const int r = mt * kGgTileM + static_cast<int>(rank) * 128 + q * 32 + lane;
      const float rs = p.row_scale != nullptr && r < p.rows ? 1.0f / __ldg(p.row_scale + r) : 1.0f;
      int ok = 1;
      if (lane == 0) ok = mbar_wait(smem_u32(&accf_bar[acc]), acc_phase, abort_flag) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_row =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);
      long long out_row = r;
      if (p.pair_rows != 0) out_row = (r & 1) ? p.pair_rows + (r >> 1) : (r >> 1);
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
          if (r >= p.rows || col >= p.cols) continue;
          if (p.splits > 1) {
            float* dst = p.partial +
                         (static_cast<long long>(sp) * p.rows + r) * static_cast<long long>(p.cols) +
                         col;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(dst + 4 * j) =
                  make_uint4(v[h][4 * j], v[h][4 * j + 1], v[h][4 * j + 2], v[h][4 * j + 3]);
          } else {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(
                  __uint_as_float(v[h][2 * j]) * rs, __uint_as_float(v[h][2 * j + 1]) * rs);
              w[j] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            __nv_bfloat16* dst = p.d + out_row * p.ld_d + col;
            *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
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

// D = the sum of the splits' partial sums, in split order, scaled and rounded
// once.
// One thread per 8 columns.
__global__ void __launch_bounds__(256)
    grad_gemm_join_kernel(const float* __restrict__ partial, int splits, int rows, int cols,
                          const float* __restrict__ row_scale, __nv_bfloat16* __restrict__ d,
                          long long ld_d, int pair_rows) {
  grid_dependents_launch();
  grid_dependency_wait();
  const long long vecs = static_cast<long long>(rows) * (cols / 8);
  const long long plane = static_cast<long long>(rows) * cols;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < vecs;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const long long r = i / (cols / 8);
    const int c = static_cast<int>(i - r * (cols / 8)) * 8;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const float* src = partial + r * cols + c;
    for (int sp = 0; sp < splits; ++sp, src += plane) {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(src));
      const float4 b = __ldcs(reinterpret_cast<const float4*>(src + 4));
      s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
      s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
    }
    const float rs = row_scale != nullptr ? 1.0f / row_scale[r] : 1.0f;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(s[2 * j] * rs, s[2 * j + 1] * rs);
      w[j] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    long long row = r;
    if (pair_rows != 0) row = (r & 1) ? pair_rows + (r >> 1) : (r >> 1);
    *reinterpret_cast<uint4*>(d + row * ld_d + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ------------------------------------------------------------------ operands

// Two FP8 codes -> two floats (exact), first from the low byte.
template <int kFmt>
__device__ __forceinline__ float2 fp8_pair_to_float(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes),
                                                   Fp8Out<kFmt>::kInterp);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The expanded weight What[r, k] = bf16(dec(W_q[r, k]) * s_w[r]), dense: one
// thread per 32 k of a row (16 kept codes, 8 index nibbles), reading the
// packed tile and writing 64 contiguous bytes.  With s_w the one rounding
// (half a bf16 step) is that of the operand; without it (null: the scales are
// in dz) the codes are exact in bf16.  What has the weight's true rows only
// (padding rows are not written).
template <int kFmt>
__global__ void __launch_bounds__(256)
    expand_weight_kernel(const uint8_t* __restrict__ packed, const float* __restrict__ s_w,
                         long long rows, long long k, __nv_bfloat16* __restrict__ out) {
  grid_dependents_launch();
  grid_dependency_wait();
  const long long chunks = k / 32;
  const long long ktiles = k / 128;
  const long long total = rows * chunks;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const long long row = i / chunks;
    const long long c = i - row * chunks;
    const int r = static_cast<int>(row % 128);
    const int j = static_cast<int>(c % 4);
    const uint8_t* tile = packed + ((row / 128) * ktiles + c / 4) * 10240;
    const uint4 v = __ldg(
        reinterpret_cast<const uint4*>(tile + 64 * r + (16 * j ^ (16 * (r >> 1 & 3)))));
    const uint32_t meta = __ldg(reinterpret_cast<const uint32_t*>(tile + 8192 + 16 * r + 4 * j));
    const float s = s_w != nullptr ? __ldg(s_w + row) : 1.0f;
    const uint32_t vals[4] = {v.x, v.y, v.z, v.w};
    uint32_t w[16];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const float2 f = fp8_pair_to_float<kFmt>((vals[g / 2] >> (16 * (g % 2))) & 0xFFFFu);
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(f.x * s, f.y * s);
      const uint32_t bits = *reinterpret_cast<const uint32_t*>(&b2);
      const uint32_t nib = (meta >> (4 * g)) & 0xFu;
      // the group's four bf16 as one 64-bit word
      const unsigned long long word =
          (static_cast<unsigned long long>(bits & 0xFFFFu) << (16 * (nib & 3u))) |
          (static_cast<unsigned long long>(bits >> 16) << (16 * (nib >> 2)));
      w[2 * g] = static_cast<uint32_t>(word);
      w[2 * g + 1] = static_cast<uint32_t>(word >> 32);
    }
    uint4* dst = reinterpret_cast<uint4*>(out + row * k + c * 32);
#pragma unroll
    for (int t = 0; t < 4; ++t)
      dst[t] = make_uint4(w[4 * t], w[4 * t + 1], w[4 * t + 2], w[4 * t + 3]);
  }
}

// The expanded checkpoint xhat[m, k] = bf16(dec(A_q[m, k]) * s_a[m]), or with
// s null the codes' own values: one thread per 16 codes.
template <int kFmt>
__global__ void __launch_bounds__(256)
    expand_rows_kernel(const uint8_t* __restrict__ q, const float* __restrict__ s, long long rows,
                       long long cols, __nv_bfloat16* __restrict__ out) {
  grid_dependents_launch();
  grid_dependency_wait();
  const long long per_row = cols / 16;
  const long long total = rows * per_row;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(q) + i);
    const float sc = s != nullptr ? __ldg(s + i / per_row) : 1.0f;
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = fp8_pair_to_float<kFmt>((in[j / 2] >> (16 * (j % 2))) & 0xFFFFu);
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(f.x * sc, f.y * sc);
      w[j] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    uint4* dst = reinterpret_cast<uint4*>(out) + 2 * i;
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// dy [m][ld] -> out [m][ld_out] (ld_out >= cols, columns past cols zero), for
// a dy whose base or row stride TMA cannot take.  One thread per element.
__global__ void __launch_bounds__(256)
    copy_rows_kernel(const __nv_bfloat16* __restrict__ in, long long rows, long long cols,
                     long long ld, __nv_bfloat16* __restrict__ out, long long ld_out) {
  grid_dependents_launch();
  grid_dependency_wait();
  const long long total = rows * ld_out;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const long long r = i / ld_out;
    const long long c = i - r * ld_out;
    out[i] = c < cols ? in[r * ld + c] : __float2bfloat16_rn(0.0f);
  }
}

// Column sums of dz [rows][ld] for the bias gradient, in fp32, in two steps:
// block (x, y) adds the rows of its run y for 64 columns (8 row lanes x 32
// column pairs) into partial[y][cols]; the second kernel adds the runs in
// order and rounds once.  row_scale and col_scale, where given, are divided
// out (a gated block's dz holds both).
constexpr int kColSumCols = 64;
__global__ void __launch_bounds__(256)
    column_sums_kernel(const __nv_bfloat16* __restrict__ dz, long long rows, long long cols,
                       long long ld, const float* __restrict__ row_scale,
                       float* __restrict__ partial) {
  grid_dependents_launch();
  grid_dependency_wait();
  __shared__ float2 sums[8][32];
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const long long col = static_cast<long long>(blockIdx.x) * kColSumCols + 2 * x;
  const long long r0 = rows * blockIdx.y / gridDim.y, r1 = rows * (blockIdx.y + 1) / gridDim.y;
  float2 s = make_float2(0.0f, 0.0f);
  if (col + 1 < cols && ld % 2 == 0 && (reinterpret_cast<uintptr_t>(dz) & 3u) == 0) {
#pragma unroll 4
    for (long long r = r0 + y; r < r1; r += 8) {
      const float2 v =
          __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(dz + r * ld + col));
      const float rs = row_scale != nullptr ? 1.0f / row_scale[r] : 1.0f;
      s.x = fmaf(v.x, rs, s.x);
      s.y = fmaf(v.y, rs, s.y);
    }
  } else if (col < cols) {
    for (long long r = r0 + y; r < r1; r += 8) {
      const float rs = row_scale != nullptr ? 1.0f / row_scale[r] : 1.0f;
      s.x = fmaf(__bfloat162float(dz[r * ld + col]), rs, s.x);
      if (col + 1 < cols) s.y = fmaf(__bfloat162float(dz[r * ld + col + 1]), rs, s.y);
    }
  }
  sums[y][x] = s;
  __syncthreads();
  if (y == 0 && col < cols) {
    for (int j = 1; j < 8; ++j) {
      s.x += sums[j][x].x;
      s.y += sums[j][x].y;
    }
    float* dst = partial + static_cast<long long>(blockIdx.y) * cols + col;
    dst[0] = s.x;
    if (col + 1 < cols) dst[1] = s.y;
  }
}

// out[c] = the runs' sums added in order; with pair_rows, column c goes to
// (c & 1) * pair_rows + c / 2 (a gated block's gate and up values).
__global__ void __launch_bounds__(256)
    column_sums_join_kernel(const float* __restrict__ partial, int runs, long long cols,
                            const float* __restrict__ col_scale, __nv_bfloat16* __restrict__ out, long long pair_rows) {
  grid_dependents_launch();
  grid_dependency_wait();
  const long long c = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (c >= cols) return;
  float s = 0.0f;
  for (int y = 0; y < runs; ++y) s += partial[y * cols + c];
  if (col_scale != nullptr) s /= col_scale[c];
  long long at = c;
  if (pair_rows != 0) at = (c & 1) ? pair_rows + (c >> 1) : (c >> 1);
  out[at] = __float2bfloat16_rn(s);
}

}  // namespace sfp8

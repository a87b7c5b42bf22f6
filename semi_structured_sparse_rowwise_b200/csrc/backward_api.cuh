// C-ABI entry points of the backward passes (declared in include/sfp8.h):
// validation, workspace layout, work splits and launches of the gradient
// GEMM (grad_gemm.cuh) and of the gated block's gradient epilogue
// (sparse_linear_pair.cuh).  Part of the library's one translation unit,
// included at its end.
#pragma once

namespace sfp8 {
namespace {

// ------------------------------------------------------------------ gradient GEMM plan

// One product's split into work items.
struct GradPlan {
  int splits;
  int m_tiles, n_tiles;
  int stages;             // of 64 along the contraction
  int items;
  size_t partial_bytes;   // fp32 partial sums (splits > 1)
};

struct GradPlans {
  int bn;                 // tile width of both
  int first;              // which product's items come first (the longer ones)
  int lag_rounds;         // see GgWalk
  GradPlan p[2];          // dx, dw
};

constexpr int kGradMinStages = 8;   // an item's epilogue takes about as long as 8 stages

GradPlan grad_split(int64_t rows, int64_t cols, int64_t contraction, int bn, int splits) {
  GradPlan g{};
  g.splits = splits;
  g.m_tiles = static_cast<int>((rows + kGgTileM - 1) / kGgTileM);
  g.n_tiles = static_cast<int>((cols + bn - 1) / bn);
  g.stages = static_cast<int>((contraction + kGgStageK - 1) / kGgStageK);
  g.items = g.m_tiles * g.n_tiles * splits;
  g.partial_bytes = splits > 1 ? static_cast<size_t>(splits) * static_cast<size_t>(rows) *
                                     static_cast<size_t>(cols) * sizeof(float)
                               : 0;
  return g;
}

// Tile width and splits that finish first by this estimate, in units of one
// 64-deep stage of a 256-wide tile (about 0.3 us): the busiest pair's stages
// by GgWalk's order (a 128-wide tile's stage costs 0.65 of a 256-wide one's,
// not half, since A's share of the loads stays), plus, where a contraction is
// split, a launch (8) and the round trip of the partial sums (4 bytes
// written and read at about 3.3 TB/s).  Contractions are split only as far as
// two items a pair.  A call for one of the two gradients uses the same split.
// Over 60 sizes drawn from 1 to 5800 tokens its choices took 1 % longer than
// the best of all widths and splits (geometric mean; the worst 15 %).
GradPlans grad_plan(int64_t m, int64_t rows, int64_t k, int num_sms) {
  GradPlans best{};
  double best_cost = 0.0;
  const int pairs = num_sms / 2 > 0 ? num_sms / 2 : 1;
  static const int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};
  for (int bn : {256, 128}) {
    const double stage = bn == 256 ? 1.0 : 0.65;
    for (int s0 : kSplits) {
      const GradPlan g0 = grad_split(m, k, rows, bn, s0);
      if (s0 > 1 && (g0.stages / s0 < kGradMinStages || g0.items > 2 * pairs)) break;
      for (int s1 : kSplits) {
        const GradPlan g1 = grad_split(rows, k, m, bn, s1);
        if (s1 > 1 && (g1.stages / s1 < kGradMinStages || g1.items > 2 * pairs)) break;
        // stages an item, longer ones first
        double u[2] = {static_cast<double>((g0.stages + s0 - 1) / s0),
                       static_cast<double>((g1.stages + s1 - 1) / s1)};
        const int64_t n[2] = {g0.items, g1.items};
        for (double& v : u) v = v < kGradMinStages ? kGradMinStages : v;
        const int first = u[1] > u[0] ? 1 : 0;
        const double ua = u[first], ub = u[first ^ 1];
        const int64_t na = n[first], nb = n[first ^ 1];
        const int64_t q = na % pairs, lag = q == 0 ? 0 : pairs - q;
        const int64_t lag_rounds = static_cast<int64_t>(ua / ub + 0.5);
        const int64_t lag_items = lag * lag_rounds < nb ? lag * lag_rounds : nb;
        const double rest = static_cast<double>((nb - lag_items + pairs - 1) / pairs) * ub;
        const double full = static_cast<double>((na + pairs - 1) / pairs) * ua;
        const double less = static_cast<double>(na / pairs) * ua +
                            (lag > 0 ? static_cast<double>((lag_items + lag - 1) / lag) * ub : 0.0);
        double cost = ((full > less ? full : less) + rest) * stage + 6.0;
        if (s0 > 1 || s1 > 1) cost += 8.0;
        if (s0 > 1) cost += static_cast<double>(g0.partial_bytes) * 2 / 1e6;
        if (s1 > 1) cost += static_cast<double>(g1.partial_bytes) * 2 / 1e6;
        if (best.bn == 0 || cost < best_cost) {
          best_cost = cost;
          best.bn = bn;
          best.first = first;
          best.lag_rounds = static_cast<int>(lag_rounds);
          best.p[0] = g0;
          best.p[1] = g1;
        }
      }
    }
  }
  return best;
}

// Row-major bf16 [outer][ld] as (inner, outer) elements, 128-byte swizzle,
// boxes of 64 x box_outer.
sfp8_status encode_bf16_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer,
                           uint64_t ld, uint32_t box_outer) {
  EncodeTiledFn enc = nullptr;
  sfp8_status s = get_encoder(&enc);
  if (s != SFP8_OK) return s;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld * 2};
  cuuint32_t box[2] = {64, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SFP8_OK : SFP8_ERR_CUDA;
}

template <int BN>
sfp8_status launch_grad_gemm(DeviceInfo* dev, const GgMaps& maps, GgParams prm, cudaStream_t st) {
  auto kern = grad_gemm_kernel<BN>;
  constexpr int slot = BN == 256 ? 0 : 1;
  constexpr int smem = GgCfg<BN>::kSmemBytes;
  static_assert(smem <= kSmemLimit, "shared memory of the gradient GEMM");
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (dev->grad_clusters[slot] == 0) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
          cudaSuccess)
        return SFP8_ERR_CUDA;
      cudaLaunchConfig_t qc{};
      qc.gridDim = dim3(2 * (dev->num_sms / 2));
      qc.blockDim = dim3(kGgThreads);
      qc.dynamicSmemBytes = smem;
      cudaLaunchAttribute ca[1];
      ca[0].id = cudaLaunchAttributeClusterDimension;
      ca[0].val.clusterDim.x = 2;
      ca[0].val.clusterDim.y = 1;
      ca[0].val.clusterDim.z = 1;
      qc.attrs = ca;
      qc.numAttrs = 1;
      int clusters = 0;
      if (cudaOccupancyMaxActiveClusters(&clusters, kern, &qc) != cudaSuccess || clusters < 1) {
        cudaGetLastError();
        return SFP8_ERR_CUDA;
      }
      dev->grad_clusters[slot] = clusters;
    }
  }
  const int items = prm.prob[0].items + prm.prob[1].items;
  prm.pairs = items < dev->grad_clusters[slot] ? items : dev->grad_clusters[slot];
  return launch_dependent(kern, dim3(2 * prm.pairs), dim3(kGgThreads), smem, st, maps, prm);
}

int blocks_for(int64_t items, int per_block, const DeviceInfo* dev, int blocks_per_sm) {
  int64_t b = (items + per_block - 1) / per_block;
  const int64_t cap = static_cast<int64_t>(dev->num_sms) * blocks_per_sm;
  if (b > cap) b = cap;
  return static_cast<int>(b);
}

// ------------------------------------------------------------------ backward plan

// Workspace of a backward pass over `rows` weight rows (2n for a gated block),
// every part on a 256-byte boundary.  It is sized for all three gradients, so
// that one query serves every call of the sizes.
struct BackwardPlan {
  GradPlans grads;
  int64_t ld_dz;          // row stride of dz in the workspace (a multiple of 8)
  int runs;               // rows of the column sums
  size_t dz_off, what_off, xhat_off, partial_off, sums_off, total;
};

constexpr int64_t kColSumMinRows = 32;   // rows a run at least: four for each of a block's warps

size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// The parts' offsets count from the workspace's first 256-byte boundary
// (stores of partial sums are 32 bytes wide); `total` leaves room for it.
uint8_t* workspace_base(void* workspace) {
  return reinterpret_cast<uint8_t*>(up256(reinterpret_cast<uintptr_t>(workspace)));
}

// sum_runs: rows of column sums that the gated gradient epilogue writes, or 0:
// as many runs as fill the device.
BackwardPlan backward_plan(int64_t m, int64_t rows, int64_t k, bool keep_dz, int sum_runs,
                           int num_sms) {
  BackwardPlan b{};
  b.ld_dz = (rows + 7) / 8 * 8;
  b.runs = sum_runs;
  if (sum_runs == 0) {
    const int64_t cols = (rows + kColSumCols - 1) / kColSumCols;
    int64_t runs = (static_cast<int64_t>(num_sms) * 3 + cols - 1) / cols;
    const int64_t most = (m + kColSumMinRows - 1) / kColSumMinRows;
    if (runs > most) runs = most;
    b.runs = static_cast<int>(runs < 1 ? 1 : runs);
  }
  size_t at = 0;
  b.dz_off = at;
  if (keep_dz) at = up256(at + static_cast<size_t>(m) * static_cast<size_t>(b.ld_dz) * 2);
  b.what_off = at;
  at = up256(at + static_cast<size_t>(rows) * static_cast<size_t>(k) * 2);
  b.xhat_off = at;
  at = up256(at + static_cast<size_t>(m) * static_cast<size_t>(k) * 2);
  b.sums_off = at;
  at = up256(at + static_cast<size_t>(b.runs) * static_cast<size_t>(rows) * sizeof(float));
  b.partial_off = at;
  b.grads = grad_plan(m, rows, k, num_sms);
  b.total = 256 + at + up256(b.grads.p[0].partial_bytes) + up256(b.grads.p[1].partial_bytes);
  return b;
}

// Whether sizes are within what the entry points accept.
bool backward_shape_ok(int64_t m, int64_t rows, int64_t k) {
  const int64_t lim = int64_t(1) << 31;
  return m > 0 && rows > 0 && k > 0 && k % kStepK == 0 && m < lim && rows < lim && k < lim;
}

struct BackwardCall {
  const void* a_q;
  sfp8_dtype a_dtype;
  const float* s_a;
  const void* packed;
  sfp8_dtype w_dtype;
  const float* s_w;
  int64_t m, rows, k;
  void* dx;
  void* dw;
  void* dbias;
};

// The expanded operands of the gradients asked for (and, for a plain linear,
// the copy and the column sums of dy), in one launch.  scaled: with the scales
// multiplied in.
sfp8_status launch_prologue(DeviceInfo* dev, const BackwardPlan& bp, const BackwardCall& c,
                            bool scaled, const void* dy, int64_t ld_dy, bool copy, bool sums,
                            uint8_t* ws, cudaStream_t st) {
  PrologueParams p{};
  p.packed = static_cast<const uint8_t*>(c.packed);
  p.s_w = scaled ? c.s_w : nullptr;
  p.w_fmt = c.w_dtype;
  p.rows = c.rows;
  p.k = c.k;
  p.what = reinterpret_cast<__nv_bfloat16*>(ws + bp.what_off);
  p.a_q = static_cast<const uint8_t*>(c.a_q);
  p.s_a = scaled ? c.s_a : nullptr;
  p.a_fmt = c.a_dtype;
  p.m = c.m;
  p.xhat = reinterpret_cast<__nv_bfloat16*>(ws + bp.xhat_off);
  p.dy = static_cast<const __nv_bfloat16*>(dy);
  p.ld_dy = ld_dy;
  p.copy = reinterpret_cast<__nv_bfloat16*>(ws + bp.dz_off);
  p.ld_copy = bp.ld_dz;
  p.sums = reinterpret_cast<float*>(ws + bp.sums_off);
  p.runs = bp.runs;
  p.sums_by_16 = aligned(dy, 16) && ld_dy % 8 == 0;
  auto units = [&](int64_t r) { return (r + kExpandRows - 1) / kExpandRows * (c.k / 128); };
  if (c.dx != nullptr) p.blocks[0] = blocks_for(units(c.rows), 1, dev, 8);
  if (c.dw != nullptr) p.blocks[1] = blocks_for(units(c.m), 1, dev, 8);
  if (copy) {
    while (p.copy_shift < 8 && (int64_t(8) << p.copy_shift) < bp.ld_dz) ++p.copy_shift;
    p.blocks[2] = blocks_for(c.m, 256 >> p.copy_shift, dev, 8);
  }
  if (sums)
    p.blocks[3] = static_cast<int>((c.rows + kColSumCols - 1) / kColSumCols) * bp.runs;
  const int64_t blocks = static_cast<int64_t>(p.blocks[0]) + p.blocks[1] + p.blocks[2] +
                         p.blocks[3];
  if (blocks == 0) return SFP8_OK;
  return launch_dependent(backward_prologue_kernel, dim3(static_cast<unsigned>(blocks)),
                          dim3(256), sums ? 8 * kColSumCols * sizeof(float) : 0, st, p);
}

// dx and dw from dz [m, rows] (row stride ld, 16-byte aligned, ld a multiple
// of 8) and the expanded operands, one launch for both products; then the
// join of split contractions and of the column sums.  pair_rows: n for a
// gated block (dz then holds both scales, dw and dbias leave in gate-then-up
// order), else 0.
sfp8_status launch_linear_grads(DeviceInfo* dev, const BackwardPlan& bp, const BackwardCall& c,
                                const void* dz, int64_t ld, int64_t pair_rows, uint8_t* ws,
                                cudaStream_t st) {
  const bool want[2] = {c.dx != nullptr, c.dw != nullptr};
  JoinParams jp{};
  if (want[0] || want[1]) {
    const GradPlans& g = bp.grads;
    GgParams prm{};
    GgMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    size_t partial = bp.partial_off;
    for (int i = 0; i < 2; ++i) {
      if (!want[i]) continue;
      // the longer items first; a lone product is the first
      const int at = i == g.first || !want[1 - i] ? 0 : 1;
      const GradPlan& pl = g.p[i];
      GgProblem& pr = prm.prob[at];
      const int64_t d_rows = i == 0 ? c.m : c.rows;
      const int64_t contraction = i == 0 ? c.rows : c.m;
      const void* b = ws + (i == 0 ? bp.what_off : bp.xhat_off);
      pr.a_rows = c.m < 128 ? static_cast<int>((c.m + 7) / 8 * 8) : 128;
      pr.t_rows = contraction < kGgStageK ? static_cast<int>((contraction + 15) / 16 * 16) : kGgStageK;
      sfp8_status s = encode_bf16_2d(&maps.a[at], dz, c.rows, c.m, ld, i == 0 ? pr.a_rows : pr.t_rows);
      if (s != SFP8_OK) return s;
      s = encode_bf16_2d(&maps.b[at], b, c.k, contraction, c.k, pr.t_rows);
      if (s != SFP8_OK) return s;
      pr.d = static_cast<__nv_bfloat16*>(i == 0 ? c.dx : c.dw);
      pr.partial = reinterpret_cast<float*>(ws + partial);
      partial += up256(pl.partial_bytes);
      pr.row_scale = pair_rows == 0 ? nullptr : i == 0 ? c.s_a : c.s_w;
      pr.rows = static_cast<int>(d_rows);
      pr.cols = static_cast<int>(c.k);
      pr.m_tiles = pl.m_tiles;
      pr.n_tiles = pl.n_tiles;
      pr.stages_total = pl.stages;
      pr.splits = pl.splits;
      pr.items = pl.items;
      pr.band = 8;   // about as many row tiles as column tiles in flight at a time
      pr.pair_rows = i == 0 ? 0 : static_cast<int>(pair_rows);
      pr.a_mn = i;
      pr.by_sector = aligned(pr.d, 32);
      pr.idesc = make_idesc_bf16(i == 1, true, kGgTileM, static_cast<uint32_t>(g.bn));
      if (pl.splits > 1) {
        jp.prob[at] = pr;
        jp.blocks[at] = blocks_for((d_rows + 15) / 16 * (c.k / 128), 1, dev, 8);
      }
    }
    prm.lag_rounds = g.lag_rounds;
    const sfp8_status s = g.bn == 256 ? launch_grad_gemm<256>(dev, maps, prm, st)
                                      : launch_grad_gemm<128>(dev, maps, prm, st);
    if (s != SFP8_OK) return s;
  }
  int blocks = jp.blocks[0] + jp.blocks[1];
  if (c.dbias != nullptr) {
    jp.sums = reinterpret_cast<const float*>(ws + bp.sums_off);
    jp.dbias = static_cast<__nv_bfloat16*>(c.dbias);
    jp.runs = bp.runs;
    jp.cols = static_cast<int>(c.rows);
    jp.pair_rows = static_cast<int>(pair_rows);
    blocks += static_cast<int>((c.rows + 31) / 32);
  }
  if (blocks == 0) return SFP8_OK;
  return launch_dependent(backward_join_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                          st, jp);
}

// Gradients of an empty problem: no tokens or no weight rows.
sfp8_status empty_grads(const BackwardCall& c, cudaStream_t st) {
  auto clear = [&](void* p, int64_t bytes) {
    if (p == nullptr || bytes == 0) return true;
    return cudaMemsetAsync(p, 0, static_cast<size_t>(bytes), st) == cudaSuccess;
  };
  if (!clear(c.dx, 2 * c.m * c.k) || !clear(c.dw, 2 * c.rows * c.k) ||
      !clear(c.dbias, 2 * c.rows)) {
    cudaGetLastError();
    return SFP8_ERR_CUDA;
  }
  return SFP8_OK;
}

// Whether the gradients share bytes with each other, with what the pass reads
// or with its workspace: it reads everything more than once, and writes one
// gradient while others are still to be computed.  Sizes are validated.
bool grads_alias(const BackwardCall& c, const void* dy, int64_t n, int64_t ld_dy,
                 const void* workspace, size_t workspace_bytes) {
  const ByteRange outs[] = {{c.dx, 2 * c.m * c.k}, {c.dw, 2 * c.rows * c.k}, {c.dbias, 2 * c.rows}};
  const ByteRange ins[] = {
      {dy, 2 * ((c.m - 1) * ld_dy + n)},
      {c.a_q, c.m * c.k},
      {c.s_a, 4 * c.m},
      {c.packed, static_cast<int64_t>(sfp8_compressed_bytes(c.rows, c.k))},
      {c.s_w, 4 * c.rows},
      {workspace, static_cast<int64_t>(workspace_bytes)}};
  return outputs_alias(outs, 3, ins, 6);
}

// Checks shared by the backward entry points: dy [m, n] with row stride ld_dy;
// need_act / need_weight say which operands are read.
sfp8_status validate_backward(const BackwardCall& c, const void* dy, int64_t n, int64_t ld_dy,
                              bool need_act, bool need_weight, bool* empty) {
  *empty = false;
  if (!is_fp8(c.a_dtype) || !is_fp8(c.w_dtype)) return SFP8_ERR_UNSUPPORTED_DTYPE;
  if (c.m < 0 || c.rows < 0 || c.k < 0 || ld_dy < n) return SFP8_ERR_INVALID_ARG;
  const int64_t lim = int64_t(1) << 31;
  if (c.k == 0 || c.k % kStepK != 0 || c.m >= lim || c.rows >= lim || c.k >= lim)
    return SFP8_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(c.dx, 16) || !aligned(c.dw, 16) || !aligned(c.dbias, 2))
    return SFP8_ERR_MISALIGNED;
  if (c.m == 0 || c.rows == 0) {
    *empty = true;
    return SFP8_OK;
  }
  if (dy == nullptr || (need_act && (c.a_q == nullptr || c.s_a == nullptr)) ||
      (need_weight && (c.packed == nullptr || c.s_w == nullptr)))
    return SFP8_ERR_INVALID_ARG;
  if (!aligned(dy, 2) || !aligned(c.a_q, 16) || !aligned(c.s_a, 4) || !aligned(c.packed, 16) ||
      !aligned(c.s_w, 4))
    return SFP8_ERR_MISALIGNED;
  return SFP8_OK;
}

// The work split of the gated block's gradient epilogue: always the CTA-pair
// kernel (no split-K).  Two weight tiles a CTA where the linear's rule takes
// them; else the token tile with the fewest rounds of tiles times their width
// (plus 32 tokens' worth of a tile's fixed cost).
LinearChoice gated_grad_choice(int64_t m, int64_t rows, int64_t k, int num_sms) {
  if (m >= kPairMinTokens) {
    const LinearChoice d = default_choice(m, rows, k, num_sms);
    if (d.wt == 2) return d;
  }
  LinearChoice c{};
  c.pair = 1;
  c.whole = 1;
  c.wt = 1;
  c.ks = (k / kStepK) % 2 == 0 ? 2 : 1;
  const int64_t groups = ((rows + kTileN - 1) / kTileN + 1) / 2;
  const int64_t pairs = num_sms / 2 > 0 ? num_sms / 2 : 1;
  int64_t best = 0;
  for (int bn = pair_bn_for(m); bn >= 32; bn -= 32) {
    const int64_t rounds = (groups * ((m + bn - 1) / bn) + pairs - 1) / pairs;
    const int64_t cost = rounds * (bn + 32);
    if (c.bn == 0 || cost < best) {
      best = cost;
      c.bn = bn;
    }
  }
  return c;
}

// Rows of column sums that its epilogue writes: one per token tile and warp of
// a lane quadrant.
int gated_grad_runs(int64_t m, int64_t rows, int64_t k, int num_sms) {
  const LinearChoice c = gated_grad_choice(m, rows, k, num_sms);
  const int parts = c.wt == 2 ? PairCfg<1, 2, kEpiGatedGrad>::kEpiParts
                              : PairCfg<1, 1, kEpiGatedGrad>::kEpiParts;
  return static_cast<int>((m + c.bn - 1) / c.bn) * parts;
}

}  // namespace
}  // namespace sfp8

extern "C" {

size_t sfp8_sparse_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (!backward_shape_ok(m, n, k)) return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return backward_plan(m, n, k, n % 8 != 0, 0, sms).total;
}

sfp8_status sfp8_sparse_linear_backward(const void* dy, int64_t ld_dy, const void* a_q,
                                        sfp8_dtype a_dtype, const float* s_a, int64_t m,
                                        const void* packed, sfp8_dtype w_dtype,
                                        const float* s_w, int64_t n, int64_t k, void* dx,
                                        void* dw, void* dbias, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  const BackwardCall c{a_q, a_dtype, s_a, packed, w_dtype, s_w, m, n, k, dx, dw, dbias};
  bool empty = false;
  sfp8_status s = validate_backward(c, dy, n, ld_dy, dw != nullptr, dx != nullptr, &empty);
  if (s != SFP8_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (empty) return empty_grads(c, st);
  // TMA reads dy in place where it can; odd widths go through a padded copy
  const bool in_place = aligned(dy, 16) && ld_dy % 8 == 0;
  if (!in_place && n % 8 == 0) return SFP8_ERR_MISALIGNED;
  if (grads_alias(c, dy, n, ld_dy, workspace, workspace_bytes)) return SFP8_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  s = current_device(&dev);
  if (s != SFP8_OK) return s;
  const BackwardPlan bp = backward_plan(m, n, k, n % 8 != 0, 0, dev->num_sms);
  if (workspace == nullptr || workspace_bytes < bp.total) return SFP8_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SFP8_ERR_MISALIGNED;
  uint8_t* ws = workspace_base(workspace);
  const bool copy = !in_place && (dx != nullptr || dw != nullptr);
  s = launch_prologue(dev, bp, c, true, dy, ld_dy, copy, dbias != nullptr, ws, st);
  if (s != SFP8_OK) return s;
  return launch_linear_grads(dev, bp, c, copy ? ws + bp.dz_off : dy, copy ? bp.ld_dz : ld_dy, 0,
                             ws, st);
}

size_t sfp8_gated_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  const int64_t rows = gated_rows(n);
  if (!backward_shape_ok(m, rows, k)) return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return backward_plan(m, rows, k, true, gated_grad_runs(m, rows, k, sms), sms).total;
}

sfp8_status sfp8_gated_linear_backward(const void* dh, int64_t ld_dh, const void* a_q,
                                       sfp8_dtype a_dtype, const float* s_a, int64_t m,
                                       const void* packed, sfp8_dtype w_dtype, const float* s_w,
                                       int64_t n, int64_t k, sfp8_activation act,
                                       const void* bias, void* dx, void* dw, void* dbias,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  sfp8_status s = validate_gated(n, act);
  if (s != SFP8_OK) return s;
  const int64_t rows = 2 * n;
  const BackwardCall c{a_q, a_dtype, s_a, packed, w_dtype, s_w, m, rows, k, dx, dw, dbias};
  bool empty = false;
  s = validate_backward(c, dh, n, ld_dh, true, true, &empty);
  if (s != SFP8_OK) return s;
  if (!aligned(bias, 2)) return SFP8_ERR_MISALIGNED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (empty) return empty_grads(c, st);
  if (grads_alias(c, dh, n, ld_dh, workspace, workspace_bytes)) return SFP8_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  s = current_device(&dev);
  if (s != SFP8_OK) return s;
  const BackwardPlan bp = backward_plan(
      m, rows, k, true, gated_grad_runs(m, rows, k, dev->num_sms), dev->num_sms);
  if (workspace == nullptr || workspace_bytes < bp.total) return SFP8_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SFP8_ERR_MISALIGNED;
  if (dx == nullptr && dw == nullptr && dbias == nullptr) return SFP8_OK;
  uint8_t* ws = workspace_base(workspace);
  s = launch_prologue(dev, bp, c, false, nullptr, 0, false, false, ws, st);
  if (s != SFP8_OK) return s;
  const LinearPlan pl =
      plan_from_choice(m, rows, k, dev->num_sms, gated_grad_choice(m, rows, k, dev->num_sms));
  const GatedCall gc{kEpiGatedGrad, act, dh, ld_dh, bp.ld_dz,
                     dbias != nullptr ? reinterpret_cast<float*>(ws + bp.sums_off) : nullptr};
  s = launch_pair(dev, pl, a_q, a_dtype, s_a, m, packed, w_dtype, s_w, rows, k, bias,
                  ws + bp.dz_off, st, &gc);
  if (s != SFP8_OK) return s;
  return launch_linear_grads(dev, bp, c, ws + bp.dz_off, bp.ld_dz, n, ws, st);
}

}  // extern "C"

// C-ABI entry points of the backward passes (declared in include/sfp8.h):
// validation, workspace layout, work splits and launches of the gradient
// GEMM (grad_gemm.cuh) and of the gated block's gradient epilogue
// (sparse_linear_pair.cuh).  Part of the library's one translation unit,
// included at its end.
#pragma once

namespace sfp8 {
namespace {

// ------------------------------------------------------------------ gradient GEMM plan

struct GradPlan {
  int bn;
  int splits;
  int m_tiles, n_tiles;
  int stages;             // of 64 along the contraction
  size_t partial_bytes;   // fp32 partial sums (splits > 1)
};

// Tile width and contraction splits that finish first by this estimate, in
// units of one 64-deep stage of a 256-wide tile (about 0.3 us): every round
// of work items takes its stages -- a 128-wide tile's stage costs 0.6 of a
// 256-wide one's, not half, since A's share of the loads stays -- plus 6
// for filling the pipeline and storing the last tile, and splitting adds a launch
// and the round trip of the partial sums (write and read, 4 bytes each, at
// about 5 TB/s).
GradPlan grad_plan(int64_t rows, int64_t cols, int64_t contraction, int num_sms) {
  GradPlan best{};
  double best_cost = 0.0;
  const int64_t pairs = num_sms / 2 > 0 ? num_sms / 2 : 1;
  const int stages = static_cast<int>((contraction + kGgStageK - 1) / kGgStageK);
  for (int bn : {256, 128}) {
    const int64_t mt = (rows + kGgTileM - 1) / kGgTileM;
    const int64_t nt = (cols + bn - 1) / bn;
    for (int splits = 1; splits <= 32; ++splits) {
      // at least 8 stages a split
      if (splits > 1 && stages / splits < 8) break;
      const int64_t rounds = (mt * nt * splits + pairs - 1) / pairs;
      const double stage = bn == 256 ? 1.0 : 0.6;
      double cost = static_cast<double>(rounds) * ((stages + splits - 1) / splits * stage) + 6.0;
      if (splits > 1)
        cost += 10.0 + 8.0 * static_cast<double>(rows) * static_cast<double>(cols) * splits / 1.5e6;
      if (best.bn == 0 || cost < best_cost) {
        best_cost = cost;
        best.bn = bn;
        best.splits = splits;
        best.m_tiles = static_cast<int>(mt);
        best.n_tiles = static_cast<int>(nt);
      }
    }
  }
  best.stages = stages;
  best.partial_bytes = best.splits > 1 ? static_cast<size_t>(best.splits) *
                                             static_cast<size_t>(rows) *
                                             static_cast<size_t>(cols) * sizeof(float)
                                       : 0;
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

template <int BN, bool A_MN>
sfp8_status launch_grad_gemm_cfg(DeviceInfo* dev, const CUtensorMap& ta, const CUtensorMap& tb,
                                 GgParams prm, cudaStream_t st) {
  auto kern = grad_gemm_kernel<BN, A_MN>;
  constexpr int slot = (BN == 256 ? 0 : 2) + (A_MN ? 1 : 0);
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
  prm.pairs = prm.items < dev->grad_clusters[slot] ? prm.items : dev->grad_clusters[slot];
  prm.idesc = make_idesc_bf16(A_MN, true, kGgTileM, BN);
  return launch_dependent(kern, dim3(2 * prm.pairs), dim3(kGgThreads), smem, st, ta, tb, prm);
}

unsigned grid_for(int64_t items, int per_block, const DeviceInfo* dev, int blocks_per_sm) {
  int64_t b = (items + per_block - 1) / per_block;
  const int64_t cap = static_cast<int64_t>(dev->num_sms) * blocks_per_sm;
  if (b > cap) b = cap;
  return static_cast<unsigned>(b < 1 ? 1 : b);
}

// D [rows, cols] = sum over t < contraction of A[r, t] B[t, c].  A is
// [rows][lda] (a_mn false) or [contraction][lda] (a_mn true), B is
// [contraction][cols]; row_scale [rows] is divided out of D (or null).
sfp8_status launch_grad_gemm(DeviceInfo* dev, const GradPlan& pl, const void* a, int64_t lda,
                             bool a_mn, const void* b, int64_t rows, int64_t cols,
                             int64_t contraction, const float* row_scale, void* d,
                             int64_t pair_rows, float* partial, cudaStream_t st) {
  CUtensorMap ta, tb;
  sfp8_status s = a_mn ? encode_bf16_2d(&ta, a, rows, contraction, lda, kGgStageK)
                       : encode_bf16_2d(&ta, a, contraction, rows, lda, 128);
  if (s != SFP8_OK) return s;
  s = encode_bf16_2d(&tb, b, cols, contraction, cols, kGgStageK);
  if (s != SFP8_OK) return s;
  GgParams prm{};
  prm.d = static_cast<__nv_bfloat16*>(d);
  prm.partial = partial;
  prm.ld_d = cols;
  prm.rows = static_cast<int>(rows);
  prm.cols = static_cast<int>(cols);
  prm.m_tiles = pl.m_tiles;
  prm.n_tiles = pl.n_tiles;
  prm.stages_total = pl.stages;
  prm.splits = pl.splits;
  prm.items = pl.m_tiles * pl.n_tiles * pl.splits;
  // about as many row tiles as column tiles in flight at a time
  prm.band = 8;
  prm.row_scale = row_scale;
  prm.pair_rows = static_cast<int>(pair_rows);
  if (pl.bn == 256)
    s = a_mn ? launch_grad_gemm_cfg<256, true>(dev, ta, tb, prm, st)
             : launch_grad_gemm_cfg<256, false>(dev, ta, tb, prm, st);
  else
    s = a_mn ? launch_grad_gemm_cfg<128, true>(dev, ta, tb, prm, st)
             : launch_grad_gemm_cfg<128, false>(dev, ta, tb, prm, st);
  if (s != SFP8_OK || pl.splits == 1) return s;
  return launch_dependent(grad_gemm_join_kernel, dim3(grid_for(rows * (cols / 8), 256, dev, 8)),
                          dim3(256), 0, st, static_cast<const float*>(partial), pl.splits,
                          static_cast<int>(rows), static_cast<int>(cols), row_scale,
                          static_cast<__nv_bfloat16*>(d), static_cast<long long>(cols),
                          static_cast<int>(pair_rows));
}

// ------------------------------------------------------------------ backward plan

// Workspace of a backward pass over `rows` weight rows (2n for a gated block),
// in this order, every part on a 256-byte boundary.
struct BackwardPlan {
  int64_t ld_dz;          // row stride of dz in the workspace (a multiple of 8)
  GradPlan dx, dw;
  int runs;               // row runs of the column sums
  size_t dz_off, expand_off, partial_off, sums_off, total;
};

constexpr int64_t kColSumMinRows = 64;   // rows a run at least

BackwardPlan backward_plan(int64_t m, int64_t rows, int64_t k, bool keep_dz, int num_sms) {
  BackwardPlan b{};
  auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  b.ld_dz = (rows + 7) / 8 * 8;
  b.dx = grad_plan(m, k, rows, num_sms);
  b.dw = grad_plan(rows, k, m, num_sms);
  // enough blocks of column sums to fill the device, with long enough runs
  const int64_t cols = (rows + kColSumCols - 1) / kColSumCols;
  int64_t runs = (static_cast<int64_t>(num_sms) * 8 + cols - 1) / cols;
  if (runs > (m + kColSumMinRows - 1) / kColSumMinRows)
    runs = (m + kColSumMinRows - 1) / kColSumMinRows;
  b.runs = static_cast<int>(runs < 1 ? 1 : runs);
  size_t at = 0;
  b.dz_off = at;
  if (keep_dz) at = up(at + static_cast<size_t>(m) * static_cast<size_t>(b.ld_dz) * 2);
  // the expanded weight, then (the input gradient done) the expanded checkpoint
  b.expand_off = at;
  at = up(at + static_cast<size_t>(rows > m ? rows : m) * static_cast<size_t>(k) * 2);
  b.partial_off = at;
  at = up(at + (b.dx.partial_bytes > b.dw.partial_bytes ? b.dx.partial_bytes
                                                        : b.dw.partial_bytes));
  b.sums_off = at;
  at = up(at + static_cast<size_t>(b.runs) * static_cast<size_t>(rows) * sizeof(float));
  b.total = at;
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

// dx, dw and dbias from dz [m, rows] (row stride ld, 16-byte aligned, ld a
// multiple of 8): expand the weight, dx; expand the checkpoint, dw; column
// sums.  pair_rows: n for a gated block (dz then holds both scales, dw and
// dbias leave in gate-then-up order), else 0.
sfp8_status launch_linear_grads(DeviceInfo* dev, const BackwardPlan& bp, const BackwardCall& c,
                                const void* dz, int64_t ld, int64_t pair_rows, uint8_t* ws,
                                cudaStream_t st) {
  __nv_bfloat16* expanded = reinterpret_cast<__nv_bfloat16*>(ws + bp.expand_off);
  float* partial = reinterpret_cast<float*>(ws + bp.partial_off);
  sfp8_status s = SFP8_OK;
  // the scales are in the expanded operand, or in dz and divided out
  const bool scaled_dz = pair_rows != 0;
  const float* none = nullptr;
  if (c.dx != nullptr) {
    auto kern = c.w_dtype == SFP8_E5M2 ? expand_weight_kernel<SFP8_E5M2>
                                       : expand_weight_kernel<SFP8_E4M3>;
    s = launch_dependent(kern, dim3(grid_for(c.rows * (c.k / 32), 256, dev, 8)), dim3(256), 0, st,
                         static_cast<const uint8_t*>(c.packed), scaled_dz ? none : c.s_w,
                         static_cast<long long>(c.rows), static_cast<long long>(c.k), expanded);
    if (s != SFP8_OK) return s;
    s = launch_grad_gemm(dev, bp.dx, dz, ld, false, expanded, c.m, c.k, c.rows,
                         scaled_dz ? c.s_a : none, c.dx, 0, partial, st);
    if (s != SFP8_OK) return s;
  }
  if (c.dw != nullptr) {
    auto kern = c.a_dtype == SFP8_E5M2 ? expand_rows_kernel<SFP8_E5M2>
                                       : expand_rows_kernel<SFP8_E4M3>;
    s = launch_dependent(kern, dim3(grid_for(c.m * (c.k / 16), 256, dev, 8)), dim3(256), 0, st,
                         static_cast<const uint8_t*>(c.a_q), scaled_dz ? none : c.s_a,
                         static_cast<long long>(c.m), static_cast<long long>(c.k), expanded);
    if (s != SFP8_OK) return s;
    s = launch_grad_gemm(dev, bp.dw, dz, ld, true, expanded, c.rows, c.k, c.m,
                         scaled_dz ? c.s_w : none, c.dw, pair_rows, partial, st);
    if (s != SFP8_OK) return s;
  }
  if (c.dbias != nullptr) {
    float* sums = reinterpret_cast<float*>(ws + bp.sums_off);
    s = launch_dependent(column_sums_kernel,
                         dim3(static_cast<unsigned>((c.rows + kColSumCols - 1) / kColSumCols),
                              static_cast<unsigned>(bp.runs)),
                         dim3(256), 0, st, static_cast<const __nv_bfloat16*>(dz),
                         static_cast<long long>(c.m), static_cast<long long>(c.rows),
                         static_cast<long long>(ld), scaled_dz ? c.s_a : none, sums);
    if (s != SFP8_OK) return s;
    s = launch_dependent(column_sums_join_kernel,
                         dim3(static_cast<unsigned>((c.rows + 255) / 256)), dim3(256), 0, st,
                         static_cast<const float*>(sums), bp.runs, static_cast<long long>(c.rows),
                         scaled_dz ? c.s_w : none, static_cast<__nv_bfloat16*>(c.dbias),
                         static_cast<long long>(pair_rows));
  }
  return s;
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
// kernel (no split-K).  The token tile is the widest that leaves a tile for
// every pair.
LinearChoice gated_grad_choice(int64_t m, int64_t rows, int64_t k, int num_sms) {
  if (m >= kPairMinTokens) return default_choice(m, rows, k, num_sms);
  LinearChoice c{};
  c.pair = 1;
  c.whole = 1;
  c.wt = 1;
  c.ks = (k / kStepK) % 2 == 0 ? 2 : 1;
  c.bn = pair_bn_for(m);
  const int64_t groups = ((rows + kTileN - 1) / kTileN + 1) / 2;
  while (c.bn > 32 && groups * ((m + c.bn - 1) / c.bn) < num_sms / 2) c.bn -= 32;
  return c;
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
  return backward_plan(m, n, k, n % 8 != 0, sms).total;
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
  DeviceInfo* dev = nullptr;
  s = current_device(&dev);
  if (s != SFP8_OK) return s;
  const BackwardPlan bp = backward_plan(m, n, k, n % 8 != 0, dev->num_sms);
  if (workspace == nullptr || workspace_bytes < bp.total) return SFP8_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SFP8_ERR_MISALIGNED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const void* dz = dy;
  int64_t ld = ld_dy;
  if (!in_place && (dx != nullptr || dw != nullptr)) {
    dz = ws + bp.dz_off;
    ld = bp.ld_dz;
    s = launch_dependent(copy_rows_kernel, dim3(grid_for(m * ld, 256, dev, 8)), dim3(256), 0, st,
                         static_cast<const __nv_bfloat16*>(dy), static_cast<long long>(m),
                         static_cast<long long>(n), static_cast<long long>(ld_dy),
                         reinterpret_cast<__nv_bfloat16*>(ws + bp.dz_off),
                         static_cast<long long>(ld));
    if (s != SFP8_OK) return s;
  }
  return launch_linear_grads(dev, bp, c, dz, ld, 0, ws, st);
}

size_t sfp8_gated_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  const int64_t rows = gated_rows(n);
  if (!backward_shape_ok(m, rows, k)) return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return backward_plan(m, rows, k, true, sms).total;
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
  DeviceInfo* dev = nullptr;
  s = current_device(&dev);
  if (s != SFP8_OK) return s;
  const BackwardPlan bp = backward_plan(m, rows, k, true, dev->num_sms);
  if (workspace == nullptr || workspace_bytes < bp.total) return SFP8_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SFP8_ERR_MISALIGNED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const LinearPlan pl =
      plan_from_choice(m, rows, k, dev->num_sms, gated_grad_choice(m, rows, k, dev->num_sms));
  const GatedCall gc{kEpiGatedGrad, act, dh, ld_dh, bp.ld_dz};
  s = launch_pair(dev, pl, a_q, a_dtype, s_a, m, packed, w_dtype, s_w, rows, k, bias,
                  ws + bp.dz_off, st, &gc);
  if (s != SFP8_OK) return s;
  return launch_linear_grads(dev, bp, c, ws + bp.dz_off, bp.ld_dz, n, ws, st);
}

}  // extern "C"

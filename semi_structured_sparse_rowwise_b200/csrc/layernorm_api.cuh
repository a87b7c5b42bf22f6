// C-ABI entry points of layer norm (declared in include/sfp8.h): validation
// and the choice of the kernel by row length, alignment and row count
// (layernorm.cuh).  Part of the library's one translation unit, included at
// its end.
#pragma once

namespace sfp8 {
namespace {

// Shared memory a stream kernel may use.
constexpr int kNormSmemBudget = 224 * 1024;

// ------------------------------------------------------------------ forward

template <typename T, int VEC, int TPR, int N, bool Q>
sfp8_status launch_norm_rows(const NormParams& p, cudaStream_t st) {
  constexpr int threads = TPR == 32 ? 256 : TPR;
  constexpr int groups = TPR == 32 ? 8 : 1;
  return launch_dependent(layernorm_kernel<T, VEC, TPR, N, Q>,
                          dim3(static_cast<unsigned>((p.rows + groups - 1) / groups)),
                          dim3(threads), 0, st, p);
}

// Row buffers of a row group: what is left of the block's shared memory after
// the parameters, at most eight rows.
int norm_slots(int groups, int params, int cols, int parts, int row_bytes) {
  const int left = kNormSmemBudget - params * cols * 4;
  const int s = left / (groups * parts * row_bytes);
  return s < kNormMaxSlots ? s : kNormMaxSlots;
}

// Co-resident blocks of a persistent kernel on the device (queried once a
// slot).
template <typename Kernel>
sfp8_status norm_resident(DeviceInfo* dev, int slot, Kernel kern, int threads, int* blocks) {
  std::lock_guard<std::mutex> lock(g_mutex);
  if (dev->norm_blocks[slot] == 0) {
    int occ = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, threads, 0) != cudaSuccess ||
        occ < 1) {
      cudaGetLastError();
      return SFP8_ERR_CUDA;
    }
    dev->norm_blocks[slot] = occ;
  }
  *blocks = dev->norm_blocks[slot] * dev->num_sms;
  return SFP8_OK;
}

// Blocks of a stream kernel: one a SM, or as many as leave every row group the
// same number of rows, give or take one.
int norm_stream_blocks(const DeviceInfo* dev, int per_block, int64_t rows) {
  const int64_t groups = static_cast<int64_t>(per_block) * dev->num_sms;
  const int64_t each = (rows + groups - 1) / groups;
  const int64_t used = (rows + each - 1) / each;
  return static_cast<int>((used + per_block - 1) / per_block);
}

// threads: of a block, per_block row groups; params, parts: fp32 parameter
// vectors and rows (x; x and dy) in shared memory.
template <typename Kernel, typename P>
sfp8_status launch_norm_stream(DeviceInfo* dev, int slot, Kernel kern, int threads,
                               int per_block, const P& p, int params, int parts, int row_bytes,
                               cudaStream_t st) {
  const int slots = norm_slots(per_block, params, p.cols, parts, row_bytes);
  if (slots < 2) return SFP8_ERR_UNSUPPORTED_SHAPE;   // no such width is sent here
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (dev->norm_blocks[slot] == 0) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kNormSmemBudget) != cudaSuccess) {
        cudaGetLastError();
        return SFP8_ERR_CUDA;
      }
      dev->norm_blocks[slot] = 1;
    }
  }
  return launch_dependent(
      kern, dim3(static_cast<unsigned>(norm_stream_blocks(dev, per_block, p.rows))),
      dim3(threads),
      static_cast<size_t>(norm_stream_smem(per_block, params, p.cols, parts, row_bytes, slots)),
      st, p, slots);
}

// 16-byte vectors.  Few rows (a decode step, fewer than two a SM): as many
// threads as vectors, so that the chain of one load, three reductions and one
// store is all a row takes.  Many rows (eight a SM and more): the stream
// kernel (8192 rows of 4096 bf16 to codes: 26 us, the row kernel with four
// vectors a thread 43 us), with as many row groups as its registers allow.
template <typename T, bool Q>
sfp8_status launch_norm_vec(DeviceInfo* dev, int kind, const NormParams& p, cudaStream_t st) {
  constexpr int V = InputTraits<T>::kPerVec;
  const int nvec = p.cols / V;
  const int s0 = kind * 12 + (Q ? 0 : 8);   // 8 slots to codes, 4 without
  if (nvec <= 32) return launch_norm_rows<T, V, 32, 1, Q>(p, st);
  if (nvec > 64 && nvec <= 1024 && p.rows >= 8ll * dev->num_sms) {
    const int bytes = p.cols * static_cast<int>(sizeof(T));
    auto go = [&](int slot, auto kern, int threads, int per_block) {
      return launch_norm_stream(dev, s0 + slot, kern, threads, per_block, p, 2, 1, bytes, st);
    };
    if constexpr (Q) {
      if (nvec == 128) return go(4, layernorm_stream_kernel<T, V, 64, 2, 960, Q, true>, 960, 15);
      if (nvec == 256) return go(5, layernorm_stream_kernel<T, V, 64, 4, 768, Q, true>, 768, 12);
      if (nvec == 512) return go(6, layernorm_stream_kernel<T, V, 64, 8, 512, Q, true>, 512, 8);
      if (nvec == 1024) return go(7, layernorm_stream_kernel<T, V, 128, 8, 512, Q, true>, 512, 4);
    }
    if (nvec <= 128) return go(0, layernorm_stream_kernel<T, V, 64, 2, 960, Q, false>, 960, 15);
    if (nvec <= 256) return go(1, layernorm_stream_kernel<T, V, 64, 4, 768, Q, false>, 768, 12);
    if (nvec <= 512) return go(2, layernorm_stream_kernel<T, V, 64, 8, 512, Q, false>, 512, 8);
    return go(3, layernorm_stream_kernel<T, V, 128, 8, 512, Q, false>, 512, 4);
  }
  if (p.rows < 2ll * dev->num_sms) {
    if (nvec <= 128) return launch_norm_rows<T, V, 128, 1, Q>(p, st);
    if (nvec <= 512) return launch_norm_rows<T, V, 512, 1, Q>(p, st);
    if (nvec <= 1024) return launch_norm_rows<T, V, 1024, 1, Q>(p, st);
  } else {
    if (nvec <= 64) return launch_norm_rows<T, V, 32, 2, Q>(p, st);
    if (nvec <= 128) return launch_norm_rows<T, V, 32, 4, Q>(p, st);
    if (nvec <= 512) return launch_norm_rows<T, V, 128, 4, Q>(p, st);
    if (nvec <= 1024) return launch_norm_rows<T, V, 256, 4, Q>(p, st);
  }
  if (nvec <= 2048) return launch_norm_rows<T, V, 512, 4, Q>(p, st);
  if (nvec <= 4096) return launch_norm_rows<T, V, 1024, 4, Q>(p, st);
  return launch_dependent(layernorm_long_kernel<T, V, Q>, dim3(static_cast<unsigned>(p.rows)),
                          dim3(1024), 0, st, p);
}

// One element at a time: odd widths and unaligned rows.
template <typename T>
sfp8_status launch_norm_scalar(const NormParams& p, cudaStream_t st) {
  if (p.cols <= 1024) return launch_norm_rows<T, 1, 128, 8, false>(p, st);
  if (p.cols <= 4096) return launch_norm_rows<T, 1, 256, 16, false>(p, st);
  if (p.cols <= 16384) return launch_norm_rows<T, 1, 1024, 16, false>(p, st);
  return launch_dependent(layernorm_long_kernel<T, 1, false>,
                          dim3(static_cast<unsigned>(p.rows)), dim3(1024), 0, st, p);
}

// kind: the type's index, for the cached occupancies.
template <typename T>
sfp8_status launch_norm(DeviceInfo* dev, int kind, const NormParams& p, bool vec,
                        cudaStream_t st) {
  if (p.q != nullptr) return launch_norm_vec<T, true>(dev, kind, p, st);
  if (vec) return launch_norm_vec<T, false>(dev, kind, p, st);
  return launch_norm_scalar<T>(p, st);
}

// ------------------------------------------------------------------ backward

// Row groups the backward pass may use (each leaves one partial sum of 2 cols
// floats): three a SM, and for many short rows up to 16 a SM as long as every
// group still has 16 rows, which keeps the partial sums' traffic a small
// part of the inputs'.
int64_t norm_groups(int64_t rows, int num_sms) {
  int64_t g = rows / 16;
  if (g > 16ll * num_sms) g = 16ll * num_sms;
  if (g < 3ll * num_sms) g = 3ll * num_sms;
  return g < rows ? g : rows;
}

template <typename T, int VEC, int TPR, int N, bool NARROW = false>
sfp8_status launch_norm_grad_rows(DeviceInfo* dev, int slot, NormGradParams& p, cudaStream_t st) {
  auto kern = layernorm_backward_kernel<T, VEC, TPR, N, NARROW>;
  constexpr int threads = TPR == 32 ? 256 : TPR;
  constexpr int per_block = TPR == 32 ? 8 : 1;
  int blocks = 0;
  const sfp8_status s = norm_resident(dev, slot, kern, threads, &blocks);
  if (s != SFP8_OK) return s;
  // one wave of co-resident blocks
  if (p.groups > static_cast<int64_t>(blocks) * per_block) p.groups = blocks * per_block;
  return launch_dependent(kern, dim3(static_cast<unsigned>((p.groups + per_block - 1) / per_block)),
                          dim3(threads), 0, st, p);
}

template <typename T, typename Kernel>
sfp8_status launch_norm_grad_stream(DeviceInfo* dev, int slot, Kernel kern, int threads,
                                    int per_block, NormGradParams& p, cudaStream_t st) {
  p.groups = norm_stream_blocks(dev, per_block, p.rows);   // one partial sum a block
  return launch_norm_stream(dev, slot, kern, threads, per_block, p, 1, 2,
                            p.cols * static_cast<int>(sizeof(T)), st);
}

// Rows too long for the registers: dx by rows, the sums by columns.
template <typename T>
sfp8_status launch_norm_grad_long(NormGradParams& p, bool vec, bool sums, cudaStream_t st) {
  if (p.dx != nullptr) {
    auto kern = vec ? layernorm_backward_long_kernel<T, InputTraits<T>::kPerVec>
                    : layernorm_backward_long_kernel<T, 1>;
    const sfp8_status s = launch_dependent(kern, dim3(static_cast<unsigned>(p.rows)), dim3(1024),
                                           0, st, p);
    if (s != SFP8_OK) return s;
  }
  if (!sums) return SFP8_OK;
  if (p.groups > 32) p.groups = 32;
  return launch_dependent(layernorm_backward_columns_kernel<T>,
                          dim3(static_cast<unsigned>((p.cols + 31) / 32),
                               static_cast<unsigned>(p.groups)),
                          dim3(256), 0, st, p);
}

// kind: the type's index, for the cached occupancies.
template <typename T>
sfp8_status launch_norm_grad(DeviceInfo* dev, int kind, NormGradParams& p, bool vec, bool sums,
                             cudaStream_t st) {
  constexpr int V = InputTraits<T>::kPerVec;
  const int s0 = 36 + kind * 12;
  if (vec) {
    const int nvec = p.cols / V;
    if (nvec <= 32) return launch_norm_grad_rows<T, V, 32, 1>(dev, s0, p, st);
    if (nvec <= 64) return launch_norm_grad_rows<T, V, 32, 2>(dev, s0 + 1, p, st);
    auto go = [&](int slot, auto kern, int threads, int per_block) {
      return launch_norm_grad_stream<T>(dev, s0 + slot, kern, threads, per_block, p, st);
    };
    if (nvec == 128)
      return go(8, layernorm_backward_stream_kernel<T, V, 128, 1, 768, true>, 768, 6);
    if (nvec == 256)
      return go(9, layernorm_backward_stream_kernel<T, V, 128, 2, 640, true>, 640, 5);
    if (nvec == 512)
      return go(10, layernorm_backward_stream_kernel<T, V, 128, 4, 512, true>, 512, 4);
    if (nvec == 1024)
      return go(11, layernorm_backward_stream_kernel<T, V, 256, 4, 512, true>, 512, 2);
    if (nvec <= 128)
      return go(2, layernorm_backward_stream_kernel<T, V, 128, 1, 768, false>, 768, 6);
    if (nvec <= 256)
      return go(3, layernorm_backward_stream_kernel<T, V, 128, 2, 640, false>, 640, 5);
    if (nvec <= 512)
      return go(4, layernorm_backward_stream_kernel<T, V, 128, 4, 512, false>, 512, 4);
    if (nvec <= 1024)
      return go(5, layernorm_backward_stream_kernel<T, V, 256, 4, 512, false>, 512, 2);
  } else {
    if (p.cols <= 32) return launch_norm_grad_rows<T, 1, 32, 1, true>(dev, 72 + kind, p, st);
    if (p.cols <= 1024) return launch_norm_grad_rows<T, 1, 128, 8>(dev, s0 + 6, p, st);
    if (p.cols <= 4096) return launch_norm_grad_rows<T, 1, 512, 8>(dev, s0 + 7, p, st);
  }
  return launch_norm_grad_long<T>(p, vec, sums, st);
}

bool norm_params_dtype(sfp8_dtype x_dtype, sfp8_dtype p_dtype) {
  return p_dtype == x_dtype || p_dtype == SFP8_F32;
}

// Whether [rows, cols] of element size es at p, row stride ld, can be moved
// 16 bytes at a time.
bool rows_by_16(const void* p, int64_t ld, int64_t cols, int es) {
  return aligned(p, 16) && (ld * es) % 16 == 0 && (cols * es) % 16 == 0;
}

}  // namespace
}  // namespace sfp8

extern "C" {

sfp8_status sfp8_layernorm(const void* x, sfp8_dtype x_dtype, int64_t rows, int64_t cols,
                           int64_t ld_x, const void* weight, const void* bias, sfp8_dtype p_dtype,
                           float eps, void* y, void* q, sfp8_dtype q_dtype, float* scales,
                           float* mean, float* rstd, void* stream) {
  if (!is_wide(x_dtype) || !norm_params_dtype(x_dtype, p_dtype)) return SFP8_ERR_UNSUPPORTED_DTYPE;
  if (q != nullptr && !is_fp8(q_dtype)) return SFP8_ERR_UNSUPPORTED_DTYPE;
  if (rows < 0 || cols < 0 || ld_x < cols || !(eps >= 0.0f) || eps > 3.0e38f)
    return SFP8_ERR_INVALID_ARG;
  if (cols == 0 || (q != nullptr && cols % 16 != 0)) return SFP8_ERR_UNSUPPORTED_SHAPE;
  if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 30)) return SFP8_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return SFP8_OK;
  if (x == nullptr || (q != nullptr && scales == nullptr)) return SFP8_ERR_INVALID_ARG;
  const int es = elem_size(x_dtype), ps = elem_size(p_dtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(weight, ps) || !aligned(bias, ps) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return SFP8_ERR_MISALIGNED;
  const bool vec = rows_by_16(x, ld_x, cols, es) && aligned(y, 16) && aligned(weight, 16) &&
                   aligned(bias, 16);
  if (q != nullptr && (!vec || !aligned(q, 16) || !aligned(scales, 4))) return SFP8_ERR_MISALIGNED;
  if (y == nullptr && q == nullptr && mean == nullptr && rstd == nullptr) return SFP8_OK;
  {
    // rows are read while others are written, and long ones more than once
    const ByteRange outs[] = {{y, rows * cols * es},
                              {q, rows * cols},
                              {q != nullptr ? scales : nullptr, 4 * rows},
                              {mean, 4 * rows},
                              {rstd, 4 * rows}};
    const ByteRange ins[] = {{x, ((rows - 1) * ld_x + cols) * es}, {weight, cols * ps},
                             {bias, cols * ps}};
    if (outputs_alias(outs, 5, ins, 3)) return SFP8_ERR_INVALID_ARG;
  }
  DeviceInfo* dev = nullptr;
  const sfp8_status s = current_device(&dev);
  if (s != SFP8_OK) return s;
  NormParams p{};
  p.x = x;
  p.rows = rows;
  p.ld_x = ld_x;
  p.cols = static_cast<int>(cols);
  p.weight = weight;
  p.bias = bias;
  p.params_f32 = p_dtype == SFP8_F32;
  p.eps = eps;
  p.y = y;
  p.q = static_cast<uint8_t*>(q);
  p.q_fmt = q_dtype;
  p.scales = scales;
  p.mean = mean;
  p.rstd = rstd;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (x_dtype) {
    case SFP8_BF16: return launch_norm<__nv_bfloat16>(dev, 0, p, vec, st);
    case SFP8_F16: return launch_norm<__half>(dev, 1, p, vec, st);
    default: return launch_norm<float>(dev, 2, p, vec, st);
  }
}

size_t sfp8_layernorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 30)) return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return static_cast<size_t>(norm_groups(rows, sms)) * 2 * static_cast<size_t>(cols) *
         sizeof(float);
}

sfp8_status sfp8_layernorm_backward(const void* dy, int64_t ld_dy, const void* x,
                                    sfp8_dtype x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                                    const void* weight, sfp8_dtype p_dtype, const float* mean,
                                    const float* rstd, void* dx, float* dweight, float* dbias,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!is_wide(x_dtype) || !norm_params_dtype(x_dtype, p_dtype)) return SFP8_ERR_UNSUPPORTED_DTYPE;
  if (rows < 0 || cols < 0 || ld_x < cols || ld_dy < cols) return SFP8_ERR_INVALID_ARG;
  if (cols == 0 || rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 30))
    return SFP8_ERR_UNSUPPORTED_SHAPE;
  const int es = elem_size(x_dtype);
  if (!aligned(x, es) || !aligned(dy, es) || !aligned(dx, es) ||
      !aligned(weight, elem_size(p_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(dweight, 4) || !aligned(dbias, 4))
    return SFP8_ERR_MISALIGNED;
  const bool sums = dweight != nullptr || dbias != nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if ((dweight != nullptr &&
         cudaMemsetAsync(dweight, 0, static_cast<size_t>(cols) * 4, st) != cudaSuccess) ||
        (dbias != nullptr &&
         cudaMemsetAsync(dbias, 0, static_cast<size_t>(cols) * 4, st) != cudaSuccess)) {
      cudaGetLastError();
      return SFP8_ERR_CUDA;
    }
    return SFP8_OK;
  }
  if (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr)
    return SFP8_ERR_INVALID_ARG;
  if (dx == nullptr && !sums) return SFP8_OK;
  {
    const ByteRange outs[] = {{dx, rows * cols * es}, {dweight, 4 * cols}, {dbias, 4 * cols}};
    const ByteRange ins[] = {{x, ((rows - 1) * ld_x + cols) * es},
                             {dy, ((rows - 1) * ld_dy + cols) * es},
                             {weight, cols * elem_size(p_dtype)},
                             {mean, 4 * rows},
                             {rstd, 4 * rows},
                             {workspace, static_cast<int64_t>(workspace_bytes)}};
    if (outputs_alias(outs, 3, ins, 6)) return SFP8_ERR_INVALID_ARG;
  }
  DeviceInfo* dev = nullptr;
  sfp8_status s = current_device(&dev);
  if (s != SFP8_OK) return s;
  const int64_t groups = norm_groups(rows, dev->num_sms);
  if (workspace == nullptr ||
      workspace_bytes < static_cast<size_t>(groups) * 2 * static_cast<size_t>(cols) * sizeof(float))
    return SFP8_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SFP8_ERR_MISALIGNED;
  NormGradParams p{};
  p.dy = dy;
  p.x = x;
  p.rows = rows;
  p.ld_dy = ld_dy;
  p.ld_x = ld_x;
  p.cols = static_cast<int>(cols);
  p.weight = weight;
  p.params_f32 = p_dtype == SFP8_F32;
  p.mean = mean;
  p.rstd = rstd;
  p.dx = dx;
  p.partial = static_cast<float*>(workspace);
  p.groups = static_cast<int>(groups);
  const bool vec = rows_by_16(x, ld_x, cols, es) && rows_by_16(dy, ld_dy, cols, es) &&
                   aligned(dx, 16) && aligned(weight, 16);
  switch (x_dtype) {
    case SFP8_BF16: s = launch_norm_grad<__nv_bfloat16>(dev, 0, p, vec, sums, st); break;
    case SFP8_F16: s = launch_norm_grad<__half>(dev, 1, p, vec, sums, st); break;
    default: s = launch_norm_grad<float>(dev, 2, p, vec, sums, st); break;
  }
  if (s != SFP8_OK || !sums) return s;
  return launch_dependent(layernorm_backward_join_kernel,
                          dim3(static_cast<unsigned>((2 * cols + 31) / 32)), dim3(1024), 0, st,
                          static_cast<const float*>(p.partial), p.groups, p.cols, dweight, dbias);
}

}  // extern "C"

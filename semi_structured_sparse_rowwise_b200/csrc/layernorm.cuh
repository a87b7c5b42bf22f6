// Layer norm, forward (to the activation's type and/or straight to row-wise
// FP8 codes) and backward (with the sums over rows of the weight's and bias's
// gradients).
//
//   forward   mean = sum_c x / C,   var = sum_c (x - mean)^2 / C
//             rstd = 1 / sqrt(var + eps)
//             y    = (x - mean) * rstd * weight + bias
//             s    = max(max_c |y|, 1e-12) / FP8_MAX,  q = fp8(y / s)
//   backward  xh = (x - mean) * rstd,  g = weight * dy
//             dx = rstd * (g - sum_c g / C - xh * sum_c (g xh) / C)
//             dweight = sum_rows dy * xh,   dbias = sum_rows dy
//
// All of it in fp32; y and dx are rounded once to x's type, the codes once
// from the fp32 y.  The variance is taken about the mean (two reductions over
// values held in registers), never as a difference of two sums.
//
// Both passes are bound by memory: a row is read once into the registers of
// TPR threads (N vectors of VEC elements each), reduced by warp shuffles and,
// for more than one warp, shared memory, and written from the registers.
// VEC elements make 16 bytes where base, row stride and width allow, else 1.
// Rows that do not fit the registers take the loop kernels, which read them
// again from L2.
//
// The backward kernel is persistent: a group of TPR threads walks rows, keeps
// its columns' dweight and dbias sums in registers, loads the next row before
// it finishes this one, and writes one partial sum per group at the end; a
// second kernel adds the groups in order (no atomics: the same bits every
// time).
#pragma once

#include <type_traits>

#include "quantize_rowwise.cuh"

namespace sfp8 {

struct NormParams {
  const void* x;
  long long rows, ld_x;
  int cols;
  const void* weight;     // [cols] or null (ones)
  const void* bias;       // [cols] or null (zeros)
  int params_f32;         // weight and bias are fp32, else x's type
  float eps;
  void* y;                // [rows][cols] or null
  uint8_t* q;             // [rows][cols] codes
  int q_fmt;              // SFP8_E4M3 / SFP8_E5M2
  float* scales;
  float* mean;            // [rows] or null
  float* rstd;            // [rows] or null
};

struct NormGradParams {
  const void* dy;
  const void* x;
  long long rows, ld_dy, ld_x;
  int cols;
  const void* weight;     // [cols] or null (ones)
  int params_f32;
  const float* mean;
  const float* rstd;
  void* dx;               // [rows][cols] or null
  float* partial;         // [groups][2][cols]
  int groups;
};

// VEC elements of T (16 bytes, or one element) as they are loaded.
template <typename T, int VEC>
struct NormVec;
template <typename T>
struct NormVec<T, 1> {
  T v;
  __device__ void load(const T* p) { v = *p; }
  __device__ void floats(float (&f)[1]) const {
    if constexpr (sizeof(T) == 4) f[0] = v;
    else if constexpr (std::is_same<T, __half>::value) f[0] = __half2float(v);
    else f[0] = __bfloat162float(v);
  }
};
template <typename T, int VEC>
struct NormVec {
  static_assert(VEC * sizeof(T) == 16, "16-byte vectors");
  uint4 v;
  __device__ void load(const T* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ void floats(float (&f)[VEC]) const { InputTraits<T>::to_float(v, f); }
};

template <typename T>
__device__ __forceinline__ T norm_round(float f) {
  if constexpr (sizeof(T) == 4) return f;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(f);
  else return __float2bfloat16_rn(f);
}

template <typename T, int VEC>
__device__ __forceinline__ void norm_store(T* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    *p = norm_round<T>(f[0]);
  } else {
    __align__(16) T out[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[i] = norm_round<T>(f[i]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(out);
  }
}

// VEC parameters from column c on, as floats.
template <typename T, int VEC>
__device__ __forceinline__ void norm_params(const void* p, int f32, int c, float missing,
                                            float (&f)[VEC]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = missing;
  } else if (f32 && sizeof(T) != 4) {
    const float* w = static_cast<const float*>(p) + c;
    if constexpr (VEC == 1) {
      f[0] = __ldg(w);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const float4 t = __ldg(reinterpret_cast<const float4*>(w + i));
        f[i] = t.x;
        f[i + 1] = t.y;
        f[i + 2] = t.z;
        f[i + 3] = t.w;
      }
    }
  } else {
    NormVec<T, VEC> v;
    v.load(static_cast<const T*>(p) + c);
    v.floats(f);
  }
}

// Codes of VEC values (VEC 4 or 8) at q.
template <int VEC>
__device__ __forceinline__ void norm_codes(uint8_t* q, const float (&f)[VEC], float s, float r,
                                           int fmt) {
  uint32_t w[VEC / 4];
  if (fmt == SFP8_E5M2) quantize_vec<SFP8_E5M2, VEC>(f, s, r, w);
  else quantize_vec<SFP8_E4M3, VEC>(f, s, r, w);
  store_codes<VEC>(q, w);
}

__device__ __forceinline__ float norm_fp8_max(int fmt) {
  return fmt == SFP8_E5M2 ? Fp8Out<SFP8_E5M2>::kMax : Fp8Out<SFP8_E4M3>::kMax;
}

// Sum (or maximum) over the TPR threads of a row group; every thread gets it.
// `red` holds one slot of TPR / 32 values per use, so that a group needs one
// barrier a reduction.  With TPR > 32 the group is the whole block.
template <int TPR, bool kMax>
__device__ __forceinline__ float norm_reduce(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float t = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, t) : v + t;
  }
  if constexpr (TPR > 32) {
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    // every warp adds the partial values itself, in the same order
    const int lane = threadIdx.x % 32;
    v = lane < TPR / 32 ? red[lane] : 0.0f;   // maxima here are of magnitudes
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float t = __shfl_xor_sync(0xffffffffu, v, o);
      v = kMax ? fmaxf(v, t) : v + t;
    }
  }
  return v;
}

// One row per group of TPR threads, in registers.
template <typename T, int VEC, int TPR, int N, bool Q>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256)
    layernorm_kernel(const NormParams p) {
  static_assert(TPR == 32 || TPR >= 128, "a warp, or a whole block");
  constexpr int kGroups = TPR == 32 ? 8 : 1;   // rows per block
  __shared__ float red[3][32];
  grid_dependents_launch();
  grid_dependency_wait();
  const int t = threadIdx.x % TPR;
  const long long row = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / TPR;
  if (row >= p.rows) return;    // whole groups only
  const T* xr = static_cast<const T*>(p.x) + row * p.ld_x;
  NormVec<T, VEC> in[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * TPR + t) * VEC;
    if (c < p.cols) in[i].load(xr + c);
  }
  float v[N][VEC];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if ((i * TPR + t) * VEC < p.cols) {
      in[i].floats(v[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum += v[i][j];
    }
  }
  const float inv = 1.0f / static_cast<float>(p.cols);
  const float mean = norm_reduce<TPR, false>(sum, red[0]) * inv;
  float dev = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if ((i * TPR + t) * VEC < p.cols) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i][j] -= mean;
        dev = fmaf(v[i][j], v[i][j], dev);
      }
    }
  }
  const float rstd = __frsqrt_rn(fmaf(norm_reduce<TPR, false>(dev, red[1]), inv, p.eps));
  if (t == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
  float amax = 0.0f;
  T* yr = static_cast<T*>(p.y) + row * p.cols;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * TPR + t) * VEC;
    if (c < p.cols) {
      float w[VEC], b[VEC];
      norm_params<T, VEC>(p.weight, p.params_f32, c, 1.0f, w);
      norm_params<T, VEC>(p.bias, p.params_f32, c, 0.0f, b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i][j] = fmaf(v[i][j] * rstd, w[j], b[j]);
        if (Q) amax = fmaxf(amax, fabsf(v[i][j]));
      }
      if (p.y != nullptr) norm_store<T, VEC>(yr + c, v[i]);
    }
  }
  if constexpr (Q) {
    amax = norm_reduce<TPR, true>(amax, red[2]);
    const float s = __fdiv_rn(fmaxf(amax, kGuardAmax), norm_fp8_max(p.q_fmt));
    const float r = __frcp_rn(s);
    if (t == 0) p.scales[row] = s;
    uint8_t* qr = p.q + row * p.cols;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (c < p.cols) norm_codes<VEC>(qr + c, v[i], s, r, p.q_fmt);
    }
  }
}

// Rows of any length, one per block: every sweep reads the row again.
template <typename T, int VEC, bool Q>
__global__ void __launch_bounds__(1024)
    layernorm_long_kernel(const NormParams p) {
  __shared__ float red[3][32];
  grid_dependents_launch();
  grid_dependency_wait();
  const long long row = blockIdx.x;
  const T* xr = static_cast<const T*>(p.x) + row * p.ld_x;
  const long long cols = p.cols;
  const long long c0 = static_cast<long long>(threadIdx.x) * VEC;
  NormVec<T, VEC> in;
  float f[VEC], w[VEC], b[VEC];
  float sum = 0.0f;
  for (long long c = c0; c < cols; c += 1024 * VEC) {
    in.load(xr + c);
    in.floats(f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum += f[j];
  }
  const float inv = 1.0f / static_cast<float>(p.cols);
  const float mean = norm_reduce<1024, false>(sum, red[0]) * inv;
  float dev = 0.0f;
  for (long long c = c0; c < cols; c += 1024 * VEC) {
    in.load(xr + c);
    in.floats(f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) dev = fmaf(f[j] - mean, f[j] - mean, dev);
  }
  const float rstd = __frsqrt_rn(fmaf(norm_reduce<1024, false>(dev, red[1]), inv, p.eps));
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
  float amax = 0.0f;
  auto values = [&](long long c) {
    in.load(xr + c);
    in.floats(f);
    norm_params<T, VEC>(p.weight, p.params_f32, static_cast<int>(c), 1.0f, w);
    norm_params<T, VEC>(p.bias, p.params_f32, static_cast<int>(c), 0.0f, b);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = fmaf((f[j] - mean) * rstd, w[j], b[j]);
  };
  T* yr = static_cast<T*>(p.y) + row * cols;
  for (long long c = c0; c < cols; c += 1024 * VEC) {
    values(c);
    if (p.y != nullptr) norm_store<T, VEC>(yr + c, f);
    if (Q) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) amax = fmaxf(amax, fabsf(f[j]));
    }
  }
  if constexpr (Q) {
    amax = norm_reduce<1024, true>(amax, red[2]);
    const float s = __fdiv_rn(fmaxf(amax, kGuardAmax), norm_fp8_max(p.q_fmt));
    const float r = __frcp_rn(s);
    if (threadIdx.x == 0) p.scales[row] = s;
    for (long long c = c0; c < cols; c += 1024 * VEC) {
      values(c);
      norm_codes<VEC>(p.q + row * cols + c, f, s, r, p.q_fmt);
    }
  }
}

// ------------------------------------------------------------------ backward

// Both sums over the row group; `red` alternates between two sets by row, so
// that one barrier a row is enough (a thread is at most one barrier behind).
template <int TPR>
__device__ __forceinline__ float2 norm_reduce2(float2 v, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (TPR > 32) {
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    const int lane = threadIdx.x % 32;
    v = lane < TPR / 32 ? red[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
  }
  return v;
}

template <typename T, int VEC, int TPR, int N>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256)
    layernorm_backward_kernel(const NormGradParams p) {
  static_assert(TPR == 32 || TPR >= 128, "a warp, or a whole block");
  constexpr int kGroups = TPR == 32 ? 8 : 1;
  __shared__ float2 red[2][32];
  grid_dependents_launch();
  grid_dependency_wait();
  const int t = threadIdx.x % TPR;
  const int group = blockIdx.x * kGroups + threadIdx.x / TPR;
  if (group >= p.groups) return;
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  float w[N][VEC], dw[N][VEC], db[N][VEC];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * TPR + t) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[i][j] = dw[i][j] = db[i][j] = 0.0f;
    if (c < p.cols) norm_params<T, VEC>(p.weight, p.params_f32, c, 1.0f, w[i]);
  }
  const float inv = 1.0f / static_cast<float>(p.cols);
  NormVec<T, VEC> xv[N], dv[N];
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](long long row, NormVec<T, VEC> (&xa)[N], NormVec<T, VEC> (&da)[N], float& mn,
                   float& rs) {
    mn = p.mean[row];
    rs = p.rstd[row];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (c < p.cols) {
        xa[i].load(x + row * p.ld_x + c);
        da[i].load(dy + row * p.ld_dy + c);
      }
    }
  };
  long long row = group;
  if (row < p.rows) fetch(row, xv, dv, mean, rstd);
  for (int it = 0; row < p.rows; row += p.groups, ++it) {
    // the next row's loads, under this row's reduction
    NormVec<T, VEC> xn[N], dn[N];
    float mean_n = 0.0f, rstd_n = 0.0f;
    if (row + p.groups < p.rows) fetch(row + p.groups, xn, dn, mean_n, rstd_n);
    float xh[N][VEC], g[N][VEC];
    float2 sums = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if ((i * TPR + t) * VEC < p.cols) {
        xv[i].floats(xh[i]);
        dv[i].floats(g[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xh[i][j] = (xh[i][j] - mean) * rstd;
          dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
          db[i][j] += g[i][j];
          g[i][j] *= w[i][j];
          sums.x += g[i][j];
          sums.y = fmaf(g[i][j], xh[i][j], sums.y);
        }
      }
    }
    sums = norm_reduce2<TPR>(sums, red[it & 1]);
    const float a = sums.x * inv, b = sums.y * inv;
    if (p.dx != nullptr) {
      T* out = static_cast<T*>(p.dx) + row * p.cols;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * TPR + t) * VEC;
        if (c < p.cols) {
          float d[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) d[j] = rstd * (g[i][j] - a - xh[i][j] * b);
          norm_store<T, VEC>(out + c, d);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      xv[i] = xn[i];
      dv[i] = dn[i];
    }
    mean = mean_n;
    rstd = rstd_n;
  }
  float* part = p.partial + static_cast<long long>(group) * 2 * p.cols;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * TPR + t) * VEC;
    if (c < p.cols) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        part[c + j] = dw[i][j];
        part[p.cols + c + j] = db[i][j];
      }
    }
  }
}

// Rows of any length: dx with two sweeps of the row, one row per block.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024)
    layernorm_backward_long_kernel(const NormGradParams p) {
  __shared__ float2 red[32];
  grid_dependents_launch();
  grid_dependency_wait();
  const long long row = blockIdx.x;
  const T* xr = static_cast<const T*>(p.x) + row * p.ld_x;
  const T* dr = static_cast<const T*>(p.dy) + row * p.ld_dy;
  const float mean = p.mean[row], rstd = p.rstd[row];
  const long long cols = p.cols;
  NormVec<T, VEC> xv, dv;
  float xh[VEC], g[VEC], w[VEC];
  auto values = [&](long long c) {
    xv.load(xr + c);
    dv.load(dr + c);
    xv.floats(xh);
    dv.floats(g);
    norm_params<T, VEC>(p.weight, p.params_f32, static_cast<int>(c), 1.0f, w);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      xh[j] = (xh[j] - mean) * rstd;
      g[j] *= w[j];
    }
  };
  float2 sums = make_float2(0.0f, 0.0f);
  for (long long c = static_cast<long long>(threadIdx.x) * VEC; c < cols; c += 1024 * VEC) {
    values(c);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      sums.x += g[j];
      sums.y = fmaf(g[j], xh[j], sums.y);
    }
  }
  sums = norm_reduce2<1024>(sums, red);
  const float inv = 1.0f / static_cast<float>(p.cols);
  const float a = sums.x * inv, b = sums.y * inv;
  T* out = static_cast<T*>(p.dx) + row * cols;
  for (long long c = static_cast<long long>(threadIdx.x) * VEC; c < cols; c += 1024 * VEC) {
    values(c);
#pragma unroll
    for (int j = 0; j < VEC; ++j) g[j] = rstd * (g[j] - a - xh[j] * b);
    norm_store<T, VEC>(out + c, g);
  }
}

// ... and the column sums of dy and dy * xh: block (x, y) takes 32 columns
// and the rows of run y, 8 row lanes.
template <typename T>
__global__ void __launch_bounds__(256)
    layernorm_backward_columns_kernel(const NormGradParams p) {
  __shared__ float2 sums[8][32];
  grid_dependents_launch();
  grid_dependency_wait();
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  const long long col = static_cast<long long>(blockIdx.x) * 32 + tx;
  const long long r0 = p.rows * blockIdx.y / gridDim.y, r1 = p.rows * (blockIdx.y + 1) / gridDim.y;
  float2 s = make_float2(0.0f, 0.0f);
  if (col < p.cols) {
    const T* x = static_cast<const T*>(p.x) + col;
    const T* dy = static_cast<const T*>(p.dy) + col;
    for (long long r = r0 + ty; r < r1; r += 8) {
      NormVec<T, 1> xv, dv;
      float xf[1], df[1];
      xv.load(x + r * p.ld_x);
      dv.load(dy + r * p.ld_dy);
      xv.floats(xf);
      dv.floats(df);
      s.x = fmaf(df[0], (xf[0] - p.mean[r]) * p.rstd[r], s.x);
      s.y += df[0];
    }
  }
  sums[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && col < p.cols) {
    for (int j = 1; j < 8; ++j) {
      s.x += sums[j][tx].x;
      s.y += sums[j][tx].y;
    }
    float* part = p.partial + static_cast<long long>(blockIdx.y) * 2 * p.cols;
    part[col] = s.x;
    part[p.cols + col] = s.y;
  }
}

// dweight and dbias: the groups' partial sums added in order, 32 columns a
// block, each of 8 row lanes adding every eighth group.
__global__ void __launch_bounds__(256)
    layernorm_backward_join_kernel(const float* __restrict__ partial, int groups, int cols,
                                   float* __restrict__ dweight, float* __restrict__ dbias) {
  __shared__ float sums[8][32];
  grid_dependents_launch();
  grid_dependency_wait();
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  const long long col = static_cast<long long>(blockIdx.x) * 32 + tx;   // of 2 * cols
  float s = 0.0f;
  if (col < 2ll * cols) {
#pragma unroll 8
    for (int g = ty; g < groups; g += 8) s += partial[g * 2ll * cols + col];
  }
  sums[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && col < 2ll * cols) {
    for (int j = 1; j < 8; ++j) s += sums[j][tx];
    if (col < cols) {
      if (dweight != nullptr) dweight[col] = s;
    } else if (dbias != nullptr) {
      dbias[col - cols] = s;
    }
  }
}

}  // namespace sfp8

// Layer norm, forward (to the activation's type and/or straight to row-wise
// FP8 codes) and backward (with the sums over rows of the weight's and bias's
// gradients).
//
//   forward   mean = sum_c x / C,   var = sum_c (x - mean)^2 / C
//             rstd = 1 / sqrt(var + eps)
//             y    = (x - mean) * rstd * weight + bias
//             s    = max(max_c |y|, 1e-12) / FP8_MAX,  q = fp8(y * (1 / s))
//   backward  xh = (x - mean) * rstd,  g = weight * dy
//             dx = rstd * (g - sum_c g / C - xh * sum_c (g xh) / C)
//             dweight = sum_rows dy * xh,   dbias = sum_rows dy
//
// All of it in fp32; y and dx are rounded once to x's type, the codes once
// from the fp32 y (multiplied by the rounded reciprocal of s, where the
// quantiser of a given tensor divides: the fp32 y is itself a few roundings
// off, so the quotient's last bit decides nothing).  The variance is taken
// about the mean (two reductions over values held in registers), never as a
// difference of two sums.
//
// Both passes are bound by memory.  Kernels by row length and count:
//   row kernel     few rows (or short ones): one row per group of TPR threads,
//                  N vectors of VEC elements each in registers, reduced by
//                  warp shuffles and, for more than one warp, shared memory.
//   stream kernel  rows of 1 to 16 KB, forward where there are many, backward
//                  any number: one persistent block a SM with two to fifteen
//                  row groups of 64 to 256 threads.  Each group
//                  has a ring of row buffers in shared memory that bulk
//                  copies keep filled ahead, so that HBM streams through the
//                  reductions' barriers; the parameters lie in shared memory
//                  as fp32.  What is left to be short of is instructions and
//                  the latency of the reductions (a row per 256 threads in
//                  scalar arithmetic issued 28 million warp instructions for
//                  8192 rows of 4096 bf16 and took 47 us to codes): hence
//                  packed fp32 pairs and few, wide threads a row.  8192 x
//                  4096 bf16: 26 us to codes (3.9 TB/s), 26 us to bf16 (5.2
//                  TB/s; 28 us with 128 threads a row), 43 us backward (4.7
//                  TB/s).
//   long kernels   rows that fit neither read them again from L2.
// VEC elements make 16 bytes where base, row stride and width allow, else 1.
//
// The backward kernels are persistent too: a group of threads walks rows,
// keeps its columns' dweight and dbias sums in registers and writes one
// partial sum per group at the end; a second kernel adds the groups in order
// (no atomics: the same bits every time).
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

// Codes of VEC values (VEC 4 or 8) times r at q.
template <int VEC>
__device__ __forceinline__ void norm_codes(uint8_t* q, const float (&f)[VEC], float r, int fmt) {
  uint32_t w[VEC / 4];
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) {
    const float* v = &f[4 * i];
    w[i] = fmt == SFP8_E5M2
               ? cvt_pair<SFP8_E5M2>(v[0] * r, v[1] * r) |
                     (cvt_pair<SFP8_E5M2>(v[2] * r, v[3] * r) << 16)
               : cvt_pair<SFP8_E4M3>(v[0] * r, v[1] * r) |
                     (cvt_pair<SFP8_E4M3>(v[2] * r, v[3] * r) << 16);
  }
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
      if (c < p.cols) norm_codes<VEC>(qr + c, v[i], r, p.q_fmt);
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
      norm_codes<VEC>(p.q + row * cols + c, f, r, p.q_fmt);
    }
  }
}

// ------------------------------------------------------------------ row ring

constexpr int kNormMaxSlots = 8;

// Ring of row buffers of a row group: its rows go through the slots in turn
// (`PARTS` rows of `bytes` each, from as many tensors), the group's position
// kept as a slot and that slot's phase.  One thread fills; the waits are
// bounded, and after one has run out (the status word says so) the others give
// up at once and the group runs through on whatever the buffers hold.
template <int PARTS>
struct NormRing {
  uint8_t* base;
  uint64_t* full;
  volatile int* abort;
  uint32_t bytes;     // of one row, a multiple of 16
  int slots;
  int at = 0;         // the current row's slot
  uint32_t phase = 0; // and its barrier's phase
  __device__ uint8_t* buffer(int slot) const {
    return base + static_cast<size_t>(slot) * PARTS * bytes;
  }
  // A row from a (and b) into `slot`, whose previous row every thread has
  // finished with.
  __device__ void fill(int slot, const void* a, const void* b) const {
    const uint32_t bar = smem_u32(&full[slot]);
    // x and dy are read again by others (a residual addition, the backward pass)
    const uint64_t pol = l2_policy_evict_normal();
    uint8_t* dst = buffer(slot);
    mbar_arrive_expect_tx(bar, PARTS * bytes);
    bulk_load(smem_u32(dst), a, bytes, bar, pol);
    if (PARTS == 2) bulk_load(smem_u32(dst + bytes), b, bytes, bar, pol);
  }
  __device__ void wait() const { mbar_wait(smem_u32(&full[at]), phase, abort); }
  __device__ int before() const { return at == 0 ? slots - 1 : at - 1; }
  __device__ void advance() {
    if (++at == slots) {
      at = 0;
      phase ^= 1u;
    }
  }
  // One thread, after the group's `rows` rows: where waits were given up, lets
  // the copies still in flight land (again with a limit) before the block
  // goes on to reuse or leave its shared memory.
  __device__ void drain(long long rows) const {
    if (!*abort) return;
    for (long long i = rows > slots ? rows - slots : 0; i < rows; ++i) {
      volatile int no_abort = 0;
      mbar_wait(smem_u32(&full[i % slots]), static_cast<uint32_t>((i / slots) & 1), &no_abort);
    }
  }
};

// VEC elements at p as pairs of floats.
template <typename T, int VEC>
__device__ __forceinline__ void load_pairs(const T* p, float2 (&f)[VEC / 2]) {
  NormVec<T, VEC> v;
  v.load(p);
  float t[VEC];
  v.floats(t);
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) f[j] = make_float2(t[2 * j], t[2 * j + 1]);
}

// Parameters in shared memory: fp32, the first four of every vector's VEC in
// one plane, the other four in the next, so that neighbouring threads read
// neighbouring 16 bytes.
template <int VEC>
__device__ __forceinline__ void shared_pairs(const float* plane, int vec, int cols,
                                             float2 (&f)[VEC / 2]) {
#pragma unroll
  for (int j = 0; j < VEC / 4; ++j) {
    const float4 t = *reinterpret_cast<const float4*>(plane + j * (cols / (VEC / 4)) + 4 * vec);
    f[2 * j] = make_float2(t.x, t.y);
    f[2 * j + 1] = make_float2(t.z, t.w);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void params_to_shared(const void* p, int f32, float missing, int cols,
                                                 float* plane) {
  for (int v = threadIdx.x; v < cols / VEC; v += blockDim.x) {
    float w[VEC];
    norm_params<T, VEC>(p, f32, v * VEC, missing, w);
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j)
      *reinterpret_cast<float4*>(plane + j * (cols / (VEC / 4)) + 4 * v) =
          make_float4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  }
}

__device__ __forceinline__ float2 pair_of(float v) { return make_float2(v, v); }

// Sum (or maximum of magnitudes) over a row group of TPR threads, with one
// barrier of the group's own; `red` holds one value a warp and is not written
// again before the group's next barrier.
template <int TPR, bool kMax>
__device__ __forceinline__ float group_reduce(float v, float* red, int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float t = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, t) : v + t;
  }
  if (threadIdx.x % 32 == 0) red[threadIdx.x % TPR / 32] = v;
  named_barrier_sync(1 + group, TPR);
  v = red[0];
#pragma unroll
  for (int i = 1; i < TPR / 32; ++i) v = kMax ? fmaxf(v, red[i]) : v + red[i];
  return v;
}

// Shared memory of a stream kernel: the parameters (`params` vectors of
// `cols` floats), then the groups' rings.
__host__ __device__ constexpr int norm_stream_smem(int groups, int params, int cols, int parts,
                                                   int row_bytes, int slots) {
  return params * cols * 4 + groups * slots * parts * row_bytes;
}

// N vectors of VEC elements a thread: cols <= TPR * N * VEC, a multiple of VEC;
// FULL: cols is all of that (a power of two, as most widths are), so that no
// vector needs a test (8192 x 4096 bf16 to codes: 26 us against 29).
template <typename T, int VEC, int TPR, int N, int THREADS, bool Q, bool FULL>
__global__ void __launch_bounds__(THREADS, 1)
    layernorm_stream_kernel(const NormParams p, int slots) {
  extern __shared__ __align__(128) uint8_t norm_smem[];
  static_assert(THREADS % TPR == 0, "whole row groups");
  constexpr int kGroups = THREADS / TPR;
  __shared__ uint64_t full[kGroups][kNormMaxSlots];
  __shared__ int abort_flag;
  __shared__ float red[kGroups][3][TPR / 32];
  grid_dependents_launch();
  const int group = threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  float* w_sm = reinterpret_cast<float*>(norm_smem);
  float* b_sm = w_sm + p.cols;
  const uint32_t bytes = static_cast<uint32_t>(p.cols * sizeof(T));
  NormRing<1> ring{norm_smem + 8ll * p.cols + static_cast<size_t>(group) * slots * bytes,
                   full[group], &abort_flag, bytes, slots};
  if (threadIdx.x == 0) {
    for (int g = 0; g < kGroups; ++g)
      for (int s = 0; s < slots; ++s) mbar_init(smem_u32(&full[g][s]), 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dependency_wait();
  const T* x = static_cast<const T*>(p.x);
  const long long first = static_cast<long long>(blockIdx.x) * kGroups + group;
  const long long stride = static_cast<long long>(gridDim.x) * kGroups;
  if (t == 0) {
    long long row = first;
    for (int s = 0; s < slots && row < p.rows; ++s, row += stride)
      ring.fill(s, x + row * p.ld_x, nullptr);
  }
  params_to_shared<T, VEC>(p.weight, p.params_f32, 1.0f, p.cols, w_sm);
  params_to_shared<T, VEC>(p.bias, p.params_f32, 0.0f, p.cols, b_sm);
  __syncthreads();
  const float inv = 1.0f / static_cast<float>(p.cols);
  for (long long row = first; row < p.rows; row += stride, ring.advance()) {
    ring.wait();
    const T* xr = reinterpret_cast<const T*>(ring.buffer(ring.at));
    float2 v[N][VEC / 2];
    float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (FULL || c < p.cols) {
        load_pairs<T, VEC>(xr + c, v[i]);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) acc = __fadd2_rn(acc, v[i][j]);
      }
    }
    const float mean = group_reduce<TPR, false>(acc.x + acc.y, red[group][0], group) * inv;
    // past the barrier every thread of the group has its part in registers
    if (t == 0 && row + slots * stride < p.rows)
      ring.fill(ring.at, x + (row + slots * stride) * p.ld_x, nullptr);
    acc = make_float2(0.0f, 0.0f);
    const float2 shift = pair_of(-mean);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (FULL || (i * TPR + t) * VEC < p.cols) {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          v[i][j] = __fadd2_rn(v[i][j], shift);
          acc = __ffma2_rn(v[i][j], v[i][j], acc);
        }
      }
    }
    const float dev = group_reduce<TPR, false>(acc.x + acc.y, red[group][1], group);
    const float rstd = __frsqrt_rn(fmaf(dev, inv, p.eps));
    if (t == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    float amax = 0.0f;
    const float2 scale = pair_of(rstd);
    T* yr = static_cast<T*>(p.y) + row * p.cols;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (FULL || c < p.cols) {
        float2 w[VEC / 2], b[VEC / 2];
        shared_pairs<VEC>(w_sm, i * TPR + t, p.cols, w);
        shared_pairs<VEC>(b_sm, i * TPR + t, p.cols, b);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          float2& o = v[i][j];
          o = __ffma2_rn(__fmul2_rn(o, scale), w[j], b[j]);
          if (Q) amax = fmaxf(fmaxf(amax, fabsf(o.x)), fabsf(o.y));
        }
        if (p.y != nullptr) {
          float f[VEC];
#pragma unroll
          for (int j = 0; j < VEC / 2; ++j) {
            f[2 * j] = v[i][j].x;
            f[2 * j + 1] = v[i][j].y;
          }
          norm_store<T, VEC>(yr + c, f);
        }
      }
    }
    if constexpr (Q) {
      amax = group_reduce<TPR, true>(amax, red[group][2], group);
      uint8_t* qr = p.q + row * p.cols;
      auto codes = [&](auto fmt) {
        constexpr int kFmt = decltype(fmt)::value;
        const float s = __fdiv_rn(fmaxf(amax, kGuardAmax), Fp8Out<kFmt>::kMax);
        const float2 r = pair_of(__frcp_rn(s));
        if (t == 0) p.scales[row] = s;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = (i * TPR + t) * VEC;
          if (FULL || c < p.cols) {
            uint32_t o[VEC / 4];
#pragma unroll
            for (int j = 0; j < VEC / 4; ++j) {
              const float2 lo = __fmul2_rn(v[i][2 * j], r), hi = __fmul2_rn(v[i][2 * j + 1], r);
              o[j] = cvt_pair<kFmt>(lo.x, lo.y) | (cvt_pair<kFmt>(hi.x, hi.y) << 16);
            }
            store_codes<VEC>(qr + c, o);
          }
        }
      };
      if (p.q_fmt == SFP8_E5M2) codes(std::integral_constant<int, SFP8_E5M2>{});
      else codes(std::integral_constant<int, SFP8_E4M3>{});
    }
  }
  if (t == 0 && first < p.rows) ring.drain((p.rows - first + stride - 1) / stride);
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

// The sums over the C columns in 64 bits, for the narrow form.
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// NARROW, rows of up to 32 columns: dx is computed in 64 bits.  What is left of g
// once its mean and its part along xh are taken out can be far smaller than g: of
// two columns 1 - xh^2 = eps rstd^2, 1e-5 of the terms, where fp32 terms left
// three to six digits of an fp32 dx (7 rows of 2: off by 2.4e-4 in the norm, now
// 1.6e-8).  A row takes a warp, not the block of 128 threads of wider rows, so it
// is no slower: 3000 x 2 fp32 9.2 -> 7.2 us, 100000 x 31 129 -> 47 us.
template <typename T, int VEC, int TPR, int N, bool NARROW = false>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256)
    layernorm_backward_kernel(const NormGradParams p) {
  static_assert(TPR == 32 || TPR >= 128, "a warp, or a whole block");
  static_assert(!NARROW || TPR == 32, "narrow rows: a warp each");
  using Wide = std::conditional_t<NARROW, double, float>;
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
    Wide xh[N][VEC], g[N][VEC];
    Wide sum_g = 0, sum_gx = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if ((i * TPR + t) * VEC < p.cols) {
        float xf[VEC], df[VEC];
        xv[i].floats(xf);
        dv[i].floats(df);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xh[i][j] = (static_cast<Wide>(xf[j]) - mean) * rstd;
          dw[i][j] = fmaf(df[j], static_cast<float>(xh[i][j]), dw[i][j]);
          db[i][j] += df[j];
          g[i][j] = static_cast<Wide>(df[j]) * w[i][j];
          sum_g += g[i][j];
          sum_gx = fma(g[i][j], xh[i][j], sum_gx);
        }
      }
    }
    Wide a, b;
    if constexpr (NARROW) {
      a = warp_sum(sum_g) / p.cols;
      b = warp_sum(sum_gx) / p.cols;
    } else {
      const float2 sums = norm_reduce2<TPR>(make_float2(sum_g, sum_gx), red[it & 1]);
      a = sums.x * inv;
      b = sums.y * inv;
    }
    if (p.dx != nullptr) {
      T* out = static_cast<T*>(p.dx) + row * p.cols;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * TPR + t) * VEC;
        if (c < p.cols) {
          float d[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            d[j] = static_cast<float>(rstd * (g[i][j] - a - xh[i][j] * b));
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

// Stream form: x and dy of a row come through the ring and are read from it
// twice, before the reduction (the sums) and after it (dx), which leaves the
// registers to the running sums.  A slot is refilled after the next row's
// barrier, when every thread has finished with it.  With c = x - mean:
//     sums      A = sum g / C,   B = rstd * sum (g c) / C
//     dx        = g rstd - A rstd - c (B rstd^2)
// FULL: as in the forward kernel (8192 x 4096 bf16: 3 % faster).
// At the end the block adds its groups' sums in group order: one partial sum
// a block.
template <typename T, int VEC, int TPR, int N, int THREADS, bool FULL>
__global__ void __launch_bounds__(THREADS, 1)
    layernorm_backward_stream_kernel(const NormGradParams p, int slots) {
  extern __shared__ __align__(128) uint8_t norm_smem[];
  static_assert(THREADS % TPR == 0, "whole row groups");
  constexpr int kGroups = THREADS / TPR;
  __shared__ uint64_t full[kGroups][kNormMaxSlots];
  __shared__ int abort_flag;
  // two sets, by row: a thread is at most one barrier behind
  __shared__ __align__(16) float2 red[kGroups][2][TPR / 32];
  grid_dependents_launch();
  const int group = threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  float* w_sm = reinterpret_cast<float*>(norm_smem);
  const uint32_t bytes = static_cast<uint32_t>(p.cols * sizeof(T));
  uint8_t* rings = norm_smem + 4ll * p.cols;
  NormRing<2> ring{rings + static_cast<size_t>(group) * slots * 2 * bytes, full[group],
                   &abort_flag, bytes, slots};
  if (threadIdx.x == 0) {
    for (int g = 0; g < kGroups; ++g)
      for (int s = 0; s < slots; ++s) mbar_init(smem_u32(&full[g][s]), 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dependency_wait();
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  const long long first = static_cast<long long>(blockIdx.x) * kGroups + group;
  const long long stride = static_cast<long long>(gridDim.x) * kGroups;
  if (t == 0) {
    long long row = first;
    for (int s = 0; s < slots && row < p.rows; ++s, row += stride)
      ring.fill(s, x + row * p.ld_x, dy + row * p.ld_dy);
  }
  params_to_shared<T, VEC>(p.weight, p.params_f32, 1.0f, p.cols, w_sm);
  __syncthreads();
  float2 dw[N][VEC / 2], db[N][VEC / 2];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) dw[i][j] = db[i][j] = make_float2(0.0f, 0.0f);
  const float inv = 1.0f / static_cast<float>(p.cols);
  int turn = 0;    // alternates by row
  float mean = 0.0f, rstd = 0.0f;
  if (first < p.rows) {
    mean = p.mean[first];
    rstd = p.rstd[first];
  }
  for (long long row = first; row < p.rows; row += stride, ring.advance(), turn ^= 1) {
    float mean_n = 0.0f, rstd_n = 0.0f;
    if (row + stride < p.rows) {
      mean_n = p.mean[row + stride];
      rstd_n = p.rstd[row + stride];
    }
    ring.wait();
    const T* xr = reinterpret_cast<const T*>(ring.buffer(ring.at));
    const T* dr = xr + p.cols;
    const float2 shift = pair_of(-mean), scale = pair_of(rstd);
    float2 sg = make_float2(0.0f, 0.0f), sgc = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (FULL || c < p.cols) {
        float2 xc[VEC / 2], d[VEC / 2], w[VEC / 2];
        load_pairs<T, VEC>(xr + c, xc);
        load_pairs<T, VEC>(dr + c, d);
        shared_pairs<VEC>(w_sm, i * TPR + t, p.cols, w);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          xc[j] = __fadd2_rn(xc[j], shift);
          dw[i][j] = __ffma2_rn(d[j], __fmul2_rn(xc[j], scale), dw[i][j]);
          db[i][j] = __fadd2_rn(db[i][j], d[j]);
          const float2 g = __fmul2_rn(d[j], w[j]);
          sg = __fadd2_rn(sg, g);
          sgc = __ffma2_rn(g, xc[j], sgc);
        }
      }
    }
    float2 sums = make_float2(sg.x + sg.y, sgc.x + sgc.y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sums.x += __shfl_xor_sync(0xffffffffu, sums.x, o);
      sums.y += __shfl_xor_sync(0xffffffffu, sums.y, o);
    }
    float2(&rd)[TPR / 32] = red[group][turn];
    if (t % 32 == 0) rd[t / 32] = sums;
    named_barrier_sync(1 + group, TPR);
    // the group has finished with the previous row: refill its slot
    if (t == 0 && row != first && row + (slots - 1) * stride < p.rows) {
      const long long next = row + (slots - 1) * stride;
      ring.fill(ring.before(), x + next * p.ld_x, dy + next * p.ld_dy);
    }
    if (p.dx != nullptr) {
      float2 total = rd[0];
#pragma unroll
      for (int i = 1; i < TPR / 32; ++i) total = __fadd2_rn(total, rd[i]);
      const float a = total.x * inv, b = total.y * inv * rstd;
      const float2 ka = pair_of(-a * rstd), kb = pair_of(-b * rstd * rstd);
      T* out = static_cast<T*>(p.dx) + row * p.cols;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * TPR + t) * VEC;
        if (FULL || c < p.cols) {
          float2 xc[VEC / 2], d[VEC / 2], w[VEC / 2];
          load_pairs<T, VEC>(xr + c, xc);
          load_pairs<T, VEC>(dr + c, d);
          shared_pairs<VEC>(w_sm, i * TPR + t, p.cols, w);
          float f[VEC];
#pragma unroll
          for (int j = 0; j < VEC / 2; ++j) {
            const float2 u = __ffma2_rn(__fmul2_rn(d[j], w[j]), scale, ka);
            const float2 o = __ffma2_rn(__fadd2_rn(xc[j], shift), kb, u);
            f[2 * j] = o.x;
            f[2 * j + 1] = o.y;
          }
          norm_store<T, VEC>(out + c, f);
        }
      }
    }
    mean = mean_n;
    rstd = rstd_n;
  }
  if (t == 0 && first < p.rows) ring.drain((p.rows - first + stride - 1) / stride);
  // The rings are done with (every copy has been waited for): the groups add
  // their sums into them in order.
  float* total = reinterpret_cast<float*>(rings);
  for (int g = 0; g < kGroups; ++g) {
    __syncthreads();
    if (g != group) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (!FULL && c >= p.cols) continue;
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        float2* a = reinterpret_cast<float2*>(total + c + 2 * j);
        float2* b = reinterpret_cast<float2*>(total + p.cols + c + 2 * j);
        *a = g == 0 ? dw[i][j] : __fadd2_rn(*a, dw[i][j]);
        *b = g == 0 ? db[i][j] : __fadd2_rn(*b, db[i][j]);
      }
    }
  }
  __syncthreads();
  float* part = p.partial + static_cast<long long>(blockIdx.x) * 2 * p.cols;
  for (int c = threadIdx.x * 4; c < 2 * p.cols; c += THREADS * 4)
    *reinterpret_cast<float4*>(part + c) = *reinterpret_cast<const float4*>(total + c);
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
// block, each of 32 row lanes adding every 32nd group.
__global__ void __launch_bounds__(1024)
    layernorm_backward_join_kernel(const float* __restrict__ partial, int groups, int cols,
                                   float* __restrict__ dweight, float* __restrict__ dbias) {
  __shared__ float sums[32][32];
  grid_dependents_launch();
  grid_dependency_wait();
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  const long long col = static_cast<long long>(blockIdx.x) * 32 + tx;   // of 2 * cols
  float s = 0.0f;
  if (col < 2ll * cols) {
#pragma unroll 4
    for (int g = ty; g < groups; g += 32) s += partial[g * 2ll * cols + col];
  }
  sums[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && col < 2ll * cols) {
    for (int j = 1; j < 32; ++j) s += sums[j][tx];
    if (col < cols) {
      if (dweight != nullptr) dweight[col] = s;
    } else if (dbias != nullptr) {
      dbias[col - cols] = s;
    }
  }
}

}  // namespace sfp8

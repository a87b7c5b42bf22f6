// The gated feed-forward block's part of the sparse GEMM's epilogue.
//
//     z[m, r] = acc[r, m] * s_a[m] * s_w[r] + bias[r]        (2n rows r)
//     h[m, j] = act(z[m, 2j]) * z[m, 2j + 1]                 (forward)
//     dz[m, 2j]     = dh[m, j] * z[m, 2j + 1] * act'(z[m, 2j])
//     dz[m, 2j + 1] = dh[m, j] * act(z[m, 2j])               (backward)
//
// The rows of the compressed weight alternate (gate j at row 2j, up j at
// 2j + 1), so the two products a hidden unit needs sit in neighbouring
// accumulator lanes of one warp, whatever the work split: whole tiles, CTA
// pairs and split-K finishers all end in the same 16-token chunk, and one
// shuffle with the neighbour lane pairs them.  z never leaves the registers
// and is not rounded; h is rounded once, to bf16, as it is stored.
//
// dz is stored as bf16 of dz[m, r] * s_a[m] * s_w[r].  With both scales in
// it, the FP8 codes themselves are the other operand of both gradient
// products -- exact in bf16, where the scaled weight or activation would be
// rounded once more -- and what each product has too much is constant along
// its output rows (s_a[m] in dx, s_w[r] in dw), so it is divided out of the
// fp32 sums:
//     dx[m, k] = 1 / s_a[m] * sum_r dz'[m, r] W_q[r, k]
//     dw[r, k] = 1 / s_w[r] * sum_m dz'[m, r] A_q[m, k]
// The quantisers' scales are at least 1e-12 / 57344, which keeps dz' and the
// quotients in range; where both scales are that small (an all-zero row of
// the activation against an all-zero row of the weight), dz' may lose its
// last bits, but then the codes it is multiplied with are zeros in both
// products.
//
// Of a chunk's 16 tokens the gate lane finishes tokens 0..7 and the up lane
// 8..15: each sends its neighbour the eight values that one needs (8 shuffles
// a chunk) and evaluates eight activations, instead of every gate lane
// evaluating sixteen while the up lanes idle.
#pragma once

#include <cuda_bf16.h>

#include "device_common.cuh"

namespace sfp8 {

// What the GEMM's epilogue does with a finished accumulator.
enum Epilogue : int {
  kEpiLinear = 0,      // y = z
  kEpiGated = 1,       // h = act(z gate) * z up
  kEpiGatedGrad = 2    // dz from dh and z
};

// act(g) and act'(g).  Both activations are g * p(g) with a logistic p:
// SiLU's p = sigma(g); GELU in its tanh form is g * sigma(2 q) with
// q = sqrt(2/pi) (g + 0.044715 g^3), since (1 + tanh q) / 2 = sigma(2 q) --
// which also keeps full relative accuracy where 1 + tanh q cancels.  Then
//     act = g p,   act' = p + act (1 - p) x'     (p = sigma(x))
// The approximate exponential and reciprocal err by a few 2^-22, far below
// the bf16 rounding of the result; they flush what is below 2^-126 to zero,
// and an exponential that overflows makes p zero.
//
// The epilogue's warps share the SM's issue slots with the warps that feed the
// tensor core, so it counts instructions: hence the raw forms of both, the
// branch on the activation outside the loops, and 16-token chunks that are
// known to lie inside the tensors as a whole.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// sigma(x) from -x log2(e).
__device__ __forceinline__ float logistic_exp2(float t) {
  float e, p;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(1.0f + e));
  return p;
}

template <int ACT>
__device__ __forceinline__ float act_logistic(float g) {
  if constexpr (ACT == SFP8_ACT_SILU) return logistic_exp2(-kLog2e * g);
  return logistic_exp2(-2.0f * kLog2e * kGeluC * fmaf(kGeluA * g * g, g, g));
}

template <int ACT>
__device__ __forceinline__ void act_value_grad(float g, float& f, float& df) {
  const float p = act_logistic<ACT>(g);
  f = g * p;
  const float t = f * (1.0f - p);
  if constexpr (ACT == SFP8_ACT_SILU) {
    df = p + t;
  } else {
    // where p has saturated t is zero, and x' may have overflowed
    const float dx = 2.0f * kGeluC * fmaf(3.0f * kGeluA * g, g, 1.0f);
    df = t != 0.0f ? fmaf(t, dx, p) : p;
  }
}

// h of eight gate and up values.
__device__ __forceinline__ void gated_values(const float (&g)[8], const float (&u)[8], int act,
                                             float (&h)[8]) {
  if (act == SFP8_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = g[j] * act_logistic<SFP8_ACT_SILU>(g[j]) * u[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = g[j] * act_logistic<SFP8_ACT_GELU>(g[j]) * u[j];
  }
}

// act and act' of eight gate values.
__device__ __forceinline__ void gated_slopes(const float (&g)[8], int act, float (&f)[8],
                                             float (&df)[8]) {
  if (act == SFP8_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < 8; ++j) act_value_grad<SFP8_ACT_SILU>(g[j], f[j], df[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) act_value_grad<SFP8_ACT_GELU>(g[j], f[j], df[j]);
  }
}

// z of a chunk: acc * (sa * sw) + bias, two tokens at a time.
__device__ __forceinline__ void gated_preactivation(const float (&acc)[16], const float (&sa)[16],
                                                    float sw, float bias, float (&z)[16]) {
  const float2 sw2 = make_float2(sw, sw), b2 = make_float2(bias, bias);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 t = __ffma2_rn(make_float2(acc[2 * j], acc[2 * j + 1]),
                                __fmul2_rn(make_float2(sa[2 * j], sa[2 * j + 1]), sw2), b2);
    z[2 * j] = t.x;
    z[2 * j + 1] = t.y;
  }
}

// Index of row r's bias: the caller's vector holds the n gate values, then
// the n up values.
__device__ __forceinline__ long long gated_bias_index(int r, int rows) {
  return (r & 1) ? (rows >> 1) + (r >> 1) : (r >> 1);
}

// Pairs a chunk's 16 values of this lane's row with the neighbour lane's:
// lane r even gets (gate, up) of tokens 0..7, lane r odd of tokens 8..15.
// Every lane of the warp takes part.
__device__ __forceinline__ void gated_pair_up(const float (&z)[16], bool odd, float (&g)[8],
                                              float (&u)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float mine = odd ? z[j + 8] : z[j];
    const float theirs = __shfl_xor_sync(0xffffffffu, odd ? z[j] : z[j + 8], 1);
    g[j] = odd ? theirs : mine;
    u[j] = odd ? mine : theirs;
  }
}

}  // namespace sfp8

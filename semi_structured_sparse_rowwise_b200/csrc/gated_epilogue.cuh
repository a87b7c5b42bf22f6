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
// which also keeps full relative accuracy where 1 + tanh q cancels.  The
// fast exponential and division err by a few 2^-22, far below the bf16
// rounding of the result.
__device__ __forceinline__ float logistic(float x) {
  // x -> -inf: exp overflows to inf and the quotient is 0
  return __fdividef(1.0f, 1.0f + __expf(-x));
}

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float act_value(float g, int act) {
  const float x = act == SFP8_ACT_SILU ? g : 2.0f * kGeluC * fmaf(kGeluA * g * g, g, g);
  return g * logistic(x);
}

__device__ __forceinline__ void act_value_grad(float g, int act, float& f, float& df) {
  const float g2 = g * g;
  const float x = act == SFP8_ACT_SILU ? g : 2.0f * kGeluC * fmaf(kGeluA * g2, g, g);
  const float dx = act == SFP8_ACT_SILU ? 1.0f : 2.0f * kGeluC * fmaf(3.0f * kGeluA, g2, 1.0f);
  const float p = logistic(x);
  f = g * p;
  const float d = p * (1.0f - p);
  // where p has saturated the second term is zero (dx may have overflowed)
  df = d > 0.0f ? fmaf(g * d, dx, p) : p;
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

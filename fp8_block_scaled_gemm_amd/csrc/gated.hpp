// The activation of a gated feed-forward block and its slope, in fp32, shared by the gated product's epilogue and the
// row operators.
#pragma once

#include "common.hpp"

namespace dg {

// Values of enum dg_act (include/dg.h).
enum Act : int { kSilu = 0, kGelu = 1 };

// e = exp(-z) and p = sigmoid(z) = 1 / (1 + e), by the hardware's exponential and reciprocal (each within 2 * 2^-24).  The
// rounded argument -z log2(e) makes that (1.5 |z| + 2) 2^-24 of e, so p lies within (1.5 |z| + 6) 2^-24 of its value where
// z < 0, and closer above.  p is 0 where it lies below 2^-126, e is then infinite; a NaN stays one.
__device__ __forceinline__ float sigmoid(float z, float& e) {
  e = __builtin_amdgcn_exp2f(z * -1.44269502f);
  return __builtin_amdgcn_rcpf(1.0f + e);
}

constexpr float kGeluRoot = 1.59576912f;   // 2 sqrt(2 / pi): 0.5 (1 + tanh(y)) = sigmoid(2 y)
constexpr float kGeluCube = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_arg(float g) {
  return ACT == kSilu ? g : kGeluRoot * __builtin_fmaf(kGeluCube * g * g, g, g);
}

// g sigmoid(g), or the tanh form of GELU.
template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  float e;
  return g * sigmoid(act_arg<ACT>(g), e);
}

// Value and slope: p + g p (1 - p) dz/dg, 1 - p = e p where that is small (the second term is 0, not a product with an
// infinity, where p (1 - p) is).
template <int ACT>
__device__ __forceinline__ void act_both(float g, float& value, float& slope) {
  float e;
  const float z = act_arg<ACT>(g), p = sigmoid(z, e);
  value = g * p;
  const float q = p * (z >= 0.0f ? e * p : 1.0f - p);
  const float dz = ACT == kSilu ? 1.0f : kGeluRoot * __builtin_fmaf(3.0f * kGeluCube * g, g, 1.0f);
  slope = q == 0.0f ? p : __builtin_fmaf(g * q, dz, p);
}

}  // namespace dg

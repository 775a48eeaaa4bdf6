// The activation of a gated feed-forward block and its slope, in fp32, shared by the gated product's epilogue and the
// row operators.
#pragma once

#include "common.hpp"

namespace dg {

// Values of enum dg_act (include/dg.h).
enum Act : int { kSilu = 0, kGelu = 1 };

// exp(-a) for a >= 0: 2^-(hi + lo), hi + lo = a log2(e) to twice fp32's bits (rounding a log2(e) alone would cost
// 2^-18 of the result at a = 88); within 3 * 2^-24 of its value, 0 below 2^-126; a NaN stays one.
__device__ __forceinline__ float exp_neg(float a) {
  constexpr float kLog2e = 1.44269502f, kLog2eLo = 1.92596299e-8f, kLn2 = 0.693147181f;
  const float hi = a * kLog2e;
  const float lo = __builtin_fmaf(a, kLog2eLo, __builtin_fmaf(a, kLog2e, -hi));
  const float e = __builtin_amdgcn_exp2f(-hi);
  return hi > 126.0f ? 0.0f : __builtin_fmaf(-lo * kLn2, e, e);
}

// sigmoid(z) and 1 - sigmoid(z), both to full relative precision (the hardware's reciprocal: within 2 * 2^-24).
__device__ __forceinline__ void sigmoid2(float z, float& p, float& rest) {
  const float e = exp_neg(fabsf(z));
  const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
  p = z >= 0.0f ? r : er;
  rest = z >= 0.0f ? er : r;
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
  float p, rest;
  sigmoid2(act_arg<ACT>(g), p, rest);
  return g * p;
}

// Value and slope: p + g p (1 - p) dz/dg (the second term is 0, not a product with an infinity, where p (1 - p) is).
template <int ACT>
__device__ __forceinline__ void act_both(float g, float& value, float& slope) {
  float p, rest;
  sigmoid2(act_arg<ACT>(g), p, rest);
  value = g * p;
  const float q = p * rest;
  const float dz = ACT == kSilu ? 1.0f : kGeluRoot * __builtin_fmaf(3.0f * kGeluCube * g, g, 1.0f);
  slope = q == 0.0f ? p : __builtin_fmaf(g * q, dz, p);
}

}  // namespace dg

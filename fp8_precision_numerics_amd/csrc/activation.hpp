// Activation functions of the feed-forward operators, in fp32.
//
//   relu   z > 0 ? z : 0
//   silu   z * s(z),        s(z) = 1 / (1 + exp(-z))
//   gelu   z * s(2u),       u = sqrt(2/pi) (z + 0.044715 z^3): the tanh form, with
//          (1 + tanh u) / 2 written as s(2u), which keeps its relative accuracy
//          for negative z, where 1 + tanh u cancels
//
// exp and the reciprocal are the hardware's V_EXP_F32 and V_RCP_F32 (about one
// unit in the last place each).  The exponent's argument is rounded to fp32, so
// s(x) carries a relative error of about |x| * 2^-23 for negative x (2e-6 at
// x = -16, where s(x) is 1e-7), far below the 8 or 16 bits that the results are
// rounded to.  exp overflowing to Inf gives s = 0, its limit.
#pragma once

#include "device_common.hpp"

namespace fp8mi {

enum : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

constexpr float kLog2e = 1.4426950408889634f;
constexpr double kGelu2C = 1.5957691216057308, kGeluA = 0.044715;  // 2 sqrt(2/pi)
// -2u log2(e) = z (kGeluK1 + kGeluK3 z^2)
constexpr float kGeluK1 = (float)(-1.4426950408889634 * kGelu2C);
constexpr float kGeluK3 = (float)(-1.4426950408889634 * kGelu2C * kGeluA);

// 1 / (1 + 2^x)
__device__ __forceinline__ float inv_one_plus_exp2(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x));
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActRelu) return z > 0.0f ? z : (z == z ? 0.0f : z);  // NaN stays NaN
  else if constexpr (ACT == kActSilu) return z * inv_one_plus_exp2(-kLog2e * z);
  else if constexpr (ACT == kActGelu) return z * inv_one_plus_exp2(z * __builtin_fmaf(z * z, kGeluK3, kGeluK1));
  else return z;
}

// Value and derivative together (the backward passes need both).
//   silu'  s + z s (1 - s)
//   gelu'  s + z s (1 - s) 2c (1 + 3 a z^2), s = s(2u); the polynomial is taken at
//          z clamped to [-20, 20], where s (1 - s) is already 0 in fp32, so that a
//          huge z does not make 0 * Inf out of it
template <int ACT>
__device__ __forceinline__ void act_value_slope(float z, float* value, float* slope) {
  if constexpr (ACT == kActRelu) {
    *value = z > 0.0f ? z : (z == z ? 0.0f : z);
    *slope = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActSilu) {
    const float s = inv_one_plus_exp2(-kLog2e * z), v = z * s;
    *value = v;
    *slope = s + v * (1.0f - s);
  } else if constexpr (ACT == kActGelu) {
    const float c = __builtin_amdgcn_fmed3f(z, -20.0f, 20.0f), c2 = c * c;
    const float s = inv_one_plus_exp2(c * __builtin_fmaf(c2, kGeluK3, kGeluK1)), v = z * s;
    *value = v;
    *slope = s + v * (1.0f - s) * __builtin_fmaf(c2, (float)(3.0 * kGeluA * kGelu2C), (float)kGelu2C);
  } else {
    *value = z;
    *slope = 1.0f;
  }
}

}  // namespace fp8mi

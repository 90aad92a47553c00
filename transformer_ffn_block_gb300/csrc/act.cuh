// Activations of the linear and gated forms, in fp32, and their derivatives.
//
// ACT values are those of QFFN_ACT_* (include/qffn.h).  The sigmoid is formed
// from e = exp(-|v|) in (0, 1], so neither branch overflows and the small
// values of the negative branch keep their relative accuracy.  NaN propagates;
// relu'(0) = 0.
#pragma once

#include "common.cuh"

namespace qffn {

constexpr int ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4;

QFFN_DEVI float sigmoid_f32(float v) {
  const float e = __expf(-fabsf(v));
  const float r = __fdividef(1.0f, 1.0f + e);
  return v >= 0.0f ? r : e * r;
}

constexpr float kGeluTanhScale = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluTanhCubic = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

template <int ACT>
QFFN_DEVI float act_f32(float z) {
  if (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;
  if (ACT == ACT_GELU) return z * normcdff(z);
  if (ACT == ACT_GELU_TANH)
    // 0.5 z (1 + tanh(s)) = z sigmoid(2 s)
    return z * sigmoid_f32(kGeluTanhScale * fmaf(kGeluTanhCubic * z * z, z, z));
  if (ACT == ACT_SILU) return z * sigmoid_f32(z);
  return z;
}

// Value and derivative.
template <int ACT>
QFFN_DEVI void act_grad_f32(float z, float& f, float& df) {
  if (ACT == ACT_RELU) {
    f = z < 0.0f ? 0.0f : z;
    df = z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  } else if (ACT == ACT_GELU) {
    const float p = normcdff(z);
    f = z * p;
    df = fmaf(z * kInvSqrt2Pi, __expf(-0.5f * z * z), p);
  } else if (ACT == ACT_GELU_TANH) {
    const float z2 = z * z;
    const float p = sigmoid_f32(kGeluTanhScale * fmaf(kGeluTanhCubic * z2, z, z));
    f = z * p;
    df = fmaf(f * (1.0f - p), kGeluTanhScale * fmaf(3.0f * kGeluTanhCubic, z2, 1.0f), p);
  } else if (ACT == ACT_SILU) {
    const float p = sigmoid_f32(z);
    f = z * p;
    df = p * fmaf(z, 1.0f - p, 1.0f);
  } else {
    f = z;
    df = 1.0f;
  }
}

}  // namespace qffn

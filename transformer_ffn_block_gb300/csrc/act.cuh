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

// Phi(-a) = exp(-a^2 / 2) R(a) for a >= 0, R the Mills ratio over sqrt(2 pi):
// smooth and free of cancellation, so a polynomial in t = 1 / (1 + 0.35 a)
// keeps the relative accuracy of the small values (own least-squares fit of
// degree 7, reweighted to the minimax on [0, 14]: 3e-7 relative, 6e-7 evaluated
// in fp32; beyond, the exponential underflows).  Returns Phi(z), and
// exp(-z^2 / 2) for the density.
QFFN_DEVI float normal_cdf_f32(float z, float& gauss) {
  const float a = fabsf(z);
  const float t = __fdividef(1.0f, fmaf(0.35f, a, 1.0f));
  float r = 0.0489424504339695f;
  r = fmaf(r, t, -0.20211930572986603f);
  r = fmaf(r, t, 0.24064083397388458f);
  r = fmaf(r, t, -0.01702345348894596f);
  r = fmaf(r, t, 0.15596149861812592f);
  r = fmaf(r, t, 0.13335509598255157f);
  r = fmaf(r, t, 0.14027033746242523f);
  r = fmaf(r, t, -2.7315563784213737e-05f);
  gauss = __expf(-0.5f * a * a);
  const float tail = gauss * r;
  return z < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
QFFN_DEVI float act_f32(float z) {
  if (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;
  if (ACT == ACT_GELU) {
    float gauss;
    return z * normal_cdf_f32(z, gauss);
  }
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
    float gauss;
    const float p = normal_cdf_f32(z, gauss);
    f = z * p;
    df = fmaf(z * kInvSqrt2Pi, gauss, p);
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

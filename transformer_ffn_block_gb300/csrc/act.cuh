// Activations of the linear and gated forms, in fp32, and their derivatives.
//
// ACT values are those of QFFN_ACT_* (include/qffn.h).  The sigmoid is 1 / (1 +
// exp(-v)): for negative v the sum is dominated by the exponential, so the small
// values keep their relative accuracy, and below -87 it is 0.  NaN propagates;
// relu'(0) = 0.
//
// An exponential's relative error grows with its argument, whose own rounding it
// multiplies.  Relative errors in fp32, without the approximations' own 2^-22 and
// 2^-23: the sigmoid 3e-7 for v >= -4, 9e-7 for v >= -16, 4e-6 to the end; Phi(-a)
// 7e-7 for a <= 2, 1e-6 for a <= 4, 2.3e-6 for a <= 6, 4.8e-6 for a <= 10 and 8.4e-6 for
// a <= 13, where it is 6e-39; Phi of positive values 7e-7.  (The results are
// rounded to bf16, 3.9e-3.)
#pragma once

#include "common.cuh"

namespace qffn {

constexpr int ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4;

// 2^v and 1/v by the PTX approximations, which the PTX ISA bounds at 2^-22
// (ex2.approx) and at one unit in the last place (rcp.approx); denormals flushed.
QFFN_DEVI float exp2_f32(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
QFFN_DEVI float rcp_f32(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

QFFN_DEVI float sigmoid_f32(float v) {
  return rcp_f32(1.0f + exp2_f32(-kLog2e * v));
}

constexpr float kGeluTanhScale = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluTanhCubic = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// Phi(-a) = exp(-a^2 / 2) R(a) for a >= 0, R the Mills ratio over sqrt(2 pi):
// smooth and free of cancellation, so a polynomial in t = 1 / (1 + 0.35 a)
// keeps the relative accuracy of the small values (own least-squares fit of
// degree 7, reweighted to the minimax on [0, 14]: R to 3e-7 relative, 6e-7 evaluated
// in fp32; beyond, the exponential underflows; Phi's own error: above).  Returns Phi(z), and
// exp(-z^2 / 2) for the density.
QFFN_DEVI float normal_cdf_f32(float z, float& gauss) {
  const float a = fabsf(z);
  const float t = rcp_f32(fmaf(0.35f, a, 1.0f));
  float r = 0.0489424504339695f;
  r = fmaf(r, t, -0.20211930572986603f);
  r = fmaf(r, t, 0.24064083397388458f);
  r = fmaf(r, t, -0.01702345348894596f);
  r = fmaf(r, t, 0.15596149861812592f);
  r = fmaf(r, t, 0.13335509598255157f);
  r = fmaf(r, t, 0.14027033746242523f);
  r = fmaf(r, t, -2.7315563784213737e-05f);
  gauss = exp2_f32(-0.5f * kLog2e * a * a);
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

// z within +-100, NaN as it is: there every derivative here has reached 0 or 1 in
// fp32, and beyond its terms would be 0 times infinity.
QFFN_DEVI float slope_range(float z) {
  float r;
  asm("{\n .reg .f32 t;\n max.NaN.f32 t, %1, 0fC2C80000;\n min.NaN.f32 %0, t, 0f42C80000;\n}" : "=f"(r) : "f"(z));
  return r;
}

// Value and derivative.
template <int ACT>
QFFN_DEVI void act_grad_f32(float z, float& f, float& df) {
  if (ACT == ACT_RELU) {
    f = z < 0.0f ? 0.0f : z;
    df = z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  } else if (ACT == ACT_GELU) {
    float gauss;
    const float c = slope_range(z);
    const float p = normal_cdf_f32(c, gauss);
    f = z * p;
    df = fmaf(c * kInvSqrt2Pi, gauss, p);
  } else if (ACT == ACT_GELU_TANH) {
    const float c = slope_range(z), c2 = c * c;
    const float p = sigmoid_f32(kGeluTanhScale * fmaf(kGeluTanhCubic * c2, c, c));
    f = z * p;
    df = fmaf(c * p * (1.0f - p), kGeluTanhScale * fmaf(3.0f * kGeluTanhCubic, c2, 1.0f), p);
  } else if (ACT == ACT_SILU) {
    const float c = slope_range(z);
    const float p = sigmoid_f32(c);
    f = z * p;
    df = p * fmaf(c, 1.0f - p, 1.0f);
  } else {
    f = z;
    df = 1.0f;
  }
}

// The same on pairs (f32x2).
QFFN_DEVI uint64_t f2_dup(float v) { return f2_pack(v, v); }

QFFN_DEVI uint64_t sigmoid_f2(uint64_t v) {
  float a, b, da, db;
  f2_unpack(f2_mul(f2_dup(-kLog2e), v), a, b);
  f2_unpack(f2_add(f2_dup(1.0f), f2_pack(exp2_f32(a), exp2_f32(b))), da, db);
  return f2_pack(rcp_f32(da), rcp_f32(db));
}

template <int ACT>
QFFN_DEVI uint64_t act_f2(uint64_t z) {
  if (ACT == ACT_RELU) {
    float a, b;
    f2_unpack(z, a, b);
    return f2_pack(a < 0.0f ? 0.0f : a, b < 0.0f ? 0.0f : b);
  }
  if (ACT == ACT_GELU) {
    // (its polynomial runs faster on single values than on pairs, whose constants
    // take register pairs: 8192 x 8192 x 64 with GELU 79 us on pairs, 73 so)
    float a, b;
    f2_unpack(z, a, b);
    return f2_pack(act_f32<ACT_GELU>(a), act_f32<ACT_GELU>(b));
  }
  if (ACT == ACT_GELU_TANH) {
    const uint64_t s = f2_mul(f2_dup(kGeluTanhScale), f2_fma(f2_mul(f2_mul(f2_dup(kGeluTanhCubic), z), z), z, z));
    return f2_mul(z, sigmoid_f2(s));
  }
  if (ACT == ACT_SILU) return f2_mul(z, sigmoid_f2(z));
  return z;
}

template <int ACT>
QFFN_DEVI void act_grad_f2(uint64_t z, uint64_t& f, uint64_t& df) {
  float a, b;
  f2_unpack(z, a, b);
  if (ACT == ACT_GELU_TANH) {
    const uint64_t c = f2_pack(slope_range(a), slope_range(b)), c2 = f2_mul(c, c);
    const uint64_t p = sigmoid_f2(f2_mul(f2_dup(kGeluTanhScale), f2_fma(f2_mul(f2_dup(kGeluTanhCubic), c2), c, c)));
    f = f2_mul(z, p);
    df = f2_fma(f2_mul(f2_mul(c, p), f2_sub(f2_dup(1.0f), p)),
                f2_mul(f2_dup(kGeluTanhScale), f2_fma(f2_dup(3.0f * kGeluTanhCubic), c2, f2_dup(1.0f))), p);
  } else if (ACT == ACT_SILU) {
    const uint64_t c = f2_pack(slope_range(a), slope_range(b));
    const uint64_t p = sigmoid_f2(c);
    f = f2_mul(z, p);
    df = f2_mul(p, f2_fma(c, f2_sub(f2_dup(1.0f), p), f2_dup(1.0f)));
  } else {
    float fa, fb, da, db;
    act_grad_f32<ACT>(a, fa, da);
    act_grad_f32<ACT>(b, fb, db);
    f = f2_pack(fa, fb);
    df = f2_pack(da, db);
  }
}

}  // namespace qffn

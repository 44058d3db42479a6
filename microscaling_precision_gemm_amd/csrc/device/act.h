// act.h -- activations in FP32 and their slopes.  With e(x) = e^x and
// sigmoid from exp.h:
//   relu       max(z, 0)                      slope 1 where z > 0, else 0
//   silu       z s, s = sigmoid(z)            s (1 + z (1 - s))
//   gelu       z P, P = erfc(-z / sqrt 2) / 2 P + z e(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z s, s = sigmoid(u),           s + z s (1 - s) u'
//              u = sqrt(8 / pi) (z + 0.044715 z^3), which is z (1 + tanh(u / 2)) / 2
// NaN stays NaN (relu's slope of it is 0).  At infinities the formulas are
// taken as they stand (0 times infinity is NaN).
// Relative errors, in units of 2^-24: silu 8, gelu 18, gelu_tanh 8 + 4 |u| (1 - s): u
// has four roundings, which matter where the sigmoid falls (13 units at z = -3, 33 at
// -5, 160 at -9, where the result is 1e-28; carrying u's rounding along would take
// four more instructions for digits of results that small).  Below -87.4 the
// sigmoid is 0 and so are silu and gelu_tanh (at u), whose values are under 2^-119
// there; gelu is 0 from -13.3 down, where it is subnormal.
#pragma once
#include "../launch_dense.h"
#include "exp.h"

namespace mxk {

// The lower tail of the normal distribution at -t for t >= 0, times
// e^(t^2 / 2): R(t) = e^(t^2 / 2) erfc(t / sqrt 2) / 2 falls smoothly from 1/2, so
// a polynomial in w = 1 / (1 + 0.23 t) holds it to 1.5 * 2^-24 relative on 0 .. 14
// (coefficients fitted for the smallest largest relative error, then rounded); in
// FP32 it comes to 9 * 2^-24 with its own roundings and the reciprocal's.
__device__ inline float normal_tail(float t) {
  const float w = __builtin_amdgcn_rcpf(fmaf(0.23f, t, 1.0f));
  float p = -0.0784666166f;
  p = fmaf(p, w, 0.290410101f);
  p = fmaf(p, w, -0.278118789f);
  p = fmaf(p, w, 0.301463544f);
  p = fmaf(p, w, -0.0329138525f);
  p = fmaf(p, w, 0.119511358f);
  p = fmaf(p, w, 0.0857636109f);
  p = fmaf(p, w, 0.092378363f);
  return fmaf(p, w, -2.77565487e-05f);
}

// e^(-t^2 / 2) for 0 <= t <= 14 (0 from 13.3 on): as exp_nonpos, and the rounding
// of the square, worth up to 87 * 2^-24 of the result, goes back in with the rest.
__device__ inline float normal_density(float t) {
  const float q = t * t, lo = fmaf(t, t, -q);
  const float x = -0.5f * q, p = x * kLog2e, y = __builtin_amdgcn_exp2f(p);
  return fmaf(y, fmaf(-0.5f, lo, exp_rest(x, p)), y);
}

// The sigmoid and 1 - sigmoid, both to 7 * 2^-24 relative: with y = e^-x and r =
// 1 / (1 + y) they are r and y r.  (Below -87.4 r is 0, and then so is the second:
// it only ever multiplies the first.)
__device__ inline float sigmoid_pair(float x, float* rest) {
  const float n = __builtin_amdgcn_fmed3f(-x, -150.0f, 88.0f);
  const float t = n * kLog2e, e = __builtin_amdgcn_exp2f(t);
  const float y = fmaf(e, exp_rest(n, t), e), d = 1.0f + y;
  const float r0 = __builtin_amdgcn_rcpf(d), r = fmaf(fmaf(-d, r0, 1.0f), r0, r0);
  *rest = y * r;
  return r;
}

constexpr float kGeluA = 1.59576912160573071176f;         // sqrt(8 / pi)
constexpr float kGeluB = 0.0713548162726002527220f;       // 0.044715 sqrt(8 / pi)
constexpr float kInvSqrt2Pi = 0.398942280401432677940f;

template <int ACT>
__device__ inline float act(float z) {
  if constexpr (ACT == ACT_RELU) return __builtin_elementwise_maximum(z, 0.0f);
  else if constexpr (ACT == ACT_SILU) return z * sigmoid(z);
  else if constexpr (ACT == ACT_GELU) {
    const float t = __builtin_elementwise_minimum(__builtin_fabsf(z), 14.0f);
    const float tail = normal_density(t) * normal_tail(t);
    return z * (z < 0.0f ? tail : 1.0f - tail);
  } else if constexpr (ACT == ACT_GELU_TANH) return z * sigmoid(z * fmaf(kGeluB, z * z, kGeluA));
  else return z;
}

template <int ACT>
__device__ inline float act_slope(float z) {
  if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  else if constexpr (ACT == ACT_SILU) {
    float o;
    const float s = sigmoid_pair(z, &o);
    return s * fmaf(z, o, 1.0f);
  } else if constexpr (ACT == ACT_GELU) {
    // P(-t) - t e / sqrt(2 pi) below 0, 1 minus that above
    const float t = __builtin_elementwise_minimum(__builtin_fabsf(z), 14.0f);
    const float s = normal_density(t) * fmaf(-kInvSqrt2Pi, t, normal_tail(t));
    return z < 0.0f ? s : 1.0f - s;
  } else if constexpr (ACT == ACT_GELU_TANH) {
    // beyond 12 the sigmoid is 0 or 1 and the second term nothing
    const float c = __builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -12.0f), 12.0f);
    float o;
    const float q = c * c, s = sigmoid_pair(c * fmaf(kGeluB, q, kGeluA), &o);
    return fmaf(c * s * o, fmaf(3.0f * kGeluB, q, kGeluA), s);
  } else return 1.0f;
}

// f(std::integral_constant) for the activation `a`, a uniform branch
template <class F>
__device__ inline void with_act(int a, F f) {
  switch (a) {
    case ACT_RELU: return f(std::integral_constant<int, ACT_RELU>());
    case ACT_SILU: return f(std::integral_constant<int, ACT_SILU>());
    case ACT_GELU: return f(std::integral_constant<int, ACT_GELU>());
    case ACT_GELU_TANH: return f(std::integral_constant<int, ACT_GELU_TANH>());
    default: return f(std::integral_constant<int, ACT_NONE>());
  }
}

}  // namespace mxk

// exp.h -- e^x in FP32 to 3 * 2^-24 relative for every x.  The hardware's 2^t is
// good to one unit in the last place, but t = x log2(e) has to be rounded, which
// is worth up to 64 * 2^-24 of the result at x = -87.  The rounding is known:
// with t the rounded product e^x = 2^t e^(x - t ln 2) exactly, and the second
// factor is 1 + (x - t ln 2) to 2^-30, taken by two fused steps that hold ln 2
// to 49 bits.
#pragma once
#include <hip/hip_runtime.h>

namespace mxk {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2Hi = 0.693147182464599609375f;      // ln 2 rounded to FP32,
constexpr float kLn2Lo = -1.90465429995776804525e-9f;   // and the rest of it

// x - t ln 2, for t = x log2(e) as rounded
__device__ inline float exp_rest(float x, float t) { return fmaf(t, -kLn2Lo, fmaf(t, -kLn2Hi, x)); }

// e^x for x <= 0.  -inf gives 0, as all below -104 do (the limit keeps the rest
// finite there); results below 2^-126 may be 0; NaN stays NaN (v_maximum3).
__device__ inline float exp_nonpos(float x) {
  x = __builtin_elementwise_maximum(x, -150.0f);
  const float t = x * kLog2e, y = __builtin_amdgcn_exp2f(t);
  return fmaf(y, exp_rest(x, t), y);
}

// 1 / (1 + e^-x) to 5 * 2^-24 relative, 0 below -87.4: there the denominator
// passes 2^126 and the hardware's reciprocal is 0 (it has no subnormal results),
// which the Newton step leaves 0.  The limits keep all of it finite; beyond them
// nothing changes.  The sigmoid of NaN is some number (its users multiply by x).
__device__ inline float sigmoid(float x) {
  const float n = __builtin_amdgcn_fmed3f(-x, -150.0f, 88.0f);
  const float t = n * kLog2e, y = __builtin_amdgcn_exp2f(t);
  const float d = fmaf(y, exp_rest(n, t), 1.0f + y);
  const float r = __builtin_amdgcn_rcpf(d);
  return fmaf(fmaf(-d, r, 1.0f), r, r);
}

}  // namespace mxk

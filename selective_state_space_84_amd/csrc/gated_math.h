// The gated recurrence of one channel, on the device (gfx950 only).
//
//   sa = sigmoid(ga), sx = sigmoid(gx), a = exp(log_a sa), m = sqrt(1 - a^2)
//   h <- a h + m sx x
// and what its gradient needs of a step: with g the gradient of the new state
// and h the state before,
//   dx = g m sx, dgx = g m x sx (1 - sx),
//   d(log a) = g (a h - (a^2 / m) sx x),
//   dga = d(log a) log_a sa (1 - sa), and d(log a) sa adds to dlog_a.
#pragma once

#include "ssm_device.h"

namespace ssm {

__device__ __forceinline__ float sigmoid(float v) { return hw_rcp(1.0f + hw_exp2(-v * kLog2e)); }

// 1 - 2^y for y <= 0 and p = 2^y.  Above -0.36 (2^y > 0.78) from the series of
// (e^v - 1) / v to fifth order, v = y ln 2 (truncation below 5e-8 relative), so
// that decays near 1 keep their distance from it; below, 1 - p loses at most
// two bits.
__device__ __forceinline__ float one_minus_exp2(float y, float p) {
  float q = __builtin_fmaf(y, 1.5403530e-4f, 1.3333558e-3f);  // ln2^6 / 6!, ln2^5 / 5!
  q = __builtin_fmaf(q, y, 9.6181291e-3f);
  q = __builtin_fmaf(q, y, 5.5504109e-2f);
  q = __builtin_fmaf(q, y, 2.4022651e-1f);
  q = __builtin_fmaf(q, y, kLn2);
  return y > -0.36f ? -y * q : 1.0f - p;
}

// Where 1 - a^2 is below fp32's normal range the input counts as nothing: m,
// and 1 / m as the gradient uses it, are 0.
constexpr float kTiny = 1.17549435e-38f;

struct GatedStep {
  float sa, sx, a, m, inv_m;
};

// c2 = log_a log2(e).
__device__ __forceinline__ GatedStep gated_step(float ga, float gx, float c2) {
  GatedStep s;
  s.sa = sigmoid(ga);
  s.sx = sigmoid(gx);
  const float y = c2 * s.sa;
  s.a = hw_exp2(y);
  const float e = one_minus_exp2(y, s.a);
  const float m2 = e * (2.0f - e);  // (1 - a)(1 + a)
  s.inv_m = m2 >= kTiny ? __builtin_amdgcn_rsqf(m2) : 0.0f;
  s.m = m2 * s.inv_m;
  return s;
}

}  // namespace ssm

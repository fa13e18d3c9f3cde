// The gated recurrence of one channel, on the device (gfx950 only).
//
//   sa = sigmoid(ga), sx = sigmoid(gx), a = exp(log_a sa), m = sqrt(1 - a^2)
//   h <- a h + m sx x
// and what its gradient needs of a step: with g the gradient of the new state
// and h the state before,
//   dx = g m sx, dgx = g m x sx (1 - sx),
//   d(log a) = g (a h - (a^2 / m) sx x),
//   dga = d(log a) log_a sa (1 - sa), and d(log a) sa adds to dlog_a.
// What is left of a gate, 1 - s = e / (1 + e) = e s with e = e^-v, is a product and
// not a difference, which in fp32 is a multiple of 2^-24: 0.6% off at v = 12, all of it at 17.
#pragma once

#include "ssm_device.h"

namespace ssm {

__device__ __forceinline__ float exp_minus(float v) { return hw_exp2(-v * kLog2e); }
// sigmoid(v) from e = e^-v, and 1 - sigmoid(v) from that (where e is infinite, the product is NaN and 1 is left).
__device__ __forceinline__ float sigmoid_of(float e) { return hw_rcp(1.0f + e); }
__device__ __forceinline__ float left_of(float e, float s) { return __builtin_fminf(e * s, 1.0f); }
__device__ __forceinline__ float sigmoid(float v) { return sigmoid_of(exp_minus(v)); }

// c ? a : b as a select: of the ternary operator the compiler makes a branch around what a or b costs, which
// takes longer than both.
__device__ __forceinline__ float pick(bool c, float a, float b) {
  typedef float f1 __attribute__((ext_vector_type(1)));
  typedef int i1 __attribute__((ext_vector_type(1)));
  const f1 r = i1(-(int)c) ? f1(a) : f1(b);
  return r[0];
}

// 1 - 4^y for y <= 0 and p = 2^y.  Above -0.18 (4^y > 0.78) from the series of
// (e^v - 1) / v to fifth order, v = y ln 4 (truncation below 5.3e-8 relative), so
// that decays near 1 keep their distance from it; below, 1 - p^2 loses at most
// two bits.
__device__ __forceinline__ float one_minus_exp4(float y, float p) {
  float q = __builtin_fmaf(y, 9.85825945e-3f, 4.26673861e-2f);  // ln4^6 / 6!, ln4^5 / 5!
  q = __builtin_fmaf(q, y, 0.153890066f);
  q = __builtin_fmaf(q, y, 0.444032869f);
  q = __builtin_fmaf(q, y, 0.960906028f);
  q = __builtin_fmaf(q, y, 1.38629436f);
  return pick(y > -0.18f, -y * q, __builtin_fmaf(-p, p, 1.0f));
}

// Where m2 = 1 - a^2 is below fp32's normal range the input counts as nothing: the hardware's root takes it as 0,
// and 1 / m as the gradient uses it is 0.
constexpr float kTiny = 1.17549435e-38f;

struct GatedStep {
  float ea, ex, sa, sx, a, m2;  // ea, ex: e^-ga, e^-gx
  __device__ __forceinline__ float m() const { return __builtin_amdgcn_sqrtf(m2); }
  __device__ __forceinline__ float inv_m() const { return m2 >= kTiny ? __builtin_amdgcn_rsqf(m2) : 0.0f; }
};

// c2 = log_a log2(e).
__device__ __forceinline__ GatedStep gated_step(float ga, float gx, float c2) {
  GatedStep s;
  s.ea = exp_minus(ga);
  s.ex = exp_minus(gx);
  s.sa = sigmoid_of(s.ea);
  s.sx = sigmoid_of(s.ex);
  const float y = c2 * s.sa;
  s.a = hw_exp2(y);
  s.m2 = one_minus_exp4(y, s.a);
  return s;
}

}  // namespace ssm

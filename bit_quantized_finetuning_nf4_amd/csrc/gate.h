// gate.h -- the activation of a gated block, act(x) = x sigma(p(x)): p(x) = x
// (silu), or 2 sqrt(2 / pi) (x + 0.044715 x^3) (gelu in its tanh form, since
// (1 + tanh z) / 2 = sigma(2 z)).
#pragma once
#include "device.h"

namespace qlora {

constexpr int kActSilu = 0, kActGelu = 1;   // the values of qlora_act
constexpr double kGeluC = 1.5957691216057307118;   // 2 sqrt(2 / pi)
constexpr double kGeluA = 0.044715;

// In fp32, for results of 16 bits: exp by the hardware's 2^x is within about
// 6e-8 |p| of its value, 5e-6 where the result has not yet become zero.
// exp(-p) = infinity gives sigma = 0, and act = -0.
template <int ACT>
__device__ __forceinline__ float act_of(float x) {
  const float p = ACT == kActSilu ? x : (float)kGeluC * (x + (float)kGeluA * x * x * x);
  return x * __builtin_amdgcn_rcpf(1.0f + __expf(-p));
}
// act(g) u: one rounding to 16 bits follows.
__device__ __forceinline__ float gate_of(float g, float u, int act) {
  return (act == kActSilu ? act_of<kActSilu>(g) : act_of<kActGelu>(g)) * u;
}

// exp(-a) for a >= 0 in fp64: a = n ln 2 + f, |f| <= ln 2 / 2, the series of
// e^-f to f^9 (the rest is below 8e-12), 2^-n.  Past 1100 it is 0.
__device__ __forceinline__ double exp_neg(double a) {
  a = fmin(a, 1100.0);
  const double n = __builtin_rint(a * 1.4426950408889634074);
  const double f = fma(n, 0.69314718055994530942, -a);   // -f of the text: e^f below
  double e = 1.0 / 362880.0;
  e = fma(e, f, 1.0 / 40320.0);
  e = fma(e, f, 1.0 / 5040.0);
  e = fma(e, f, 1.0 / 720.0);
  e = fma(e, f, 1.0 / 120.0);
  e = fma(e, f, 1.0 / 24.0);
  e = fma(e, f, 1.0 / 6.0);
  e = fma(e, f, 0.5);
  e = fma(e, f, 1.0);
  e = fma(e, f, 1.0);
  return __builtin_ldexp(e, -(int)n);
}

// sigma(p(x)) and act'(x) = sigma + x sigma (1 - sigma) p'(x), in fp64 (about
// 1e-11): the gradients made of them are rounded to 16 bits in between, and in
// fp32 one in some 50 thousand would round the other way, which alone leaves
// 2e-5 of the 32-bit gradients behind them.
__device__ __forceinline__ void gate_slope(double x, int act, double& sigma, double& slope) {
  double p = x, dp = 1.0;
  if (act == kActGelu) {
    const double x2 = x * x;
    p = kGeluC * fma(kGeluA * x2, x, x);
    dp = kGeluC * fma(3.0 * kGeluA, x2, 1.0);
  }
  const double e = exp_neg(__builtin_fabs(p)), d = 1.0 + e;
  double inv = __builtin_amdgcn_rcp(d);
  inv = fma(fma(-d, inv, 1.0), inv, inv);   // 2^-24 to 2^-48
  const double lo = e * inv;   // sigma(-|p|)
  sigma = p < 0.0 ? lo : inv;
  slope = fma(x * (inv * lo), dp, sigma);
}

}  // namespace qlora

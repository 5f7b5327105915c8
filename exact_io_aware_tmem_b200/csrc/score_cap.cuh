// The tanh cap of shaped scores, in base-2 units: x = A tanh(s scale / cap) with
// A = cap log2 e, from the raw product s.
#pragma once

#include <math.h>

#include "common.cuh"

namespace fa {

// tanh(u) ~ u (C0 + C1 w + .. + C6 w^6), w = u^2, |u| <= 1: the coefficients
// minimise the largest absolute error over [0, 1], 2.0e-8 (a linear program
// over 2000 points; three more roundings of 2^-24 come with fp32). Under a cap
// of 50 that moves a logit by 1e-6. tanh.approx (2^-11 relative) would move
// one of 20 by 0.01, a relative error of P five times its rounding to bf16.
constexpr int CAP_TERMS = 7;
constexpr double CAP_C[CAP_TERMS] = {0.9999997019767761,   -0.3333212733268738,
                                     0.13319575786590576,  -0.05326556786894798,
                                     0.019972829148173332, -0.005950915161520243,
                                     0.0009636600152589381};

// By value to the kernels. poly[i] = A (scale / cap)^(2 i + 1) C[i], so that the
// polynomial runs on s itself; it holds for |s| <= limit.
struct CapArgs {
  float poly[CAP_TERMS];
  float tpoly[CAP_TERMS];   // the same without A: tanh itself
  float limit;              // cap / scale, or -1: always the exponential form
  float amp;                // A
  float k2;                 // 2 log2 e scale / cap: e^(2u) = 2^(k2 s)
};

inline CapArgs cap_args(float cap, float scale) {
  CapArgs a = {};
  const double log2e = 1.4426950408889634, c1 = static_cast<double>(scale) / cap;
  a.amp = static_cast<float>(cap * log2e);
  a.k2 = static_cast<float>(2.0 * log2e * c1);
  a.limit = static_cast<float>(1.0 / c1);
  double pw = c1;
  for (int i = 0; i < CAP_TERMS; ++i, pw *= c1 * c1) {
    a.poly[i] = static_cast<float>(cap * log2e * pw * CAP_C[i]);
    a.tpoly[i] = static_cast<float>(pw * CAP_C[i]);
    // Powers of an extreme scale / cap that leave fp32's normal range (both
    // ways) leave the polynomial without its terms.
    const double least = fmin(fabs(a.poly[i]), fabs(a.tpoly[i]));
    if (!isfinite(a.poly[i]) || !isfinite(a.tpoly[i]) || least < 1e-37) a.limit = -1.f;
  }
  if (!isfinite(a.limit)) a.limit = -1.f;
  return a;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The exponential form, for any s: tanh(u) = 1 - 2 / (e^(2u) + 1), to a few
// steps of 2^-24 absolutely; e^(2u) = inf and 0 give 1 and -1.
__device__ __forceinline__ float cap_tanh(const CapArgs& a, float s) {
  return fmaf(-2.f, rcp_approx(ex2_approx(s * a.k2) + 1.f), 1.f);
}

__device__ __forceinline__ float cap_exact(const CapArgs& a, float s) {
  return a.amp * cap_tanh(a, s);
}

// Two scores within the limit, on packed fp32 pairs: x + add.
__device__ __forceinline__ float2 cap_poly2(const CapArgs& a, float2 s, float2 add) {
  const float2 w = __fmul2_rn(s, s);
  float2 t = make_float2(a.poly[CAP_TERMS - 1], a.poly[CAP_TERMS - 1]);
#pragma unroll
  for (int i = CAP_TERMS - 2; i >= 0; --i)
    t = __ffma2_rn(t, w, make_float2(a.poly[i], a.poly[i]));
  return __ffma2_rn(s, t, add);
}

}  // namespace fa

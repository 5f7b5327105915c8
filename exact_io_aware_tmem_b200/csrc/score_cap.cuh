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
__host__ __device__ constexpr float cap_c(int i) {
  constexpr float c[CAP_TERMS] = {0.9999997019767761f,   -0.3333212733268738f,
                                  0.13319575786590576f,  -0.05326556786894798f,
                                  0.019972829148173332f, -0.005950915161520243f,
                                  0.0009636600152589381f};
  return c[i];
}

// The same over |u| <= 0.6 with five coefficients: 2.0e-8 too.
constexpr int CAP_FEW = 5;
constexpr double CAP_FEW_C[CAP_FEW] = {0.9999996423721313, -0.33331209421157837, 0.13299210369586945,
                                       -0.051696743816137314, 0.01497695967555046};
constexpr double CAP_FEW_END = 0.6;

// By value to the kernels.
struct CapArgs {
  float few[CAP_FEW];       // A c1^(2 i + 1) CAP_FEW_C[i], on s itself: one product less
  float few_limit;          // 0.6 / c1, or -1 where a power of c1 leaves fp32's normal range
  float poly[CAP_TERMS];    // A cap_c(i)
  float c1;                 // scale / cap: u = c1 s
  float limit;              // 1 / c1: the polynomial holds for |s| <= limit
  float amp;                // A
  float k2;                 // 2 log2 e c1: e^(2u) = 2^(k2 s)
};

inline CapArgs cap_args(float cap, float scale) {
  CapArgs a = {};
  const double log2e = 1.4426950408889634, c1 = static_cast<double>(scale) / cap;
  a.amp = static_cast<float>(cap * log2e);
  a.c1 = static_cast<float>(c1);
  a.k2 = static_cast<float>(2.0 * log2e * c1);
  a.limit = static_cast<float>(1.0 / c1);
  a.few_limit = static_cast<float>(CAP_FEW_END / c1);
  double pw = cap * log2e * c1;
  for (int i = 0; i < CAP_FEW; ++i, pw *= c1 * c1) {
    a.few[i] = static_cast<float>(pw * CAP_FEW_C[i]);
    if (!isfinite(a.few[i]) || fabs(a.few[i]) < 1e-37) a.few_limit = -1.f;
  }
  for (int i = 0; i < CAP_TERMS; ++i) a.poly[i] = static_cast<float>(cap * log2e * cap_c(i));
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

// Two scores within the limit, on packed fp32 pairs: A tanh + add.
__device__ __forceinline__ float2 cap_poly2(const CapArgs& a, float2 s, float2 add) {
  const float2 u = __fmul2_rn(s, make_float2(a.c1, a.c1));
  const float2 w = __fmul2_rn(u, u);
  float2 t = make_float2(a.poly[CAP_TERMS - 1], a.poly[CAP_TERMS - 1]);
#pragma unroll
  for (int i = CAP_TERMS - 2; i >= 0; --i)
    t = __ffma2_rn(t, w, make_float2(a.poly[i], a.poly[i]));
  return __ffma2_rn(u, t, add);
}

// The same for |s| <= few_limit.
__device__ __forceinline__ float2 cap_few2(const CapArgs& a, float2 s, float2 add) {
  const float2 w = __fmul2_rn(s, s);
  float2 t = make_float2(a.few[CAP_FEW - 1], a.few[CAP_FEW - 1]);
#pragma unroll
  for (int i = CAP_FEW - 2; i >= 0; --i) t = __ffma2_rn(t, w, make_float2(a.few[i], a.few[i]));
  return __ffma2_rn(s, t, add);
}

// The same without A and add: tanh itself.
__device__ __forceinline__ float2 cap_tanh2(const CapArgs& a, float2 s) {
    const float2 u = __fmul2_rn(s, make_float2(a.c1, a.c1));
  const float2 w = __fmul2_rn(u, u);
  float2 t = make_float2(cap_c(CAP_TERMS - 1), cap_c(CAP_TERMS - 1));
#pragma unroll
  for (int i = CAP_TERMS - 2; i >= 0; --i) t = __ffma2_rn(t, w, make_float2(cap_c(i), cap_c(i)));
  return __fmul2_rn(u, t);
}

}  // namespace fa

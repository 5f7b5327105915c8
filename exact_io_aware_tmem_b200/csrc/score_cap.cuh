// The tanh cap of shaped scores, in base-2 units: x = A tanh(u), A = cap log2 e,
// u = s scale / cap, from the raw product s.
#pragma once

#include <math.h>

#include "common.cuh"

namespace fa {

// tanh(u) ~ u (C0 + C1 w + C2 w^2 + ..), w = u^2. The coefficients minimise the
// largest absolute error over [0, END] (a linear program over 2000 points): 1.9e-8
// for both forms; roundings of 2^-24 come with fp32. Under a cap of 50 that moves a
// logit by 1e-6. (tanh.approx, 2^-11 relative, would move one of 20 by 0.01: a
// relative error of P five times that of its rounding to bf16.)
constexpr int CAP_FEW = 4;
constexpr double CAP_FEW_END = 0.4;
constexpr double CAP_FEW_C[CAP_FEW] = {0.9999995734191381, -0.33329726033647633,
                                       0.13250565802189446, -0.04682569275562819};
constexpr int CAP_MORE = 6;
constexpr double CAP_MORE_END = 0.8;
constexpr double CAP_MORE_C[CAP_MORE] = {0.9999996699521561,  -0.3333183347279361,
                                         0.1331373978673793,  -0.05285471703904532,
                                         0.018689375804664888, -0.004126559774304747};

// By value to the kernels. The polynomials run on s itself: coefficient i holds
// A (scale / cap)^(2 i + 1) C_i.
struct CapArgs {
  float few[CAP_FEW];
  float more[CAP_MORE];
  float few_limit;    // 0.4 cap / scale: the first holds for |s| up to it
  float more_limit;   // 0.8 cap / scale; beyond it the exponential form
  float amp;          // A
  float inv_amp2;     // 1 / A^2
  float k2;           // e^(2u) = 2^(k2 s)
};

// For an extreme scale / cap the coefficients leave fp32's normal range. Too large: the
// form gets a limit of -1 and nothing takes it. Too small, under a large cap: term i and
// those behind it are dropped and the form ends where they would reach 2^-26 of the
// first, |u| <= 2^(-13 / i); the exponential form, good to cap 2^-22 only, would lose
// logits far below such a cap.
inline CapArgs cap_args(float cap, float scale) {
  CapArgs a = {};
  const double log2e = 1.4426950408889634, c1 = static_cast<double>(scale) / cap;
  const double amp = cap * log2e;
  // Coefficients into `to`; returns the largest |s| for the form.
  auto fill = [&](float* to, const double* c, int n, double end) {
    double pw = amp * c1;
    bool ok = 1.0 / (amp * amp) < 1e37 && pw > 1e-37, drop = false;
    for (int i = 0; i < n; ++i, pw *= c1 * c1) {
      if (!drop && fabs(pw * c[i]) < 1e-37) {
        drop = true;
        if (i > 0) end = fmin(end, exp2(-13.0 / i));
      }
      ok = ok && fabs(pw * c[i]) < 1e37;
      to[i] = drop ? 0.f : static_cast<float>(pw * c[i]);
    }
    return ok ? static_cast<float>(fmin(end / c1, 1e18)) : -1.f;   // s^2 stays finite
  };
  a.amp = static_cast<float>(amp);
  a.inv_amp2 = static_cast<float>(1.0 / (amp * amp));
  a.k2 = static_cast<float>(2.0 * log2e * c1);
  a.few_limit = fill(a.few, CAP_FEW_C, CAP_FEW, CAP_FEW_END);
  a.more_limit = fill(a.more, CAP_MORE_C, CAP_MORE, CAP_MORE_END);
  return a;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The exponential form, for any s: tanh(u) = 1 - 2 / (e^(2u) + 1), to a few steps of
// 2^-24 absolutely; e^(2u) = inf and 0 give 1 and -1.
__device__ __forceinline__ float cap_tanh(const CapArgs& a, float s) {
  return fmaf(-2.f, rcp_approx(ex2_approx(s * a.k2) + 1.f), 1.f);
}

__device__ __forceinline__ float cap_exact(const CapArgs& a, float s) {
  return a.amp * cap_tanh(a, s);
}

// The polynomial part q(w) of two scores on packed fp32 pairs: x = s q. FORM 0: |s| <=
// few_limit, 1: |s| <= more_limit.
template <int FORM>
__device__ __forceinline__ float2 cap_poly2(const CapArgs& a, float2 s) {
  constexpr int N = FORM == 0 ? CAP_FEW : CAP_MORE;
  const float* c = FORM == 0 ? a.few : a.more;
  const float2 w = __fmul2_rn(s, s);
  float2 t = make_float2(c[N - 1], c[N - 1]);
#pragma unroll
  for (int i = N - 2; i >= 0; --i) t = __ffma2_rn(t, w, make_float2(c[i], c[i]));
  return t;
}

// Which form the scores of a warp's registers take, from this lane's largest |s|.
__device__ __forceinline__ int cap_form(const CapArgs& a, float most) {
  if (!__any_sync(0xffffffffu, most > a.few_limit)) return 0;
  return __any_sync(0xffffffffu, most > a.more_limit) ? 2 : 1;
}

}  // namespace fa

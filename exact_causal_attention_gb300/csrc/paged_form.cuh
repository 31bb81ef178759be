// The tanh cap of the score forms, on the scores of one thread.
//
// cap tanh(scale x / cap) takes one exponential and one reciprocal as 1 - 2 / (1 + e^2y), which
// would treble the work of the unit that the softmax's own exponential needs.  Scores are
// mostly well inside the cap, where tanh(y) = y P(y^2) takes multiply-adds alone: P is a
// polynomial of degree 7 fitted to tanh(y) / y on |y| <= 1.25 by iteratively reweighted least squares
// (relative error 8e-8 before rounding).  A group of scores with one outside takes the other way.
#pragma once
#include "paged_common.cuh"

namespace eca {

// Score forms as the kernels' template argument.
constexpr int kFormPlain = 0;
constexpr int kFormBias = 1;  // distance bias
constexpr int kFormCap = 2;   // tanh cap, with or without a bias

// Scales of the cap: cap_scores gives unit * cap tanh(x scale / cap).
struct CapScale {
  float in;     // scale / cap
  float out;    // cap unit
  float limit;  // |x| up to which the polynomial holds
  float2 c[8];  // its coefficients for x^2, with the scales folded in, for pairs of scores
};

__device__ __forceinline__ CapScale cap_scale(float scale, float softcap, float unit) {
  constexpr float kRange = 1.25f;
  constexpr float kCoef[8] = {0.99999994f,    -0.333327f,     0.13324507f,    -0.05349034f,
                              0.020557173f, -0.0067961547f, 0.0015881141f, -0.00018259805f};
  CapScale r;
  r.in = softcap > 0.f ? scale / softcap : 0.f;
  r.out = softcap * unit;
  r.limit = r.in > 0.f ? kRange / r.in : 0.f;
  float f = r.out * r.in;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.c[i] = make_float2(kCoef[i] * f, kCoef[i] * f);
    f *= r.in * r.in;
  }
  return r;
}

// tanh(y) = 1 - 2 / (1 + e^2y), for any y.
__device__ __forceinline__ float tanh_wide(float y) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(y * (2.f * kLog2e)) + 1.f));
  return fmaf(-2.f, r, 1.f);
}

// A whole warp: 32 scores per thread, x to unit cap tanh(x scale / cap).
__device__ __forceinline__ void cap_scores(uint32_t (&s)[32], const CapScale& k) {
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 32; i += 2) mx = fmax3(mx, fabsf(__uint_as_float(s[i])), fabsf(__uint_as_float(s[i + 1])));
  if (__all_sync(0xffffffffu, mx <= k.limit)) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 x = make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
      const float2 z = __fmul2_rn(x, x);
      float2 a = k.c[7];
#pragma unroll
      for (int j = 6; j >= 0; --j) a = __ffma2_rn(a, z, k.c[j]);
      a = __fmul2_rn(a, x);
      s[i] = __float_as_uint(a.x);
      s[i + 1] = __float_as_uint(a.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = __float_as_uint(k.out * tanh_wide(__uint_as_float(s[i]) * k.in));
  }
}

}  // namespace eca

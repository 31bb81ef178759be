// The tanh cap of the score forms, on the scores of one thread.
//
// cap tanh(scale x / cap) takes one exponential and one reciprocal as 1 - 2 / (1 + e^2y), which
// would treble the work of the unit that the softmax's own exponential needs.  Scores are
// mostly well inside the cap, where tanh(y) = y P(y^2) takes multiply-adds alone: P is a
// polynomial fitted to tanh(y) / y by iteratively reweighted least squares, of degree 5 on
// |y| <= 0.75 or 7 on |y| <= 1.25 (relative errors 3e-8 and 8e-8 before rounding).  In a group of
// scores with some outside those take the exponential.  (Weights of 500 tokens over 12000 keys, two requests: 154 us with
// a cap of 50, 253 with 20, where most groups have some outside.)
#pragma once
#include <type_traits>

#include "paged_common.cuh"

namespace eca {

// Score forms as the kernels' template argument.
constexpr int kFormPlain = 0;
constexpr int kFormBias = 1;  // distance bias
constexpr int kFormCap = 2;   // tanh cap
constexpr int kFormBoth = 3;  // cap, then bias
__host__ __device__ constexpr bool form_caps(int form) { return form == kFormCap || form == kFormBoth; }
__host__ __device__ constexpr bool form_biases(int form) { return form == kFormBias || form == kFormBoth; }

// Scales of the cap: cap_scores gives big * unit * cap tanh(x scale / cap).  The polynomials run in
// x^2, with powers of scale / cap folded into their coefficients; `big`, a power of two of about
// (cap / scale)^7, keeps the highest coefficient from underflowing, and goes out again with a
// multiplication that the caller does anyway.
struct CapScale {
  float out;        // cap unit
  float big, inv_big;
  float wide;       // 2 log2e scale / cap
  float near, far;  // |x| up to which the shorter and the longer polynomial hold
  float2 n[6], f[8];  // their coefficients for x^2, for pairs of scores
};

__device__ __forceinline__ CapScale cap_scale(float scale, float softcap, float unit) {
  constexpr float kNear = 0.75f, kFar = 1.25f;
  constexpr float kNearCoef[6] = {1.0f, -0.333329588f, 0.133254066f, -0.0533444285f, 0.0195829086f, -0.0047162571f};
  constexpr float kFarCoef[8] = {0.99999994f,    -0.333327f,     0.13324507f,    -0.05349034f,
                                 0.020557173f, -0.0067961547f, 0.0015881141f, -0.00018259805f};
  CapScale r;
  const float in = softcap > 0.f ? scale / softcap : 0.f;
  r.out = softcap * unit;
  // Outside 2^-12 .. 2^12 the coefficients would leave the type.  Below, the low terms alone reach as far
  // as 0.05; above, an error of 3e-7 of the cap is below a score's own rounding.
  const bool low = in < 0x1p-12f, high = in > 0x1p12f;
  r.big = low || high ? 1.f : exp2f(rintf(-7.f * log2f(in)));
  r.inv_big = 1.f / r.big;
  r.wide = 2.f * kLog2e * in;
  r.near = high ? -1.f : (low ? fminf(0.05f / in, 1e18f) : kNear / in);
  r.far = high ? -1.f : (low ? r.near : kFar / in);
  float f = scale * unit * r.big;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < 6) r.n[i] = make_float2(kNearCoef[i] * f, kNearCoef[i] * f);
    r.f[i] = make_float2(kFarCoef[i] * f, kFarCoef[i] * f);
    f *= in * in;
  }
  return r;
}

// big out tanh(x in) + plus by tanh(y) = 1 - 2 / (1 + e^2y), for x that is not small.  `plus` joins the
// leading term, so that where the sum is small its rounding is too.
__device__ __forceinline__ float cap_wide(float x, const CapScale& k, float plus) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(fabsf(x) * k.wide) + 1.f));
  const float side = copysignf(k.out * k.big, x);
  return fmaf(-2.f * side, r, side + plus);
}

// A whole warp: 32 scores per thread, x to big unit cap tanh(x scale / cap), plus add[i] where
// there is one (in shared memory, 16-byte aligned, the same for every thread).  kNear: with
// the shorter polynomial, and the longer one in mixed groups too; a kernel whose warps wait for
// instructions does better without (a mixed step: chunk attention 209 us, with them 227).
template <bool kAdd, bool kNear>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[32], const CapScale& k, const float* add) {
  float m4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    m4[i / 2 % 4] = fmax3(m4[i / 2 % 4], fabsf(__uint_as_float(s[i])), fabsf(__uint_as_float(s[i + 1])));
  }
  const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
  // all: each score that lies outside the polynomial's range takes the exponential instead.
  auto polynomial = [&](const auto& c, auto all) {
    constexpr int kTerms = sizeof(c) / sizeof(float2);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 x = make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
      const float2 z = __fmul2_rn(x, x);
      float2 a = c[kTerms - 1];
#pragma unroll
      for (int j = kTerms - 2; j >= 0; --j) a = __ffma2_rn(a, z, c[j]);
      float2 plus = make_float2(0.f, 0.f);
      if constexpr (kAdd) plus = *reinterpret_cast<const float2*>(add + i);
      if constexpr (kAdd) {
        a = __ffma2_rn(a, x, plus);
      } else {
        a = __fmul2_rn(a, x);
      }
      if constexpr (decltype(all)::value) {
        if (!(fabsf(x.x) <= k.far)) a.x = cap_wide(x.x, k, plus.x);
        if (!(fabsf(x.y) <= k.far)) a.y = cap_wide(x.y, k, plus.y);
      }
      s[i] = __float_as_uint(a.x);
      s[i + 1] = __float_as_uint(a.y);
    }
  };
  if (kNear && __all_sync(0xffffffffu, mx <= k.near)) {
    polynomial(k.n, std::false_type{});
  } else if (__all_sync(0xffffffffu, mx <= k.far)) {
    polynomial(k.f, std::false_type{});
  } else if constexpr (kNear) {
    polynomial(k.f, std::true_type{});
  } else {
    // All of them by the exponential: off by 3e-7 of the cap at small scores, in a quarter of the code.
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = __float_as_uint(cap_wide(__uint_as_float(s[i]), k, kAdd ? add[i] : 0.f));
  }
}

}  // namespace eca

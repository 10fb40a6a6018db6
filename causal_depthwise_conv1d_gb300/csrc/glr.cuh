// Shared by the kernels of the gated linear recurrence.
//
//   r = sigmoid(p), i = sigmoid(q), l = -rate r, a = exp(l), m = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + m_t i_t x_t
//
// Where the decay is close to one both a and 1 - a^2 come from E = expm1(l):
// a = 1 + E, 1 - a^2 = -E (2 + E).  For -0.85 <= l E is l times a polynomial of
// degree 6 (fitted for the least relative error on that interval by exchange:
// 8e-10, 6e-9 with FP32 coefficients; the Taylor polynomial needs degree 8), below that 2^(l log2 e) - 1 with
// the hardware's exponential (2^-22 relative, while 1 - a >= 0.57).  So a
// is within 2^-24 of the exact decay where a state lasts longer than two
// tokens, and m keeps its relative precision down to the smallest rates; from
// a rounded to FP32, 1 - a^2 would have lost 10 of its 24 bits at a = 0.9995.
// As -rate <= l, channels whose rate is at most 0.85 need no exponential here,
// and a warp that has no others takes the shorter code (the same values).
//
// A decay is positive, and so is every product of decays: neither is let down to
// zero (glr_positive), so an infinite state stays infinite where 0 * inf would
// make it NaN.  To a finite state h that adds at most 2^-149 |h|, as much as
// the rounding of such a decay.
#pragma once

#include "ccv_common.cuh"
#include "rec_internal.h"

namespace ccv {

constexpr float kGlrSeries = -0.85f;  // down to here the polynomial
// Coefficients of (e^l - 1) / l, highest power first.
__host__ __device__ constexpr float glr_poly(int i) {
  constexpr float c[7] = {0x1.1f4de2p-13f, 0x1.5a4692p-10f, 0x1.0fcc68p-7f, 0x1.553d2cp-5f,
                          0x1.555478p-3f,  0x1.fffffap-2f,  1.f};
  return c[i];
}

struct GlrGate {
  float a, m2;   // decay, 1 - a^2
  float r, omr;  // sigmoid of the decay gate, and 1 minus it
  float l;       // log a
  float i, omi;  // sigmoid of the input gate, and 1 minus it
};

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// +0 as the smallest positive number, 2^-149; -0 and NaN as they are.
__device__ __forceinline__ float glr_positive(float a) { return __uint_as_float(max(__float_as_uint(a), 1u)); }

__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// sigmoid(z) and 1 - sigmoid(z) = e^-z sigmoid(z) (one where e^-z leaves the
// exponent's range).
__device__ __forceinline__ void glr_sigmoid(float z, float& s, float& om) {
  const float e = ex2_approx(__fmul_rn(z, -kLog2e));
  s = rcp_approx(__fadd_rn(1.f, e));
  om = e < 0x1p100f ? __fmul_rn(e, s) : 1.f;
}

__device__ __forceinline__ void glr_decay(float l, float& a, float& m2) {
  float E = glr_poly(0);
#pragma unroll
  for (int i = 1; i < 7; ++i) E = fmaf(E, l, glr_poly(i));
  E = __fmul_rn(E, l);
  const float far = glr_positive(ex2_approx(__fmul_rn(l, kLog2e)));
  const bool near = l >= kGlrSeries;
  a = near ? __fadd_rn(1.f, E) : far;
  E = near ? E : __fadd_rn(far, -1.f);
  m2 = __fmul_rn(-E, __fadd_rn(2.f, E));
}

__device__ __forceinline__ GlrGate glr_gate(float p, float q, float rate) {
  GlrGate g;
  glr_sigmoid(p, g.r, g.omr);
  glr_sigmoid(q, g.i, g.omi);
  g.l = __fmul_rn(-rate, g.r);
  glr_decay(g.l, g.a, g.m2);
  return g;
}

}  // namespace ccv

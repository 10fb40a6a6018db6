// Pairs of the recurrence's and the group norm's kernels (packed FP32, see
// ccv_common.cuh).
#pragma once

#include "ccv_common.cuh"

namespace ccv {

__device__ __forceinline__ uint64_t twice(float c) { return pk(c, c); }

__device__ __forceinline__ float pair_sum(uint64_t v) {
  float a, b;
  upk(v, a, b);
  return a + b;
}

// Vectors as pairs.
template <int DT>
__device__ __forceinline__ void unpack_pairs(const uint4& v, uint64_t* f) {
  constexpr int V = Fmt<DT>::VEC;
  float x[V];
  unpack16<DT>(v, x);
#pragma unroll
  for (int j = 0; j < V / 2; ++j) f[j] = pk(x[2 * j], x[2 * j + 1]);
}

// a b + c, results below 2^-126 as zero.
__device__ __forceinline__ uint64_t ffma2_ftz(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// The larger one; NaN where one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// SiLU of a pair with one reciprocal for both: 1 / d0 = d1 / (d0 d1).  The
// special-function unit takes 16 reciprocals a clock and SM but 32 exponentials,
// so a pair takes two thirds of its time.  d = 2^-63 (1 + 2^(-z log2 e)), the
// exponent cut at 2^62, so neither the product nor its reciprocal leaves the
// range and a value far in the tail (or one that is not finite) says nothing
// about its neighbour.  From z = -86 down the sigmoid would stay at 2^-125, which
// is taken off again: it is zero there to within its own rounding, 2^-146, and
// flushed, so that -1e38 gives zero too.
__device__ __forceinline__ uint64_t silu_pair(uint64_t z) {
  float a0, a1;
  upk(ffma2(z, twice(-kLog2e), twice(-63.f)), a0, a1);
  const uint64_t d = fadd2(pk(ex2_approx(fminf(a0, 62.f)), ex2_approx(fminf(a1, 62.f))), twice(0x1p-63f));
  float d0, d1;
  upk(d, d0, d1);
  const float r = rcp_approx(__fmul_rn(d0, d1));
  return fmul2(z, ffma2_ftz(fmul2(pk(r, r), pk(d1, d0)), twice(0x1p-63f), twice(-0x1p-125f)));
}

// g times SiLU's derivative s (1 + z (1 - s)), in the same way with 2^-60: from
// z = -80 down, where the derivative is below 1e-32, s is zero.
__device__ __forceinline__ uint64_t silu_grad_pair(uint64_t z, uint64_t g) {
  float a0, a1;
  upk(ffma2(z, twice(-kLog2e), twice(-60.f)), a0, a1);
  const uint64_t e = pk(ex2_approx(fminf(a0, 55.f)), ex2_approx(fminf(a1, 55.f)));
  float d0, d1;
  upk(fadd2(e, twice(0x1p-60f)), d0, d1);
  const float r = rcp_approx(__fmul_rn(d0, d1));
  const uint64_t u = fmul2(pk(r, r), pk(d1, d0));  // 2^60 s
  return fmul2(fmul2(g, ffma2_ftz(u, twice(0x1p-60f), twice(-0x1p-115f))), ffma2(z, fmul2(e, u), twice(1.f)));
}

// The same with a reciprocal each, z itself cut at -80.
__device__ __forceinline__ uint64_t silu_grad_pair2(uint64_t z, uint64_t g) {
  float z0, z1, a0, a1, d0, d1;
  upk(z, z0, z1);
  z = pk(max_nan(z0, -80.f), max_nan(z1, -80.f));
  upk(fmul2(z, twice(-kLog2e)), a0, a1);
  const uint64_t e = pk(ex2_approx(a0), ex2_approx(a1));
  upk(fadd2(e, twice(1.f)), d0, d1);
  const uint64_t s = pk(rcp_approx(d0), rcp_approx(d1));
  return fmul2(g, fmul2(s, ffma2(z, fmul2(e, s), twice(1.f))));
}

// SiLU's derivative of one value, in the same way.
__device__ __forceinline__ float silu_grad_cut(float z) {
  z = max_nan(z, -80.f);
  const float e = ex2_approx(__fmul_rn(z, -kLog2e)), s = rcp_approx(__fadd_rn(1.f, e));
  return __fmul_rn(s, fmaf(z, __fmul_rn(e, s), 1.f));
}

}  // namespace ccv

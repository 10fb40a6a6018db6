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

// SiLU of a pair with one reciprocal for both: 1 / d0 = d1 / (d0 d1).  The
// special-function unit takes 16 reciprocals a clock and SM but 32 exponentials,
// so a pair takes two thirds of its time.  d = 2^-63 (1 + 2^(-z log2 e)), the
// exponent cut at 2^62, so neither the product nor its reciprocal leaves the
// range and a value far in the tail (or infinite) says nothing about its
// neighbour.  Below z = -86 the sigmoid stays at 2^-125 instead of falling on:
// the result is off by less than 1e-35.
__device__ __forceinline__ uint64_t silu_pair(uint64_t z) {
  float a0, a1;
  upk(ffma2(z, twice(-kLog2e), twice(-63.f)), a0, a1);
  const uint64_t d = fadd2(pk(ex2_approx(fminf(a0, 62.f)), ex2_approx(fminf(a1, 62.f))), twice(0x1p-63f));
  float d0, d1;
  upk(d, d0, d1);
  const float r = rcp_approx(__fmul_rn(d0, d1));
  return fmul2(z, fmul2(fmul2(pk(r, r), pk(d1, d0)), twice(0x1p-63f)));
}

// g times SiLU's derivative s (1 + z (1 - s)), in the same way with 2^-60: z is
// cut at -80, where the derivative is below 1e-32.
__device__ __forceinline__ uint64_t silu_grad_pair(uint64_t z, uint64_t g) {
  float z0, z1, a0, a1;
  upk(z, z0, z1);
  upk(ffma2(pk(fmaxf(z0, -80.f), fmaxf(z1, -80.f)), twice(-kLog2e), twice(-60.f)), a0, a1);
  const uint64_t e = pk(ex2_approx(a0), ex2_approx(a1));
  float d0, d1;
  upk(fadd2(e, twice(0x1p-60f)), d0, d1);
  const float r = rcp_approx(__fmul_rn(d0, d1));
  const uint64_t u = fmul2(pk(r, r), pk(d1, d0));  // 2^60 s
  return fmul2(fmul2(g, fmul2(u, twice(0x1p-60f))), ffma2(z, fmul2(e, u), twice(1.f)));
}

}  // namespace ccv

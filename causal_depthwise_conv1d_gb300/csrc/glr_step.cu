// Gated linear recurrence, the decode step: a thread owns a channel of a
// request, its state in a register, one token after the other.
#include "glr.cuh"

namespace ccv {
namespace {

constexpr int kThreads = 128;

template <int DT>
__device__ __forceinline__ float glr_ld(const void* p, const int64_t* s, int64_t b, int64_t t, int64_t c) {
  return Fmt<DT>::to_f(static_cast<const typename Fmt<DT>::E*>(p)[b * s[0] + t * s[1] + c * s[2]]);
}
template <int DT>
__device__ __forceinline__ void glr_st(void* p, const int64_t* s, int64_t b, int64_t t, int64_t c, float v) {
  static_cast<typename Fmt<DT>::E*>(p)[b * s[0] + t * s[1] + c * s[2]] = Fmt<DT>::from_f(v);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) glr_seq_kernel(const GlrArgs a) {
  pdl_enter();
  const unsigned tiles = static_cast<unsigned>((a.C + kThreads - 1) / kThreads);
  const int64_t b = blockIdx.x / tiles, c = static_cast<int64_t>(blockIdx.x % tiles) * kThreads + threadIdx.x;
  if (c >= a.C) return;
  int64_t slot = b;
  if (a.slots != nullptr) slot = a.slots[b * a.slot_stride];
  if (slot < 0 || slot >= a.n_slots) {  // a padding row: no state, zero outputs
    for (int64_t t = 0; t < a.L; ++t) glr_st<DT>(a.out, a.os, b, t, c, 0.f);
    return;
  }
  const float rate = a.rate[c * a.rs];
  float h = a.s0 != nullptr ? a.s0[slot * a.s0s[0] + c * a.s0s[1]] : 0.f;
  for (int64_t t = 0; t < a.L; ++t) {
    const GlrGate g = glr_gate(glr_ld<DT>(a.p, a.ps, b, t, c), glr_ld<DT>(a.q, a.qs, b, t, c), rate);
    const float in = sqrt_approx(g.m2) * (g.i * glr_ld<DT>(a.x, a.xs, b, t, c));
    h = fmaf(g.a, h, in);
    glr_st<DT>(a.out, a.os, b, t, c, h);
  }
  if (a.s1 != nullptr) a.s1[slot * a.s1s[0] + c * a.s1s[1]] = h;
}

template <int DT>
cudaError_t fwd_dt(const GlrArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.C + kThreads - 1) / kThreads * a.B);
  return launch_pdl(glr_seq_kernel<DT>, grid, kThreads, 0, s, a);
}
}  // namespace

cudaError_t launch_glr_step(const GlrArgs& a, Dtype dt, cudaStream_t stream) {
  switch (dt) {
    case kF32: return fwd_dt<kF32>(a, stream);
    case kF16: return fwd_dt<kF16>(a, stream);
    case kBF16: return fwd_dt<kBF16>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ccv

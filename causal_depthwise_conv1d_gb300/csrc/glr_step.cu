// Gated linear recurrence, one token after the other: a thread owns a channel
// of a batch row, its state in a register.  The decode step, and (as the
// simplest form) whole sequences and their backward pass.
#include "glr.cuh"

namespace ccv {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ bool glr_new(const GlrArgs& a, int64_t b, int64_t t) {
  if (a.seq == nullptr || t == 0) return false;
  const int32_t* s = a.seq + b * a.ss[0] + t * a.ss[1];
  return s[0] != s[-a.ss[1]];
}

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
    if (a.cs != nullptr && t % kGlrChunk == 0) a.cs[b * a.css[0] + t / kGlrChunk * a.css[1] + c * a.css[2]] = h;
    const GlrGate g = glr_gate(glr_ld<DT>(a.p, a.ps, b, t, c), glr_ld<DT>(a.q, a.qs, b, t, c), rate);
    const float in = sqrt_approx(g.m2) * (g.i * glr_ld<DT>(a.x, a.xs, b, t, c));
    h = glr_new(a, b, t) ? in : fmaf(g.a, h, in);
    if (a.out != nullptr) glr_st<DT>(a.out, a.os, b, t, c, h);
  }
  if (a.s1 != nullptr) a.s1[slot * a.s1s[0] + c * a.s1s[1]] = h;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) glr_seq_bwd_kernel(const GlrArgs a, const GlrGrads gr) {
  pdl_enter();
  const unsigned tiles = static_cast<unsigned>((a.C + kThreads - 1) / kThreads);
  const int64_t b = blockIdx.x / tiles, c = static_cast<int64_t>(blockIdx.x % tiles) * kThreads + threadIdx.x;
  if (c >= a.C) return;
  const float rate = a.rate[c * a.rs];
  float G = gr.ds1 != nullptr ? gr.ds1[b * gr.ds1s[0] + c * gr.ds1s[1]] : 0.f;
  float dr = 0.f;
  float prev[kGlrChunk];
  for (int64_t k = (a.L + kGlrChunk - 1) / kGlrChunk - 1; k >= 0; --k) {
    const int64_t t0 = k * kGlrChunk;
    const int n = static_cast<int>(a.L - t0 < kGlrChunk ? a.L - t0 : kGlrChunk);
    float h = a.cs[b * a.css[0] + k * a.css[1] + c * a.css[2]];
    for (int j = 0; j < n; ++j) {
      const GlrGate g = glr_gate(glr_ld<DT>(a.p, a.ps, b, t0 + j, c), glr_ld<DT>(a.q, a.qs, b, t0 + j, c), rate);
      const float in = sqrt_approx(g.m2) * (g.i * glr_ld<DT>(a.x, a.xs, b, t0 + j, c));
      if (glr_new(a, b, t0 + j)) h = 0.f;
      prev[j] = h;
      h = fmaf(g.a, h, in);
    }
    for (int j = n - 1; j >= 0; --j) {
      const GlrGate g = glr_gate(glr_ld<DT>(a.p, a.ps, b, t0 + j, c), glr_ld<DT>(a.q, a.qs, b, t0 + j, c), rate);
      const float ix = g.i * glr_ld<DT>(a.x, a.xs, b, t0 + j, c);
      const float m = sqrt_approx(g.m2);
      G += glr_ld<DT>(gr.dout, gr.dos, b, t0 + j, c);
      // dm/dl = -a^2 / m, taken as zero where m is
      const float dm = g.m2 >= 0x1p-126f ? g.a * g.a * rsqrt_approx(g.m2) : g.m2 * 0.f;
      const float W = G * (g.a * prev[j] - ix * dm);
      glr_st<DT>(gr.dx, gr.dxs, b, t0 + j, c, G * (m * g.i));
      glr_st<DT>(gr.dq, gr.dqs, b, t0 + j, c, G * (m * ix) * g.omi);
      glr_st<DT>(gr.dp, gr.dps, b, t0 + j, c, W * (g.l * g.omr));
      dr = fmaf(W, -g.r, dr);
      G = glr_new(a, b, t0 + j) ? 0.f : G * g.a;
    }
  }
  if (a.L > 0) gr.part[b * a.C + c] = dr;
  if (gr.ds0 != nullptr) gr.ds0[b * gr.ds0s[0] + c * gr.ds0s[1]] = G;
}

template <int DT>
cudaError_t fwd_dt(const GlrArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.C + kThreads - 1) / kThreads * a.B);
  return launch_pdl(glr_seq_kernel<DT>, grid, kThreads, 0, s, a);
}
template <int DT>
cudaError_t bwd_dt(const GlrArgs& a, const GlrGrads& g, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.C + kThreads - 1) / kThreads * a.B);
  return launch_pdl(glr_seq_bwd_kernel<DT>, grid, kThreads, 0, s, a, g);
}

// drate: the partial sums in order.
__global__ void __launch_bounds__(kThreads) glr_rate_kernel(const float* part, int64_t P, int64_t C, float* drate,
                                                            int64_t drs) {
  pdl_enter();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (c >= C) return;
  float x = 0.f;
  for (int64_t i = 0; i < P; ++i) x += part[i * C + c];
  drate[c * drs] = x;
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

cudaError_t launch_glr_bwd(const GlrArgs& a, const GlrGrads& g, Dtype dt, cudaStream_t stream) {
  cudaError_t e = a.B == 0 ? cudaSuccess : cudaErrorInvalidValue;
  if (a.B > 0) switch (dt) {
    case kF32: e = bwd_dt<kF32>(a, g, stream); break;
    case kF16: e = bwd_dt<kF16>(a, g, stream); break;
    case kBF16: e = bwd_dt<kBF16>(a, g, stream); break;
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(glr_rate_kernel, static_cast<unsigned>((a.C + kThreads - 1) / kThreads), kThreads, 0, stream,
                    static_cast<const float*>(g.part), a.L > 0 ? a.B : 0, a.C, g.drate, g.drs);
}

}  // namespace ccv

// Gated linear recurrence, the decode step: a thread owns one channel of a
// request, or four adjacent ones where all rows allow vectors, its states in
// registers, one token after the other.
//
// What bounds it: the launch, and two dependent loads (slot, then state).  One
// request of 5120 channels in bf16 4.4 us, 128 requests of a cache with 192 slots
// 5.9 us (10.2 MB: 16 bytes an element and token, the state in FP32).
#include "glr.cuh"

namespace ccv {
namespace {

constexpr int kThreads = 128;

// V adjacent elements (V = 4: vectors of 8 or 16 bytes; V = 1: any stride).
template <int DT, int V>
__device__ __forceinline__ void load(const void* p, int64_t off, float* f) {
  using F = Fmt<DT>;
  const typename F::E* e = static_cast<const typename F::E*>(p) + off;
  if constexpr (V == 1) {
    f[0] = F::to_f(*e);
  } else if constexpr (DT == kF32) {
    const float4 v = *reinterpret_cast<const float4*>(e);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(e);
    f[0] = F::word_elem(v.x, 0), f[1] = F::word_elem(v.x, 1), f[2] = F::word_elem(v.y, 0), f[3] = F::word_elem(v.y, 1);
  }
}

template <int DT, int V>
__device__ __forceinline__ void store(void* p, int64_t off, const float* f) {
  using F = Fmt<DT>;
  typename F::E* e = static_cast<typename F::E*>(p) + off;
  if constexpr (V == 1) {
    *e = F::from_f(f[0]);
  } else if constexpr (DT == kF32) {
    *reinterpret_cast<float4*>(e) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    *reinterpret_cast<uint2*>(e) = make_uint2(F::pack2(f[0], f[1]), F::pack2(f[2], f[3]));
  }
}

template <int DT, int V>
__global__ void __launch_bounds__(kThreads) glr_step_kernel(const GlrArgs a, unsigned tiles) {
  pdl_enter();
  const int64_t b = blockIdx.x / tiles, c = (static_cast<int64_t>(blockIdx.x % tiles) * kThreads + threadIdx.x) * V;
  if (c >= a.C) return;
  int64_t slot = b;
  if (a.slots != nullptr) slot = a.slots[b * a.slot_stride];
  float h[V], rate[V];
  if (slot < 0 || slot >= a.n_slots) {  // a padding row: no state, zero outputs
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = 0.f;
    for (int64_t t = 0; t < a.L; ++t) store<DT, V>(a.out, b * a.os[0] + t * a.os[1] + c * a.os[2], h);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = 0.f;
  if (a.s0 != nullptr) load<kF32, V>(a.s0, slot * a.s0s[0] + c * a.s0s[1], h);
  load<kF32, V>(a.rate, c * a.rs, rate);
  for (int64_t t = 0; t < a.L; ++t) {
    float x[V], p[V], q[V];
    load<DT, V>(a.p, b * a.ps[0] + t * a.ps[1] + c * a.ps[2], p);
    load<DT, V>(a.q, b * a.qs[0] + t * a.qs[1] + c * a.qs[2], q);
    load<DT, V>(a.x, b * a.xs[0] + t * a.xs[1] + c * a.xs[2], x);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const GlrGate g = glr_gate(p[i], q[i], rate[i]);
      h[i] = fmaf(g.a, h[i], sqrt_approx(g.m2) * (g.i * x[i]));
    }
    store<DT, V>(a.out, b * a.os[0] + t * a.os[1] + c * a.os[2], h);
  }
  if (a.s1 != nullptr) store<kF32, V>(a.s1, slot * a.s1s[0] + c * a.s1s[1], h);
}

// Rows whose pieces of four elements are aligned.
bool vec4(const void* p, const int64_t* s, int nd, int64_t esize) {
  if (p == nullptr) return true;
  bool ok = s[nd - 1] == 1 && reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(4 * esize) == 0;
  for (int d = 0; d + 1 < nd; ++d) ok = ok && s[d] % 4 == 0;
  return ok;
}

template <int DT>
cudaError_t launch_dt(const GlrArgs& a, cudaStream_t s) {
  const int64_t e = DT == kF32 ? 4 : 2;
  // Vectors where they leave every SM (152) a block: one request of 5120 channels takes 4.5 us with single channels.
  const bool vec = a.C % 4 == 0 && a.B * a.C >= 152 * 4 * kThreads && vec4(a.x, a.xs, 3, e) && vec4(a.p, a.ps, 3, e) &&
                   vec4(a.q, a.qs, 3, e) && vec4(a.out, a.os, 3, e) && vec4(a.s0, a.s0s, 2, 4) &&
                   vec4(a.s1, a.s1s, 2, 4) && vec4(a.rate, &a.rs, 1, 4);
  const int64_t tiles = (a.C + kThreads * (vec ? 4 : 1) - 1) / (kThreads * (vec ? 4 : 1));
  const unsigned grid = static_cast<unsigned>(a.B * tiles), n = static_cast<unsigned>(tiles);
  if (vec) return launch_pdl(glr_step_kernel<DT, 4>, grid, kThreads, 0, s, a, n);
  return launch_pdl(glr_step_kernel<DT, 1>, grid, kThreads, 0, s, a, n);
}

}  // namespace

cudaError_t launch_glr_step(const GlrArgs& a, Dtype dt, cudaStream_t stream) {
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, stream);
    case kF16: return launch_dt<kF16>(a, stream);
    case kBF16: return launch_dt<kBF16>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ccv

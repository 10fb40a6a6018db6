// Group normalisation of channels-last tensors [N,S,C] with an activation,
// forward and backward: any strides, any sizes.
//
//   xh = (x - mean) rstd over the S positions and C / G channels of a group;  z = xh w + b;  y = act(z)
//   dz = dy act'(z);  d = dz w;  dx = rstd (d - mean(d) - xh mean(d xh));  dw = sum dz xh;  db = sum dz
//
// A group's positions are cut into slabs.  A block takes a slab's mean and the
// sum of squares about that mean (two sweeps), and the slabs' pairs are merged
// exactly as sums of n_k (mean_k - mean)^2: no difference of large sums.  All
// sums are FP32 in a fixed order.
#include "ccv_common.cuh"
#include "rec_internal.h"
#include "rec_pairs.cuh"

#include <initializer_list>

namespace ccv {
namespace {

constexpr int kThreads = 256, kMaxThreads = 1024;  // of a block (see block_threads)

// Sums over the block; every thread gets them.
template <int NS>
__device__ __forceinline__ void block_sum(float (&v)[NS], float* red) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] += __shfl_xor_sync(kFullMask, v[i], m);
  __syncthreads();
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < NS; ++i) red[(threadIdx.x >> 5) * NS + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    v[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kMaxThreads / 32; ++w)
      if (w < static_cast<int>(blockDim.x >> 5)) v[i] += red[w * NS + i];
  }
}

// One block's part: sample n, group g, positions [s0, s1).  A thread keeps
// its channel over a column block of at most blockDim.x channels.
struct Slab {
  int64_t n, g, k, s0, s1;
  int cg, cols, rows, r, c;
  bool on;
  __device__ Slab(const GnArgs& a, const GnPlan& p, int64_t n_, int64_t g_, int64_t k_) : n(n_), g(g_), k(k_) {
    s0 = k * p.rows;
    s1 = s0 + p.rows < a.S ? s0 + p.rows : a.S;
    cg = static_cast<int>(a.C / a.G);
    cols = cg < static_cast<int>(blockDim.x) ? cg : static_cast<int>(blockDim.x);
    rows = static_cast<int>(blockDim.x) / cols;
    r = threadIdx.x / cols;
    c = threadIdx.x - r * cols;
    on = r < rows;
  }
  __device__ float count() const { return static_cast<float>(s1 - s0) * static_cast<float>(cg); }
};

template <int DT>
__device__ __forceinline__ float ld(const void* p, const int64_t* s, int64_t n, int64_t t, int64_t c) {
  return Fmt<DT>::to_f(static_cast<const typename Fmt<DT>::E*>(p)[n * s[0] + t * s[1] + c * s[2]]);
}

template <int DT>
__device__ float2 slab_stats(const GnArgs& a, const Slab& b, float* red) {
  const int64_t c0 = b.g * b.cg;
  float s[1] = {0.f};
  if (b.on)
    for (int c = b.c; c < b.cg; c += b.cols)
      for (int64_t t = b.s0 + b.r; t < b.s1; t += b.rows) s[0] += ld<DT>(a.x, a.xs, b.n, t, c0 + c);
  block_sum(s, red);
  const float mean = s[0] / b.count();
  float q[1] = {0.f};
  if (b.on)
    for (int c = b.c; c < b.cg; c += b.cols)
      for (int64_t t = b.s0 + b.r; t < b.s1; t += b.rows) {
        const float d = ld<DT>(a.x, a.xs, b.n, t, c0 + c) - mean;
        q[0] = fmaf(d, d, q[0]);
      }
  block_sum(q, red);
  return make_float2(mean, q[0]);
}

// Mean and rstd of a whole group from its slabs' pairs.
__device__ float2 merged_stats(const GnArgs& a, const GnPlan& p, const Slab& b, float* red) {
  const float2* st = a.stats + (b.n * a.G + b.g) * p.slabs;
  const float total = static_cast<float>(a.S) * static_cast<float>(b.cg);
  auto count = [&](int64_t k) {
    const int64_t n = (k + 1) * p.rows < a.S ? p.rows : a.S - k * p.rows;
    return static_cast<float>(n) * static_cast<float>(b.cg);
  };
  float s[1] = {0.f};
  for (int64_t k = threadIdx.x; k < p.slabs; k += blockDim.x) s[0] += st[k].x * (count(k) / total);
  block_sum(s, red);
  const float mean = s[0];
  float q[1] = {0.f};
  for (int64_t k = threadIdx.x; k < p.slabs; k += blockDim.x) {
    const float d = st[k].x - mean;
    q[0] += fmaf(d * d, count(k), st[k].y);
  }
  block_sum(q, red);
  return make_float2(mean, rsqrtf(q[0] / total + a.eps));
}

template <int DT>
__device__ void apply(const GnArgs& a, const Slab& b, float2 st) {
  using F = Fmt<DT>;
  if (!b.on) return;
  for (int c = b.c; c < b.cg; c += b.cols) {
    const int64_t ch = b.g * b.cg + c;
    const float w = a.w != nullptr ? ld_param(a.w, ch * a.ws, a.wdt) : 1.f;
    const float bias = a.b != nullptr ? ld_param(a.b, ch * a.bs, a.wdt) : 0.f;
    for (int64_t t = b.s0 + b.r; t < b.s1; t += b.rows) {
      const float z = fmaf((ld<DT>(a.x, a.xs, b.n, t, ch) - st.x) * st.y, w, bias);
      static_cast<typename F::E*>(a.out)[b.n * a.os[0] + t * a.os[1] + ch * a.os[2]] =
          F::from_f(a.silu ? silu(z) : z);
    }
  }
}

__device__ __forceinline__ Slab slab_of(const GnArgs& a, const GnPlan& p) {
  const int64_t k = blockIdx.x % p.slabs, ng = blockIdx.x / p.slabs;
  return Slab(a, p, ng / a.G, ng % a.G, k);
}

template <int DT>
__global__ void __launch_bounds__(kMaxThreads) gn_any_stats(const GnArgs a, const GnPlan p) {
  pdl_enter();
  __shared__ float red[kMaxThreads / 32];
  const Slab b = slab_of(a, p);
  const float2 st = slab_stats<DT>(a, b, red);
  if (threadIdx.x == 0) a.stats[(b.n * a.G + b.g) * p.slabs + b.k] = st;
}

template <int DT, bool WHOLE>
__global__ void __launch_bounds__(kMaxThreads) gn_any_fwd(const GnArgs a, const GnPlan p) {
  pdl_enter();
  __shared__ float red[kMaxThreads / 32];
  const Slab b = slab_of(a, p);
  float2 st;
  if constexpr (WHOLE) {
    st = slab_stats<DT>(a, b, red);
    st.y = rsqrtf(st.y / b.count() + a.eps);
  } else {
    st = merged_stats(a, p, b, red);
  }
  apply<DT>(a, b, st);
}

// dz of one element and xh.
template <int DT>
__device__ __forceinline__ float dz_of(const GnArgs& a, const Slab& b, float2 st, int64_t t, int64_t ch, float w,
                                       float bias, float& xh) {
  xh = (ld<DT>(a.x, a.xs, b.n, t, ch) - st.x) * st.y;
  const float g = ld<DT>(a.dout, a.gs, b.n, t, ch);
  return a.silu ? g * silu_grad_cut(fmaf(xh, w, bias)) : g;
}

// Sums of d and d xh over the slab, and the columns' dw and db added to
// part[2][C] (written where `first`).
template <int DT>
__device__ float2 slab_sums(const GnArgs& a, const Slab& b, float2 st, float* part, bool first, float* red,
                            float* cw, float* cb) {
  float q[2] = {0.f, 0.f};
  for (int c = 0; c < b.cg; c += b.cols) {
    float dw = 0.f, db = 0.f;
    const bool on = b.on && c + b.c < b.cg;
    const int64_t ch = b.g * b.cg + c + b.c;
    if (on) {
      const float w = a.w != nullptr ? ld_param(a.w, ch * a.ws, a.wdt) : 1.f;
      const float bias = a.b != nullptr ? ld_param(a.b, ch * a.bs, a.wdt) : 0.f;
      for (int64_t t = b.s0 + b.r; t < b.s1; t += b.rows) {
        float xh;
        const float dz = dz_of<DT>(a, b, st, t, ch, w, bias, xh);
        dw = fmaf(dz, xh, dw);
        db += dz;
      }
      q[0] = fmaf(db, w, q[0]);
      q[1] = fmaf(dw, w, q[1]);
    }
    if (part != nullptr) {
      __syncthreads();
      cw[threadIdx.x] = dw, cb[threadIdx.x] = db;
      __syncthreads();
      if (on && b.r == 0) {
        for (int r = 1; r < b.rows; ++r) dw += cw[r * b.cols + b.c], db += cb[r * b.cols + b.c];
        part[ch] = first ? dw : part[ch] + dw;
        part[a.C + ch] = first ? db : part[a.C + ch] + db;
      }
    }
  }
  block_sum(q, red);
  return make_float2(q[0], q[1]);
}

template <int DT>
__device__ void slab_dx(const GnArgs& a, const Slab& b, float2 st, float2 q) {
  using F = Fmt<DT>;
  if (!b.on) return;
  const float inv = 1.f / (static_cast<float>(a.S) * static_cast<float>(b.cg));
  const float c1 = q.x * inv, c2 = q.y * inv;
  for (int c = b.c; c < b.cg; c += b.cols) {
    const int64_t ch = b.g * b.cg + c;
    const float w = a.w != nullptr ? ld_param(a.w, ch * a.ws, a.wdt) : 1.f;
    const float bias = a.b != nullptr ? ld_param(a.b, ch * a.bs, a.wdt) : 0.f;
    for (int64_t t = b.s0 + b.r; t < b.s1; t += b.rows) {
      float xh;
      const float dz = dz_of<DT>(a, b, st, t, ch, w, bias, xh);
      static_cast<typename F::E*>(a.dx)[b.n * a.dxs[0] + t * a.dxs[1] + ch * a.dxs[2]] =
          F::from_f(st.y * (dz * w - c1 - xh * c2));
    }
  }
}

// A block takes samples slot, slot + slots, ... of one group and slab.
template <int DT, bool WHOLE>
__global__ void __launch_bounds__(kMaxThreads) gn_any_bwd_sums(const GnArgs a, const GnPlan p) {
  pdl_enter();
  __shared__ float red[2 * kMaxThreads / 32], cw[kMaxThreads], cb[kMaxThreads];
  const int64_t k = blockIdx.x % p.slabs, pg = blockIdx.x / p.slabs, slot = pg / a.G, g = pg % a.G;
  float* part = a.part != nullptr ? a.part + (slot * p.slabs + k) * 2 * a.C : nullptr;
  for (int64_t n = slot; n < a.N; n += p.slots) {
    const Slab b(a, p, n, g, k);
    float2 st;
    if constexpr (WHOLE) {
      st = slab_stats<DT>(a, b, red);
      st.y = rsqrtf(st.y / b.count() + a.eps);
    } else {
      st = merged_stats(a, p, b, red);
    }
    const float2 q = slab_sums<DT>(a, b, st, part, n == slot, red, cw, cb);
    if constexpr (WHOLE) {
      slab_dx<DT>(a, b, st, q);
    } else if (threadIdx.x == 0) {
      a.sums[(n * a.G + g) * p.slabs + k] = q;
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(kMaxThreads) gn_any_bwd_dx(const GnArgs a, const GnPlan p) {
  pdl_enter();
  __shared__ float red[2 * kMaxThreads / 32];
  const Slab b = slab_of(a, p);
  const float2 st = merged_stats(a, p, b, red);
  const float2* sums = a.sums + (b.n * a.G + b.g) * p.slabs;
  float q[2] = {0.f, 0.f};
  for (int64_t k = threadIdx.x; k < p.slabs; k += blockDim.x) q[0] += sums[k].x, q[1] += sums[k].y;
  block_sum(q, red);
  slab_dx<DT>(a, b, st, make_float2(q[0], q[1]));
}

// Few blocks of many elements take 1024 threads: 3 x 77 x 1000 in eight groups,
// FP32, 7.9 us instead of 10.2.
unsigned block_threads(const GnArgs& a, const GnPlan& p) {
  return a.N * a.G * p.slabs <= 2 * 152 && p.rows * (a.C / a.G) >= 4096 ? kMaxThreads : kThreads;
}

template <int DT>
cudaError_t fwd_dt(const GnArgs& a, cudaStream_t s) {
  const GnPlan p = gn_plan(a.N, a.S, a.C, a.G);
  const unsigned grid = static_cast<unsigned>(a.N * a.G * p.slabs);
  if (p.slabs == 1) return launch_pdl(gn_any_fwd<DT, true>, grid, block_threads(a, p), 0, s, a, p);
  const cudaError_t e = launch_pdl(gn_any_stats<DT>, grid, block_threads(a, p), 0, s, a, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(gn_any_fwd<DT, false>, grid, block_threads(a, p), 0, s, a, p);
}

template <int DT>
cudaError_t bwd_dt(const GnArgs& a, cudaStream_t s) {
  const GnPlan p = gn_plan(a.N, a.S, a.C, a.G);
  const unsigned grid = static_cast<unsigned>(a.N * a.G * p.slabs);
  const unsigned sums = static_cast<unsigned>(p.slots * a.G * p.slabs);
  if (p.slabs == 1) return launch_pdl(gn_any_bwd_sums<DT, true>, sums, block_threads(a, p), 0, s, a, p);
  cudaError_t e = launch_pdl(gn_any_stats<DT>, grid, block_threads(a, p), 0, s, a, p);
  if (e == cudaSuccess) e = launch_pdl(gn_any_bwd_sums<DT, false>, sums, block_threads(a, p), 0, s, a, p);
  if (e == cudaSuccess) e = launch_pdl(gn_any_bwd_dx<DT>, grid, block_threads(a, p), 0, s, a, p);
  return e;
}

}  // namespace

// Slabs enough for eight blocks an SM of 152 unless that leaves them below
// 8192 elements, and never more positions than fill 2^18 elements, the last one
// rounded up: at most 2048 elements a thread and sum.
GnPlan gn_plan(int64_t N, int64_t S, int64_t C, int64_t G) {
  GnPlan p = {1, S > 0 ? S : 1, 1};
  if (N <= 0 || S <= 0 || C <= 0 || G <= 0) return p;
  const int64_t elems = S * (C / G);
  int64_t slabs = 1216 / (N * G);
  if (slabs > elems / 8192) slabs = elems / 8192;
  const int64_t least = (elems + (1 << 18) - 1) >> 18;
  if (slabs < least) slabs = least;
  if (slabs < 1) slabs = 1;
  if (slabs > S) slabs = S;
  p.rows = (S + slabs - 1) / slabs;
  p.slabs = (S + p.rows - 1) / p.rows;
  p.slots = 1216 / (G * p.slabs);
  if (p.slots < 1) p.slots = 1;
  if (p.slots > N) p.slots = N;
  return p;
}

int64_t gn_parts(int64_t N, int64_t S, int64_t C, int64_t G) {
  const GnPlan p = gn_plan(N, S, C, G);
  int64_t most = p.slots * p.slabs;
  if (gn_narrow_eligible(S, C, G)) {
    const int64_t n = gn_narrow_slots(N, C, G);
    if (n > most) most = n;
  }
  for (const int64_t esize : {2, 4}) {
    const int64_t v = 16 / esize;
    if (C / G % v != 0) continue;
    const int64_t n = S == 1 && C / G / v <= 128 ? gn_rows_slots(N, C, G, esize, true) : 0;
    const int64_t m = gn_cluster_parts(N, S, C, G, esize);
    if (n > most) most = n;
    if (m > most) most = m;
  }
  return most;
}

cudaError_t launch_gn_fwd(const GnArgs& a, Dtype dt, cudaStream_t stream) {
  if (gn_rows_eligible(a, dt, false)) return launch_gn_rows(a, dt, false, stream);
  if (gn_narrow_eligible(a.S, a.C, a.G)) return launch_gn_narrow(a, dt, false, stream);
  if (gn_cluster_eligible(a, dt, false)) return launch_gn_cluster(a, dt, false, stream);
  switch (dt) {
    case kF32: return fwd_dt<kF32>(a, stream);
    case kF16: return fwd_dt<kF16>(a, stream);
    case kBF16: return fwd_dt<kBF16>(a, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_gn_bwd(const GnArgs& a, Dtype dt, cudaStream_t stream) {
  const bool some = a.N > 0 && a.S > 0;
  const int64_t esize = dt == kF32 ? 4 : 2;
  int64_t parts = 0;
  cudaError_t e = cudaSuccess;
  if (some && gn_rows_eligible(a, dt, true)) {
    e = launch_gn_rows(a, dt, true, stream);
    parts = gn_rows_slots(a.N, a.C, a.G, esize, true);
  } else if (some && gn_narrow_eligible(a.S, a.C, a.G)) {
    e = launch_gn_narrow(a, dt, true, stream);
    parts = gn_narrow_slots(a.N, a.C, a.G);
  } else if (some && gn_cluster_eligible(a, dt, true)) {
    e = launch_gn_cluster(a, dt, true, stream);
    parts = gn_cluster_parts(a.N, a.S, a.C, a.G, esize);
  } else if (some) {
    switch (dt) {
      case kF32: e = bwd_dt<kF32>(a, stream); break;
      case kF16: e = bwd_dt<kF16>(a, stream); break;
      case kBF16: e = bwd_dt<kBF16>(a, stream); break;
    }
    const GnPlan p = gn_plan(a.N, a.S, a.C, a.G);
    parts = p.slots * p.slabs;
  }
  if (e != cudaSuccess || (a.dw == nullptr && a.db == nullptr)) return e;
  return launch_param_sums(a.part, parts, a.C, a.dw, a.dws, a.db, a.dbs, a.wdt, stream);
}

}  // namespace ccv

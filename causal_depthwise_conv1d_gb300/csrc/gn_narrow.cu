// Group normalisation of rows on their own (S = 1) in groups that are no whole
// vectors, any strides: as gn_rows.cu with single elements, LPG lanes a group
// and NV channels a lane.  A block a group, as gn.cu has for every other case,
// would leave 250 of 256 threads idle in groups of six channels: 179200 x 36 in
// bf16 takes 28 us here (0.9 TB/s), bound by loads of single elements.
#include "ccv_common.cuh"
#include "rec_internal.h"
#include "rec_pairs.cuh"

namespace ccv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWidest = 256;

template <int LPG, int NS>
__device__ __forceinline__ void lanes_sum(float (&v)[NS]) {
#pragma unroll
  for (int m = LPG / 2; m > 0; m >>= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] += __shfl_xor_sync(kFullMask, v[i], m);
}

template <int DT, int LPG, int NV, bool BWD>
__global__ void __launch_bounds__(kThreads) gn_narrow_kernel(const GnArgs a, int colblocks) {
  using F = Fmt<DT>;
  using E = typename F::E;
  __shared__ float sums[BWD ? kWarps : 1][32][NV];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPG;
  const int64_t cb = blockIdx.x % colblocks, slot = blockIdx.x / colblocks;
  const int64_t g = cb * (32 / LPG) + lane / LPG;
  const int cg = static_cast<int>(a.C / a.G);
  const float inv = 1.f / static_cast<float>(cg);
  const int64_t step = static_cast<int64_t>(gridDim.x / colblocks) * kWarps;
  float w[NV], b[NV], dw[NV], db[NV];
  bool in[NV];
  int64_t ch[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = sub + i * LPG;
    ch[i] = g * cg + col;
    in[i] = g < a.G && col < cg;
    w[i] = a.w == nullptr ? 1.f : in[i] ? ld_param(a.w, ch[i] * a.ws, a.wdt) : 0.f;
    b[i] = a.b == nullptr || !in[i] ? 0.f : ld_param(a.b, ch[i] * a.bs, a.wdt);
    dw[i] = db[i] = 0.f;
  }
  E rx[NV], rg[NV];
  auto fetch = [&](int64_t n) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool on = in[i] && n < a.N;
      rx[i] = on ? static_cast<const E*>(a.x)[n * a.xs[0] + ch[i] * a.xs[2]] : E(0);
      if (BWD) rg[i] = on ? static_cast<const E*>(a.dout)[n * a.gs[0] + ch[i] * a.gs[2]] : E(0);
    }
  };
  int64_t n = slot * kWarps + warp;
  fetch(n);
  for (; n < a.N; n += step) {
    float f[NV], d[NV], s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      f[i] = F::to_f(rx[i]);
      if (BWD) d[i] = F::to_f(rg[i]);
      s[0] += f[i];
    }
    fetch(n + step);
    lanes_sum<LPG>(s);
    const float mean = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      f[i] = in[i] ? f[i] - mean : 0.f;
      s[0] = fmaf(f[i], f[i], s[0]);
    }
    lanes_sum<LPG>(s);
    const float r = rsqrtf(fmaf(s[0], inv, a.eps));
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      f[i] *= r;
      if constexpr (BWD) {
        if (a.silu) d[i] *= silu_grad_cut(fmaf(f[i], w[i], b[i]));
        dw[i] = fmaf(d[i], f[i], dw[i]);
        db[i] += d[i];
        d[i] *= w[i];
        q[0] += d[i];
        q[1] = fmaf(d[i], f[i], q[1]);
      } else if (in[i]) {
        const float z = fmaf(f[i], w[i], b[i]);
        static_cast<E*>(a.out)[n * a.os[0] + ch[i] * a.os[2]] = F::from_f(a.silu ? silu(z) : z);
      }
    }
    if constexpr (BWD) {
      lanes_sum<LPG>(q);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in[i])
          static_cast<E*>(a.dx)[n * a.dxs[0] + ch[i] * a.dxs[2]] =
              F::from_f(r * (d[i] - q[0] * inv - f[i] * (q[1] * inv)));
    }
  }
  if constexpr (BWD) {
    if (a.part == nullptr) return;
    // the block's warps in order, one partial sum a block
    float* part = a.part + slot * 2 * a.C;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) sums[warp][lane][i] = which == 0 ? dw[i] : db[i];
      __syncthreads();
      if (warp == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float v = 0.f;
#pragma unroll
          for (int k = 0; k < kWarps; ++k) v += sums[k][lane][i];
          if (in[i]) part[which * a.C + ch[i]] = v;
        }
    }
  }
}

struct Shape {
  int lpg, nv;
};
Shape shape_of(int64_t cg) {
  if (cg <= 8) return {8, 1};
  if (cg <= 32) return {32, 1};
  if (cg <= 64) return {32, 2};
  return {32, 8};
}

template <int DT, int LPG, int NV>
cudaError_t launch(const GnArgs& a, bool bwd, cudaStream_t s) {
  const int colblocks = static_cast<int>((a.G + 32 / LPG - 1) / (32 / LPG));
  const unsigned grid = static_cast<unsigned>(colblocks * gn_narrow_slots(a.N, a.C, a.G));
  if (bwd) return launch_pdl(gn_narrow_kernel<DT, LPG, NV, true>, grid, kThreads, 0, s, a, colblocks);
  return launch_pdl(gn_narrow_kernel<DT, LPG, NV, false>, grid, kThreads, 0, s, a, colblocks);
}

template <int DT>
cudaError_t launch_dt(const GnArgs& a, bool bwd, cudaStream_t s) {
  const Shape h = shape_of(a.C / a.G);
  return h.lpg == 8   ? launch<DT, 8, 1>(a, bwd, s)
         : h.nv == 1  ? launch<DT, 32, 1>(a, bwd, s)
         : h.nv == 2  ? launch<DT, 32, 2>(a, bwd, s)
                      : launch<DT, 32, 8>(a, bwd, s);
}

}  // namespace

bool gn_narrow_eligible(int64_t S, int64_t C, int64_t G) { return S == 1 && C / G <= kWidest; }

// Blocks side by side over the rows: four an SM (152 of them) over the column blocks.
int64_t gn_narrow_slots(int64_t N, int64_t C, int64_t G) {
  const Shape h = shape_of(C / G);
  const int64_t colblocks = (G + 32 / h.lpg - 1) / (32 / h.lpg), rows = (N + kWarps - 1) / kWarps;
  int64_t slots = (152 * 4 + colblocks - 1) / colblocks;
  if (slots > rows) slots = rows;
  return slots < 1 ? 1 : slots;
}

cudaError_t launch_gn_narrow(const GnArgs& a, Dtype dt, bool bwd, cudaStream_t s) {
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, bwd, s);
    case kF16: return launch_dt<kF16>(a, bwd, s);
    case kBF16: return launch_dt<kBF16>(a, bwd, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ccv

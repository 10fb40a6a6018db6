// Gated delta rule, the decode step of a serving batch: one token a request
// against states in a cache.
//
//   S <- a S + k u^T,  u = beta (v - a p),  o = scale (a r + (q.k) u),  p = k^T S,  r = q^T S
//
// (gdr_token.cu has the derivation).  One sweep over the state in registers
// gives p and r, one exchange between the warps sums them, and a second sweep
// writes the new state: each state element is read and written once.
//
// What bounds it: HBM, 8 bytes a state element.  A block owns 64 columns of
// one head; a thread holds four adjacent columns of every 16th row, so a
// warp's loads are two 256-byte row pieces, all rows in flight at once, and
// four blocks an SM overlap their loads, exchanges and stores.  128 requests x
// 32 heads of 128 x 128, 542 MB: 83.5 us, 6.5 TB/s, 0.96 of the copy rate (a
// block of 128 columns, two an SM: 104 us).  The block's indices are divided
// in 64 bits: with 32-bit divisions, which end some hundred cycles earlier,
// the same kernel measures 88.9 us in every run.
#include "ccv_common.cuh"
#include "mix_internal.h"

namespace ccv {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 64;
constexpr int kLanes = kCols / 4;         // lanes of one row
constexpr int kRows = kThreads / kLanes;  // rows of one sweep step
constexpr int kWarps = kThreads / 32;

template <int DT, int MAXK>
__global__ void __launch_bounds__(kThreads, 4) gdr_step_kernel(const GdrArgs a, int tiles) {
  using F = Fmt<DT>;
  using E = typename F::E;
  constexpr int R = MAXK / kRows;  // rows of one thread
  __shared__ float sk[MAXK], sq[MAXK];
  __shared__ __align__(16) float red[2][kWarps][kCols];
  __shared__ float redqk[kWarps];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cl = tid % kLanes, rg = tid / kLanes;
  const int64_t bh = blockIdx.x / tiles;
  const int64_t b = bh / a.Hv, h = bh - b * a.Hv;
  const int64_t hk = h / (a.Hv / a.Hk);
  const int64_t col = static_cast<int64_t>(blockIdx.x % tiles) * kCols + cl * 4;
  const bool in = col < a.Dv;  // Dv is a multiple of four here
  const int64_t slot = a.slots != nullptr ? a.slots[b * a.slot_stride] : b;
  E* out = static_cast<E*>(a.out) + b * a.os[0] + h * a.os[2];
  if (slot < 0 || slot >= a.n_slots) {  // a padding row: no state, zero outputs
    if (rg == 0 && in)
      for (int j = 0; j < 4; ++j) out[(col + j) * a.os[3]] = F::from_f(0.f);
    return;
  }
  const float* sp = a.s0 + slot * a.s0s[0] + h * a.s0s[1] + col;
  float4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = rg + kRows * i;
    s[i] = in && row < a.Dk ? *reinterpret_cast<const float4*>(sp + row * a.s0s[2]) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float qk = 0.f;
  if (tid < MAXK) {
    const float kv = tid < a.Dk ? F::to_f(static_cast<const E*>(a.k)[b * a.ks[0] + hk * a.ks[2] + tid * a.ks[3]]) : 0.f;
    const float qv = tid < a.Dk ? F::to_f(static_cast<const E*>(a.q)[b * a.qs[0] + hk * a.qs[2] + tid * a.qs[3]]) : 0.f;
    sk[tid] = kv;
    sq[tid] = qv;
    qk = kv * qv;
  }
  const float dec = expf(a.g[b * a.gs[0] + h * a.gs[2]]);
  const float bet = F::to_f(static_cast<const E*>(a.beta)[b * a.bs[0] + h * a.bs[2]]);
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = in ? F::to_f(static_cast<const E*>(a.v)[b * a.vs[0] + h * a.vs[2] + (col + j) * a.vs[3]]) : 0.f;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) qk += __shfl_xor_sync(kFullMask, qk, m);
  if (lane == 0) redqk[warp] = qk;
  __syncthreads();

  float p[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float kv = sk[rg + kRows * i], qv = sq[rg + kRows * i];
    p[0] = fmaf(kv, s[i].x, p[0]), p[1] = fmaf(kv, s[i].y, p[1]);
    p[2] = fmaf(kv, s[i].z, p[2]), p[3] = fmaf(kv, s[i].w, p[3]);
    r[0] = fmaf(qv, s[i].x, r[0]), r[1] = fmaf(qv, s[i].y, r[1]);
    r[2] = fmaf(qv, s[i].z, r[2]), r[3] = fmaf(qv, s[i].w, r[3]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    p[j] += __shfl_xor_sync(kFullMask, p[j], 16);
    r[j] += __shfl_xor_sync(kFullMask, r[j], 16);
  }
  if (lane < kLanes) {
    *reinterpret_cast<float4*>(&red[0][warp][cl * 4]) = make_float4(p[0], p[1], p[2], p[3]);
    *reinterpret_cast<float4*>(&red[1][warp][cl * 4]) = make_float4(r[0], r[1], r[2], r[3]);
  }
  __syncthreads();
  qk = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = r[j] = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    qk += redqk[w];
    const float4 x = *reinterpret_cast<const float4*>(&red[0][w][cl * 4]);
    p[0] += x.x, p[1] += x.y, p[2] += x.z, p[3] += x.w;
  }
  float u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = bet * (v[j] - dec * p[j]);
  if (!in) return;
  float* wp = a.s1 + slot * a.s1s[0] + h * a.s1s[1] + col;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = rg + kRows * i;
    const float kv = sk[row];
    if (row < a.Dk)
      *reinterpret_cast<float4*>(wp + row * a.s1s[2]) =
          make_float4(fmaf(kv, u[0], dec * s[i].x), fmaf(kv, u[1], dec * s[i].y), fmaf(kv, u[2], dec * s[i].z),
                      fmaf(kv, u[3], dec * s[i].w));
  }
  if (rg == 0) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(&red[1][w][cl * 4]);
      r[0] += x.x, r[1] += x.y, r[2] += x.z, r[3] += x.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) out[(col + j) * a.os[3]] = F::from_f(a.scale * fmaf(qk, u[j], dec * r[j]));
  }
}

template <int DT, int MAXK>
cudaError_t launch_tile(const GdrArgs& a, cudaStream_t s) {
  const int64_t tiles = (a.Dv + kCols - 1) / kCols, grid = a.B * a.Hv * tiles;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  gdr_step_kernel<DT, MAXK><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, static_cast<int>(tiles));
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_dt(const GdrArgs& a, cudaStream_t s) {
  return a.Dk <= 64 ? launch_tile<DT, 64>(a, s) : launch_tile<DT, 128>(a, s);
}

}  // namespace

// One token, whole four-column pieces, and enough heads to give every SM four
// blocks: then the state's bytes count; below that a token's latency does, and
// gdr_token.cu takes it.
bool gdr_step_eligible(const GdrArgs& a, const Device& dev) {
  return a.L == 1 && a.seq == nullptr && a.Dk <= 128 && a.Dv % 4 == 0 && a.s0 != nullptr && a.s1 != nullptr &&
         gdr_vec4_state(a.s0, a.s0s) && gdr_vec4_state(a.s1, a.s1s) &&
         a.B * a.Hv * ((a.Dv + kCols - 1) / kCols) >= 4 * static_cast<int64_t>(dev.sm_count);
}

cudaError_t launch_gdr_step(const GdrArgs& a, Dtype dt, cudaStream_t stream) {
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, stream);
    case kF16: return launch_dt<kF16>(a, stream);
    case kBF16: return launch_dt<kBF16>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ccv

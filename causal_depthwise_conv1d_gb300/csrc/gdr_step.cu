// Gated delta rule, one token after the other, the state in registers.
//
// Per value head, with the state S [Dk, Dv] in FP32:
//
//   S <- a S,  a = exp(g);   u = beta (v - k^T S);   S <- S + k u^T;   o = scale q^T S
//
// Both products of a token are taken from the state as it was before it:
// with p = k^T S and r = q^T S,  u = beta (v - a p)  and
// o = scale (a r + (q.k) u),  so one sweep over the registers gives p and r,
// one exchange between the row groups sums them, and a second sweep writes
// a S + k u^T.  A decode step reads and writes each state element once.
//
// What bounds it: HBM (8 bytes a state element) for serving batches, latency
// for a single request.  A block owns one head and a tile of columns; a thread
// holds VEC adjacent columns of every RG-th row, so a warp's loads are whole
// 128- or 256-byte row pieces, all in flight at once.
#include "ccv_common.cuh"
#include "mix_internal.h"

namespace ccv {
namespace {

constexpr int kThreads = 256;
constexpr int kTok = 8;  // tokens staged at a time

// MAXK: rows of the register tile (Dk <= MAXK); CL lanes of VEC columns.
template <int DT, int MAXK, int CL, int VEC>
__global__ void __launch_bounds__(kThreads, MAXK * CL * VEC > 8192 ? 2 : 4) gdr_step_kernel(const GdrArgs a, int tiles) {
  using F = Fmt<DT>;
  using E = typename F::E;
  constexpr int RG = kThreads / CL;   // row groups
  constexpr int R = MAXK / RG;        // rows of one thread
  constexpr int COLS = CL * VEC;
  constexpr int NW = kThreads / 32;
  __shared__ float sk[kTok][MAXK], sq[kTok][MAXK];
  __shared__ float sv[kTok][COLS];
  __shared__ float sa[kTok], sb[kTok];
  __shared__ __align__(16) float red[2][2][NW][COLS];  // of even and odd tokens: one barrier a token
  __shared__ float redqk[2][NW];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cl = tid % CL, rg = tid / CL;
  const int64_t bh = blockIdx.x / tiles;
  const int64_t b = bh / a.Hv, h = bh - b * a.Hv;
  const int64_t hk = h / (a.Hv / a.Hk);
  const int64_t col0 = static_cast<int64_t>(blockIdx.x % tiles) * COLS;
  const int64_t col = col0 + cl * VEC;
  const int64_t Dk = a.Dk, Dv = a.Dv;
  const bool incol = col < Dv;  // VEC > 1 only where Dv is a multiple of VEC

  int64_t slot = b;
  if (a.slots != nullptr) {
    slot = a.slots[b * a.slot_stride];
    if (slot < 0 || slot >= a.n_slots) {  // a padding row: no state, zero outputs
      for (int64_t t = rg; t < a.L; t += RG)
        for (int j = 0; j < VEC; ++j)
          if (col + j < Dv)
            static_cast<E*>(a.out)[b * a.os[0] + t * a.os[1] + h * a.os[2] + (col + j) * a.os[3]] = F::from_f(0.f);
      return;
    }
  }

  float s[R][VEC];
  const float* sp = a.s0 == nullptr ? nullptr : a.s0 + slot * a.s0s[0] + h * a.s0s[1] + col * a.s0s[3];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = rg + RG * i;
    const bool in = sp != nullptr && incol && row < Dk;
    if constexpr (VEC == 4) {
      const float4 x = in ? *reinterpret_cast<const float4*>(sp + row * a.s0s[2]) : make_float4(0.f, 0.f, 0.f, 0.f);
      s[i][0] = x.x, s[i][1] = x.y, s[i][2] = x.z, s[i][3] = x.w;
    } else {
      s[i][0] = in ? sp[row * a.s0s[2]] : 0.f;
    }
  }

  for (int64_t t0 = 0; t0 < a.L; t0 += kTok) {
    const int nt = static_cast<int>(a.L - t0 < kTok ? a.L - t0 : kTok);
    __syncthreads();
    for (int i = tid; i < nt * MAXK; i += kThreads) {
      const int t = i / MAXK, r = i % MAXK;
      float kv = 0.f, qv = 0.f;
      if (r < Dk) {
        kv = F::to_f(static_cast<const E*>(a.k)[b * a.ks[0] + (t0 + t) * a.ks[1] + hk * a.ks[2] + r * a.ks[3]]);
        qv = F::to_f(static_cast<const E*>(a.q)[b * a.qs[0] + (t0 + t) * a.qs[1] + hk * a.qs[2] + r * a.qs[3]]);
      }
      sk[t][r] = kv;
      sq[t][r] = qv;
    }
    for (int i = tid; i < nt * COLS; i += kThreads) {
      const int t = i / COLS, c = i % COLS;
      sv[t][c] = col0 + c < Dv ? F::to_f(static_cast<const E*>(a.v)[b * a.vs[0] + (t0 + t) * a.vs[1] + h * a.vs[2] +
                                                                    (col0 + c) * a.vs[3]])
                               : 0.f;
    }
    if (tid < nt) {
      const int64_t t = t0 + tid;
      float dec = expf(a.g[b * a.gs[0] + t * a.gs[1] + h * a.gs[2]]);
      // a new sequence: its first token sees the zero state (marked by a negative decay)
      if (a.seq != nullptr && t > 0 && a.seq[b * a.ss[0] + t * a.ss[1]] != a.seq[b * a.ss[0] + (t - 1) * a.ss[1]])
        dec = -1.f;
      sa[tid] = dec;
      sb[tid] = F::to_f(static_cast<const E*>(a.beta)[b * a.bs[0] + t * a.bs[1] + h * a.bs[2]]);
    }
    __syncthreads();

    for (int t = 0; t < nt; ++t) {
      float dec = sa[t];
      const float bet = sb[t];
      if (dec == -1.f) {  // selected, not multiplied: a state with infinities must not leak
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) s[i][j] = 0.f;
        dec = 0.f;
      }
      float p[VEC], r[VEC], qk = 0.f;
#pragma unroll
      for (int j = 0; j < VEC; ++j) p[j] = r[j] = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float kv = sk[t][rg + RG * i], qv = sq[t][rg + RG * i];
        qk = fmaf(kv, qv, qk);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          p[j] = fmaf(kv, s[i][j], p[j]);
          r[j] = fmaf(qv, s[i][j], r[j]);
        }
      }
      // sum over the row groups: within the warp, then between the warps
#pragma unroll
      for (int m = CL; m < 32; m <<= 1) {
        qk += __shfl_xor_sync(kFullMask, qk, m);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          p[j] += __shfl_xor_sync(kFullMask, p[j], m);
          r[j] += __shfl_xor_sync(kFullMask, r[j], m);
        }
      }
      if (lane < CL) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          red[t & 1][0][warp][cl * VEC + j] = p[j];
          red[t & 1][1][warp][cl * VEC + j] = r[j];
        }
        if (lane == 0) redqk[t & 1][warp] = qk;
      }
      __syncthreads();
      qk = 0.f;
#pragma unroll
      for (int j = 0; j < VEC; ++j) p[j] = r[j] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        qk += redqk[t & 1][w];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          p[j] += red[t & 1][0][w][cl * VEC + j];
          r[j] += red[t & 1][1][w][cl * VEC + j];
        }
      }
      float u[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) u[j] = bet * (sv[t][cl * VEC + j] - dec * p[j]);
      if (rg == 0) {
        E* o = static_cast<E*>(a.out) + b * a.os[0] + (t0 + t) * a.os[1] + h * a.os[2];
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (col + j < Dv) o[(col + j) * a.os[3]] = F::from_f(a.scale * fmaf(qk, u[j], dec * r[j]));
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float kv = sk[t][rg + RG * i];
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[i][j] = fmaf(kv, u[j], dec * s[i][j]);
      }
    }
  }

  if (a.s1 != nullptr && incol) {
    float* wp = a.s1 + slot * a.s1s[0] + h * a.s1s[1] + col * a.s1s[3];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int row = rg + RG * i;
      if (row < Dk) {
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(wp + row * a.s1s[2]) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
        else
          wp[row * a.s1s[2]] = s[i][0];
      }
    }
  }
}

template <int DT, int MAXK, int CL, int VEC>
cudaError_t launch_tile(const GdrArgs& a, cudaStream_t s) {
  const int64_t cols = CL * VEC, tiles = (a.Dv + cols - 1) / cols;
  const int64_t grid = a.B * a.Hv * tiles;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  gdr_step_kernel<DT, MAXK, CL, VEC><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, static_cast<int>(tiles));
  return cudaGetLastError();
}

bool vec4_state(const float* p, const int64_t* st) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && st[3] == 1 && st[0] % 4 == 0 && st[1] % 4 == 0 &&
                          st[2] % 4 == 0);
}

template <int DT, int MAXK>
cudaError_t launch_k(const GdrArgs& a, const Device& dev, cudaStream_t s) {
  const bool vec = a.Dv % 4 == 0 && vec4_state(a.s0, a.s0s) && vec4_state(a.s1, a.s1s);
  if (!vec) return launch_tile<DT, MAXK, 32, 1>(a, s);
  // Narrow tiles while half rows would not give every SM four blocks: more
  // blocks share one head's latency.  Half rows of 64 columns once they do.
  if (a.B * a.Hv * ((a.Dv + 63) / 64) < 4 * dev.sm_count) return launch_tile<DT, MAXK, 8, 4>(a, s);
  return launch_tile<DT, MAXK, 16, 4>(a, s);
}

template <int DT>
cudaError_t launch_dt(const GdrArgs& a, const Device& dev, cudaStream_t s) {
  if (a.Dk <= 64) return launch_k<DT, 64>(a, dev, s);
  if (a.Dk <= 128) return launch_k<DT, 128>(a, dev, s);
  if (a.Dk <= kGdrMaxDk) return launch_tile<DT, 256, 32, 1>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_gdr_step(const GdrArgs& a, Dtype dt, const Device& dev, cudaStream_t stream) {
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, dev, stream);
    case kF16: return launch_dt<kF16>(a, dev, stream);
    case kBF16: return launch_dt<kBF16>(a, dev, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ccv

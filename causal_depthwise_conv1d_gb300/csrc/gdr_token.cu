// Gated delta rule, one token after the other, the state in registers: short
// sequences, sizes the chunked kernels do not take, and decode steps of
// several tokens or few requests.
//
// Per value head, with the state S [Dk, Dv] in FP32:
//
//   S <- a S,  a = exp(g);   u = beta (v - k^T S);   S <- S + k u^T;   o = scale q^T S
//
// Both products of a token are taken from the state as it was before it:
// with p = k^T S and r = q^T S,  u = beta (v - a p)  and  o = scale (a r + (q.k) u).
//
// What bounds it: the latency of a token's chain.  A warp owns four columns
// and all rows (R of them a lane), so a token needs no barrier: the eight sums
// p and r go through a halving exchange (4 + 2 + 1 + 1 + 1 shuffles), four
// lanes form u, four shuffles hand it back.  A block is eight warps on 32
// columns of one head that share the tokens' k, q, v and gates, staged kTok
// at a time, the next ones while these are worked on.  128 x 128 heads, bf16:
// 0.37 us a token once running; one token of one request with 32 heads (4.2 MB
// of states) 6.2 us a call, of which 4.2 us are left when calls are replayed
// from a graph; five tokens of 16 requests x 16 heads 14.3 us.  Fetching a
// token's operands into registers one token ahead measured 0.49 us a token.
#include "ccv_common.cuh"
#include "mix_internal.h"

namespace ccv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCols = 4;                    // columns of a warp
constexpr int kBlockCols = kWarps * kCols;
constexpr int kTok = 8;                     // tokens of one stage: one a warp

// A store under a predicate instead of a branch: the token loop stays converged.
__device__ __forceinline__ void store_if(uint16_t* p, uint16_t v, bool on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.u16 [%0], %1;\n\t}" ::"l"(p), "h"(v),
               "r"(static_cast<uint32_t>(on))
               : "memory");
}
__device__ __forceinline__ void store_if(uint32_t* p, uint32_t v, bool on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.u32 [%0], %1;\n\t}" ::"l"(p), "r"(v),
               "r"(static_cast<uint32_t>(on))
               : "memory");
}

template <int DT, int R>
__global__ void __launch_bounds__(kThreads) gdr_token_kernel(const GdrArgs a, unsigned tiles, bool svec, bool kvec) {
  using F = Fmt<DT>;
  using E = typename F::E;
  constexpr int MAXK = 32 * R;
  // two stages: k and q of a token interleaved by lane (R of k, R of q)
  __shared__ __align__(16) float skq[2][kTok][2 * MAXK];
  __shared__ float sv[2][kTok][kBlockCols];
  __shared__ float4 sg[2][kTok];  // decay, beta, q.k, 1 where a new sequence begins

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // indices below 2^31 (checked on the host): 32-bit divisions
  const unsigned Hv = static_cast<unsigned>(a.Hv), ubh = blockIdx.x / tiles, ub = ubh / Hv, uh = ubh - ub * Hv;
  const int64_t b = ub, h = uh, hk = uh / (Hv / static_cast<unsigned>(a.Hk));
  const int64_t bcol = static_cast<int64_t>(blockIdx.x % tiles) * kBlockCols;
  const int64_t col = bcol + warp * kCols;
  const int row0 = lane * R;
  const int64_t Dk = a.Dk, Dv = a.Dv;

  // The warp's token of the stage that begins at t0: into registers, then to shared memory.
  float lk[R], lq[R], lv = 0.f, lg = 0.f, lb = 0.f;
  bool lnew = false;
  auto fetch = [&](int64_t t0) {
    const int64_t t = t0 + warp;
#pragma unroll
    for (int i = 0; i < R; ++i) lk[i] = lq[i] = 0.f;
    lv = 0.f;
    if (t >= a.L) return;
    const E* kp = static_cast<const E*>(a.k) + b * a.ks[0] + t * a.ks[1] + hk * a.ks[2];
    const E* qp = static_cast<const E*>(a.q) + b * a.qs[0] + t * a.qs[1] + hk * a.qs[2];
    if (kvec) {  // R elements in words of at least 4 bytes
      constexpr int W = R * static_cast<int>(sizeof(E)) / 4;
      uint32_t wk[W], wq[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        wk[i] = __ldg(reinterpret_cast<const uint32_t*>(kp + row0) + i);
        wq[i] = __ldg(reinterpret_cast<const uint32_t*>(qp + row0) + i);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        lk[i] = F::word_elem(wk[i / F::PER_WORD], i % F::PER_WORD);
        lq[i] = F::word_elem(wq[i / F::PER_WORD], i % F::PER_WORD);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (row0 + i < Dk) {
          lk[i] = F::to_f(kp[(row0 + i) * a.ks[3]]);
          lq[i] = F::to_f(qp[(row0 + i) * a.qs[3]]);
        }
    }
    if (bcol + lane < Dv)
      lv = F::to_f(static_cast<const E*>(a.v)[b * a.vs[0] + t * a.vs[1] + h * a.vs[2] + (bcol + lane) * a.vs[3]]);
    lg = a.g[b * a.gs[0] + t * a.gs[1] + h * a.gs[2]];
    lb = F::to_f(static_cast<const E*>(a.beta)[b * a.bs[0] + t * a.bs[1] + h * a.bs[2]]);
    lnew = a.seq != nullptr && t > 0 && a.seq[b * a.ss[0] + t * a.ss[1]] != a.seq[b * a.ss[0] + (t - 1) * a.ss[1]];
  };
  auto put = [&](int s) {
    float qk = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      skq[s][warp][lane * 2 * R + i] = lk[i];
      skq[s][warp][lane * 2 * R + R + i] = lq[i];
      qk = fmaf(lk[i], lq[i], qk);
    }
    sv[s][warp][lane] = lv;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) qk += __shfl_xor_sync(kFullMask, qk, m);
    if (lane == 0) sg[s][warp] = make_float4(expf(lg), lb, qk, lnew ? 1.f : 0.f);
  };
  fetch(0);

  int64_t slot = b;
  if (a.slots != nullptr) {
    slot = a.slots[b * a.slot_stride];
    if (slot < 0 || slot >= a.n_slots) {  // a padding row: no state, zero outputs
      for (int64_t t = warp; t < a.L; t += kWarps)
        if (bcol + lane < Dv)
          static_cast<E*>(a.out)[b * a.os[0] + t * a.os[1] + h * a.os[2] + (bcol + lane) * a.os[3]] = F::from_f(0.f);
      return;
    }
  }

  float s[R][kCols];
  const float* sp = a.s0 == nullptr ? nullptr : a.s0 + slot * a.s0s[0] + h * a.s0s[1];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const bool in = sp != nullptr && row0 + i < Dk;
    if (svec) {
      const float4 x = in && col < Dv ? *reinterpret_cast<const float4*>(sp + (row0 + i) * a.s0s[2] + col)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
      s[i][0] = x.x, s[i][1] = x.y, s[i][2] = x.z, s[i][3] = x.w;
    } else {
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        s[i][j] = in && col + j < Dv ? sp[(row0 + i) * a.s0s[2] + (col + j) * a.s0s[3]] : 0.f;
    }
  }
  put(0);
  __syncthreads();

  const int vi = lane >> 2;   // the sum this lane holds after the exchange: p of column 0..3, r of column 0..3
  const int vc = vi & 3;
  // lanes 16, 20, 24, 28 write the outputs of the four columns
  const bool writes = lane >= 16 && (lane & 3) == 0 && col + vc < Dv;
  E* op = static_cast<E*>(a.out) + b * a.os[0] + h * a.os[2] + (col + vc) * a.os[3];
  int st = 0;
  for (int64_t t0 = 0; t0 < a.L; t0 += kTok, st ^= 1) {
    const int nt = static_cast<int>(a.L - t0 < kTok ? a.L - t0 : kTok);
    const bool more = t0 + kTok < a.L;
    if (more) fetch(t0 + kTok);
    for (int t = 0; t < nt; ++t) {
      const float4 gate = sg[st][t];
      const float vv = sv[st][t][warp * kCols + vc];
      float dec = gate.x;
      if (__any_sync(kFullMask, gate.w != 0.f)) {  // selected, not multiplied: a state with infinities must not leak
        dec = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < kCols; ++j) s[i][j] = 0.f;
      }
      float k[R], q[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        k[i] = skq[st][t][lane * 2 * R + i];
        q[i] = skq[st][t][lane * 2 * R + R + i];
      }
      float x[8];
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        x[j] = k[0] * s[0][j];
        x[4 + j] = q[0] * s[0][j];
#pragma unroll
        for (int i = 1; i < R; ++i) {
          x[j] = fmaf(k[i], s[i][j], x[j]);
          x[4 + j] = fmaf(q[i], s[i][j], x[4 + j]);
        }
      }
      // halving exchange: bit 4 of the lane chooses p or r, bits 3 and 2 the column
      float y[4], z[2], w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float mine = (lane & 16) ? x[4 + j] : x[j], other = (lane & 16) ? x[j] : x[4 + j];
        y[j] = mine + __shfl_xor_sync(kFullMask, other, 16);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float mine = (lane & 8) ? y[2 + j] : y[j], other = (lane & 8) ? y[j] : y[2 + j];
        z[j] = mine + __shfl_xor_sync(kFullMask, other, 8);
      }
      {
        const float mine = (lane & 4) ? z[1] : z[0], other = (lane & 4) ? z[0] : z[1];
        w = mine + __shfl_xor_sync(kFullMask, other, 4);
      }
      w += __shfl_xor_sync(kFullMask, w, 2);
      w += __shfl_xor_sync(kFullMask, w, 1);
      const float uw = gate.y * (vv - dec * w);  // u of column vc in the lanes below 16
      float u[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) u[j] = __shfl_sync(kFullMask, uw, 4 * j);
      const float uc = vc < 2 ? (vc == 0 ? u[0] : u[1]) : (vc == 2 ? u[2] : u[3]);
      store_if(op, F::from_f(a.scale * fmaf(gate.z, uc, dec * w)), writes);
      op += a.os[1];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < kCols; ++j) s[i][j] = fmaf(k[i], u[j], dec * s[i][j]);
    }
    // the other stage was left by every warp before the last barrier
    if (more) put(st ^ 1);
    __syncthreads();
  }

  if (a.s1 == nullptr) return;
  float* wp = a.s1 + slot * a.s1s[0] + h * a.s1s[1];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (row0 + i >= Dk) continue;
    if (svec) {
      if (col < Dv)
        *reinterpret_cast<float4*>(wp + (row0 + i) * a.s1s[2] + col) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    } else {
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        if (col + j < Dv) wp[(row0 + i) * a.s1s[2] + (col + j) * a.s1s[3]] = s[i][j];
    }
  }
}

template <int DT, int R>
cudaError_t launch(const GdrArgs& a, cudaStream_t s) {
  using E = typename Fmt<DT>::E;
  const int64_t tiles = (a.Dv + kBlockCols - 1) / kBlockCols, grid = a.B * a.Hv * tiles;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  constexpr int64_t W = 4 / sizeof(E);  // elements of a word
  auto words = [&](const void* p, const int64_t* st) {
    return st[3] == 1 && reinterpret_cast<uintptr_t>(p) % 4 == 0 && st[0] % W == 0 && st[1] % W == 0 && st[2] % W == 0;
  };
  const bool kvec = a.Dk == 32 * R && words(a.k, a.ks) && words(a.q, a.qs);
  const bool svec = a.Dv % 4 == 0 && gdr_vec4_state(a.s0, a.s0s) && gdr_vec4_state(a.s1, a.s1s);
  gdr_token_kernel<DT, R><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, static_cast<unsigned>(tiles), svec, kvec);
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_dt(const GdrArgs& a, cudaStream_t s) {
  if (a.Dk <= 64) return launch<DT, 2>(a, s);
  if (a.Dk <= 128) return launch<DT, 4>(a, s);
  if (a.Dk <= kGdrMaxDk) return launch<DT, 8>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace

bool gdr_vec4_state(const float* p, const int64_t* st) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && st[3] == 1 && st[0] % 4 == 0 && st[1] % 4 == 0 &&
                          st[2] % 4 == 0);
}

cudaError_t launch_gdr_token(const GdrArgs& a, Dtype dt, cudaStream_t stream) {
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, stream);
    case kF16: return launch_dt<kF16>(a, stream);
    case kBF16: return launch_dt<kBF16>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ccv

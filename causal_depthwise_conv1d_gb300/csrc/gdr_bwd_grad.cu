// Gated delta rule, backward: the gradients of q, k, g and beta, one block
// per chunk and key head.
//
// From the two scans: S0 (the state before the chunk), D (the gradient of the
// state after it), U, dR; and dO (scaled by `scale` below):
//
//   dP = dO U^T (j <= i),  A = dP Gam;   B = -(dR U^T) Gam (j < i);   Y = gi (dR S0^T)
//   Z  = B K - Y
//   dQ = gi (dO S0^T) + A K
//   dK = gc (U D^T) + beta Z + A^T Q + (beta B)^T K
//   dbeta_i = dR_i.v_i + k_i.Z_i
//   dG_i = q_i.dQ_i - k_i.dK_i + 2 beta_i k_i.Z_i,  and at the last token  + ga <S0, D> + sum_i k_i.(gc U D^T)_i
//   dg_t = sum of dG_i over the tokens i >= t of t's sequence in the chunk
//
// (the row sums of dP P and dL L are dot products of q and k with the products
// above, so neither matrix is formed again).  A chunk needs nothing of
// another, so all of them run at once; the value heads that share a key head
// are summed here one after the other, in registers and in a fixed order.
//
// What bounds it: the tensor instructions (about 7400 of 16 x 8 x 16 a chunk
// and head of 128 x 128, products of two FP32 operands taking three) and the
// reading of S0 and D.
#include "gdr_chunk.cuh"

namespace ccv {
namespace {

constexpr int kThreads = 256;
constexpr int kVB = 64;  // value channels staged at a time

template <int DT, int DK>
struct Cfg {
  static constexpr int TERMS = DT == kF32 ? 2 : 1;
  static constexpr int TILE = qk_tile_bytes(DK);
  static constexpr int QKB = qk_pack_bytes(DK, TERMS);
  static constexpr int TOK = kC * kVB * 2;                 // a [64 tokens][64 v] tile
  static constexpr int ST = DK * kVB * 2;                  // a [DK][64 v] tile
  static constexpr int BIG = 4 * ST > 8 * kMatBytes ? 4 * ST : 8 * kMatBytes;
  static constexpr int O_DO = QKB + kVecBytes;
  static constexpr int O_DR = O_DO + TERMS * TOK;
  static constexpr int O_U = O_DR + 2 * TOK;
  static constexpr int O_S = O_U + 2 * TOK;                // S hi, S lo, D hi, D lo; then the four matrices
  static constexpr int O_F = O_S + BIG;                    // floats
  static constexpr int BYTES = O_F + 1024 * 4;
};

// Float scratch.
enum { kFDo = 0, kFDr = 64, kFU = 128, kFVdr = 192, kFPart = 256 /* [2][3][64] */, kFdG = 640, kFRed = 704 /* [2][8] */,
       kFMax = 720 /* 4 unsigned */, kFCarry = 724 };

template <int DT>
__device__ __forceinline__ float ld1(const void* p, int64_t off) {
  return Fmt<DT>::to_f(static_cast<const typename Fmt<DT>::E*>(p)[off]);
}

template <int DT, int DK>
__global__ void __launch_bounds__(kThreads, 1)
    gdr_bwd_grad_kernel(const GdrArgs a, const GdrGrads gr, const GdrBwdWs w, int nc) {
  pdl_enter();
  using C = Cfg<DT, DK>;
  using F = Fmt<DT>;
  using E = typename F::E;
  constexpr int RB = DK * 2, VRB = kVB * 2;
  constexpr int NT = DK / 16;  // column tiles of 8 of one warp (half of DK)
  extern __shared__ __align__(128) uint8_t sm[];
  float* fs = reinterpret_cast<float*>(sm + C::O_F);
  const float* vecs = reinterpret_cast<const float*>(sm + C::QKB);
  const float* slot = vecs + kVecHead;
  const int* seg = reinterpret_cast<const int*>(slot + kVSeg * kC);
  const uint32_t base = smem_u32(sm);
  const uint32_t kt_hi = base, kt_lo = base + C::TILE, qt_hi = base + C::TERMS * C::TILE, qt_lo = qt_hi + C::TILE;
  const uint32_t do_hi = base + C::O_DO, do_lo = do_hi + C::TOK, dr_hi = base + C::O_DR, dr_lo = dr_hi + C::TOK;
  const uint32_t u_hi = base + C::O_U, u_lo = u_hi + C::TOK;
  const uint32_t s_hi = base + C::O_S, s_lo = s_hi + C::ST, d_hi = s_lo + C::ST, d_lo = d_hi + C::ST;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, qd = lane & 3;
  const int wr = warp & 3, wc = warp >> 2;
  const int i0 = wr * 16 + g, i1 = i0 + 8;
  const int64_t id = blockIdx.x;
  const int64_t c = id % nc, bk_ = id / nc;
  const int64_t hk = bk_ % a.Hk, b = bk_ / a.Hk;
  const int64_t t0 = c * kC;
  const int nt = static_cast<int>(a.L - t0 < kC ? a.L - t0 : kC);
  const int64_t rep = a.Hv / a.Hk;
  const int64_t dvp = (a.Dv + 15) / 16 * 16;

  {  // k and q tiles
    const uint4* src = reinterpret_cast<const uint4*>(w.qk + id * C::QKB);
    uint4* dst = reinterpret_cast<uint4*>(sm);
#pragma unroll 8
    for (int i = tid; i < C::QKB / 16; i += kThreads) dst[i] = src[i];
  }
  float tq[NT][4], tk[NT][4];  // sums over the value heads
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) tq[n][j] = tk[n][j] = 0.f;

  for (int64_t r = 0; r < rep; ++r) {
    const int64_t h = hk * rep + r, bh = b * a.Hv + h, ch = bh * nc + c;
    const float* sw = w.s + ch * DK * dvp;
    const float* dw = w.d + ch * DK * dvp;
    const float* uw = w.u + ch * kC * dvp;
    const float* rw = w.r + ch * kC * dvp;
    const int64_t go = b * gr.dos[0] + t0 * gr.dos[1] + h * gr.dos[2];
    const int64_t vo = b * a.vs[0] + t0 * a.vs[1] + h * a.vs[2];
    __syncthreads();
    reinterpret_cast<uint4*>(sm + C::QKB)[tid] = reinterpret_cast<const uint4*>(w.pack + ch * kPackBytes)[tid];
    if (tid < 4) reinterpret_cast<unsigned*>(fs + kFMax)[tid] = 0;
    // row factors of dO, dR and U over all value channels, and dR.v
    float fdo[8], fdr[8], fu[8];
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
      const int row = warp * 8 + i;
      unsigned mo = 0, mr = 0, mu = 0;
      float vd = 0.f;
      for (int64_t v = lane; v < dvp; v += 32) {
        const float x = rw[row * dvp + v];
        mr = max(mr, mag(x));
        mu = max(mu, mag(uw[row * dvp + v]));
        if (row < nt && v < a.Dv) {
          mo = max(mo, mag(ld1<DT>(gr.dout, go + row * gr.dos[1] + v * gr.dos[3])));
          vd = fmaf(x, ld1<DT>(a.v, vo + row * a.vs[1] + v * a.vs[3]), vd);
        }
      }
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) vd += __shfl_xor_sync(kFullMask, vd, m);
      float io, ir, iu;
      row_factor(warp_max(mo), fdo[i], io);
      row_factor(warp_max(mr), fdr[i], ir);
      row_factor(warp_max(mu), fu[i], iu);
      if (lane == 0) fs[kFDo + row] = io, fs[kFDr + row] = ir, fs[kFU + row] = iu, fs[kFVdr + row] = vd;
    }
    float f_s, i_s, f_d, i_d;
    row_factor(w.s_max[ch], f_s, i_s);
    row_factor(w.d_max[ch], f_d, i_d);

    float dq[NT][4], z[NT][4], dk[NT][4], dp[4][4], dl[4][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) dq[n][j] = z[n][j] = dk[n][j] = 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) dp[n][j] = dl[n][j] = 0.f;
    float sd = 0.f;

    for (int64_t v0 = 0; v0 < dvp; v0 += kVB) {
      __syncthreads();
      // token tiles: a warp's eight rows, two channels a lane
#pragma unroll 4
      for (int i = 0; i < 8; ++i) {
        const int row = warp * 8 + i;
        const int64_t v = v0 + 2 * lane;
        float2 x = make_float2(0.f, 0.f), y = x, o = x;
        if (v < dvp) {
          x = *reinterpret_cast<const float2*>(rw + row * dvp + v);
          y = *reinterpret_cast<const float2*>(uw + row * dvp + v);
        }
        if (row < nt) {
          if (v < a.Dv) o.x = ld1<DT>(gr.dout, go + row * gr.dos[1] + v * gr.dos[3]);
          if (v + 1 < a.Dv) o.y = ld1<DT>(gr.dout, go + row * gr.dos[1] + (v + 1) * gr.dos[3]);
        }
        const uint32_t off = tile_off<VRB>(row, lane >> 2) + (lane & 3) * 4;
        uint32_t hi, lo;
        split2(x.x * fdr[i], x.y * fdr[i], hi, lo);
        *reinterpret_cast<uint32_t*>(sm + C::O_DR + off) = hi;
        *reinterpret_cast<uint32_t*>(sm + C::O_DR + C::TOK + off) = lo;
        split2(y.x * fu[i], y.y * fu[i], hi, lo);
        *reinterpret_cast<uint32_t*>(sm + C::O_U + off) = hi;
        *reinterpret_cast<uint32_t*>(sm + C::O_U + C::TOK + off) = lo;
        split2(o.x * fdo[i], o.y * fdo[i], hi, lo);
        *reinterpret_cast<uint32_t*>(sm + C::O_DO + off) = hi;
        if constexpr (DT == kF32) *reinterpret_cast<uint32_t*>(sm + C::O_DO + C::TOK + off) = lo;
      }
      // S0 and D
#pragma unroll 4
      for (int x = tid; x < DK * (kVB / 4); x += kThreads) {
        const int row = x / (kVB / 4), q4 = x % (kVB / 4);
        const int64_t v = v0 + 4 * q4;
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f), q = p;
        if (v < dvp) {
          p = *reinterpret_cast<const float4*>(sw + row * dvp + v);
          q = *reinterpret_cast<const float4*>(dw + row * dvp + v);
        }
        sd = fmaf(p.x, q.x, fmaf(p.y, q.y, fmaf(p.z, q.z, fmaf(p.w, q.w, sd))));
        const uint32_t off = tile_off<VRB>(row, q4 >> 1) + (q4 & 1) * 8;
        uint2 hi, lo;
        split2(p.x * f_s, p.y * f_s, hi.x, lo.x);
        split2(p.z * f_s, p.w * f_s, hi.y, lo.y);
        *reinterpret_cast<uint2*>(sm + C::O_S + off) = hi;
        *reinterpret_cast<uint2*>(sm + C::O_S + C::ST + off) = lo;
        split2(q.x * f_d, q.y * f_d, hi.x, lo.x);
        split2(q.z * f_d, q.w * f_d, hi.y, lo.y);
        *reinterpret_cast<uint2*>(sm + C::O_S + 2 * C::ST + off) = hi;
        *reinterpret_cast<uint2*>(sm + C::O_S + 3 * C::ST + off) = lo;
      }
      __syncthreads();
#pragma unroll
      for (int kt = 0; kt < kVB / 16; ++kt) {
        uint32_t oh[4], ol[4], rh[4], rl[4], uh[4], ul[4];
        ldsm4(oh, addr_a<VRB>(do_hi, wr * 16, 2 * kt, lane));
        if constexpr (DT == kF32) ldsm4(ol, addr_a<VRB>(do_lo, wr * 16, 2 * kt, lane));
        ldsm4(rh, addr_a<VRB>(dr_hi, wr * 16, 2 * kt, lane));
        ldsm4(rl, addr_a<VRB>(dr_lo, wr * 16, 2 * kt, lane));
        ldsm4(uh, addr_a<VRB>(u_hi, wr * 16, 2 * kt, lane));
        ldsm4(ul, addr_a<VRB>(u_lo, wr * 16, 2 * kt, lane));
#pragma unroll
        for (int np = 0; np < NT / 2; ++np) {
          const int n0 = wc * (DK / 2) + np * 16;
          uint32_t bh_[4], bl_[4];
          ldsm4(bh_, addr_b<VRB>(s_hi, n0, 2 * kt, lane));
          ldsm4(bl_, addr_b<VRB>(s_lo, n0, 2 * kt, lane));
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            mma(dq[2 * np + t], oh, bh_[2 * t], bh_[2 * t + 1]);
            mma(z[2 * np + t], rh, bh_[2 * t], bh_[2 * t + 1]);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            mma(dq[2 * np + t], oh, bl_[2 * t], bl_[2 * t + 1]);
            mma(z[2 * np + t], rh, bl_[2 * t], bl_[2 * t + 1]);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            mma(z[2 * np + t], rl, bh_[2 * t], bh_[2 * t + 1]);
            if constexpr (DT == kF32) mma(dq[2 * np + t], ol, bh_[2 * t], bh_[2 * t + 1]);
          }
          ldsm4(bh_, addr_b<VRB>(d_hi, n0, 2 * kt, lane));
          ldsm4(bl_, addr_b<VRB>(d_lo, n0, 2 * kt, lane));
#pragma unroll
          for (int t = 0; t < 2; ++t) mma(dk[2 * np + t], uh, bh_[2 * t], bh_[2 * t + 1]);
#pragma unroll
          for (int t = 0; t < 2; ++t) mma(dk[2 * np + t], uh, bl_[2 * t], bl_[2 * t + 1]);
#pragma unroll
          for (int t = 0; t < 2; ++t) mma(dk[2 * np + t], ul, bh_[2 * t], bh_[2 * t + 1]);
        }
#pragma unroll
        for (int np = 0; np < 2; ++np) {
          const int n0 = wc * 32 + np * 16;
          if (n0 > wr * 16 + 15) continue;
          uint32_t bh_[4], bl_[4];
          ldsm4(bh_, addr_b<VRB>(u_hi, n0, 2 * kt, lane));
          ldsm4(bl_, addr_b<VRB>(u_lo, n0, 2 * kt, lane));
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            mma(dp[2 * np + t], oh, bh_[2 * t], bh_[2 * t + 1]);
            mma(dl[2 * np + t], rh, bh_[2 * t], bh_[2 * t + 1]);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            mma(dp[2 * np + t], oh, bl_[2 * t], bl_[2 * t + 1]);
            mma(dl[2 * np + t], rh, bl_[2 * t], bl_[2 * t + 1]);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            mma(dl[2 * np + t], rl, bh_[2 * t], bh_[2 * t + 1]);
            if constexpr (DT == kF32) mma(dp[2 * np + t], ol, bh_[2 * t], bh_[2 * t + 1]);
          }
        }
      }
    }

    // true values of the products with the states
    const float be0 = slot[kVBeta * kC + i0], be1 = slot[kVBeta * kC + i1];
    float klast = 0.f;  // sum of k.(gc U D^T) over this thread's elements
    {
      const float gi0 = slot[kVGi * kC + i0], gi1 = slot[kVGi * kC + i1];
      const float gc0 = slot[kVGc * kC + i0], gc1 = slot[kVGc * kC + i1];
      const float q0 = a.scale * gi0 * (fs[kFDo + i0] * i_s), q1 = a.scale * gi1 * (fs[kFDo + i1] * i_s);
      const float z0 = -gi0 * (fs[kFDr + i0] * i_s), z1 = -gi1 * (fs[kFDr + i1] * i_s);
      const float k0 = gc0 * (fs[kFU + i0] * i_d), k1 = gc1 * (fs[kFU + i1] * i_d);
      const float ki0 = slot[kVKInv * kC + i0], ki1 = slot[kVKInv * kC + i1];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // factors of zero (another sequence) select
          dq[n][j] = (j < 2 ? gi0 : gi1) == 0.f ? 0.f : dq[n][j] * (j < 2 ? q0 : q1);
          z[n][j] = (j < 2 ? gi0 : gi1) == 0.f ? 0.f : z[n][j] * (j < 2 ? z0 : z1);
          dk[n][j] = (j < 2 ? gc0 : gc1) == 0.f ? 0.f : dk[n][j] * (j < 2 ? k0 : k1);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int col = wc * (DK / 2) + n * 8 + qd * 2;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = e ? i1 : i0;
          const float ki = e ? ki1 : ki0;
          const uint32_t off = tile_off<RB>(row, col >> 3) + (col & 7) * 2;
          float2 k2 = __half22float2(*reinterpret_cast<const __half2*>(sm + off));
          if constexpr (DT == kF32) {
            const float2 l2 = __half22float2(*reinterpret_cast<const __half2*>(sm + C::TILE + off));
            k2.x += l2.x, k2.y += l2.y;
          }
          klast = fmaf(k2.x * ki, dk[n][2 * e], fmaf(k2.y * ki, dk[n][2 * e + 1], klast));
        }
      }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      klast += __shfl_xor_sync(kFullMask, klast, m);
      sd += __shfl_xor_sync(kFullMask, sd, m);
    }
    if (lane == 0) fs[kFRed + warp] = klast, fs[kFRed + 8 + warp] = sd;

    // A and B with the factors of the products they enter; one power of two a matrix
    unsigned mx[4] = {0, 0, 0, 0};
    {
      const float gh0 = slot[kVGHi * kC + i0], gl0 = slot[kVGLo * kC + i0];
      const float gh1 = slot[kVGHi * kC + i1], gl1 = slot[kVGLo * kC + i1];
      const int s0 = seg[i0], s1 = seg[i1];
      const float po0 = a.scale * fs[kFDo + i0], po1 = a.scale * fs[kFDo + i1];
      const float ro0 = -fs[kFDr + i0], ro1 = -fs[kFDr + i1];
      const float qi0 = slot[kVQInv * kC + i0], qi1 = slot[kVQInv * kC + i1];
      const float bk0 = be0 * slot[kVKInv * kC + i0], bk1 = be1 * slot[kVKInv * kC + i1];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = wc * 32 + n * 8 + qd * 2 + (e & 1);
          const int i = e < 2 ? i0 : i1;
          const bool in = j <= i && seg[j] == (e < 2 ? s0 : s1);
          const float ju = fs[kFU + j];
          const float gam = in ? ex2_approx(((e < 2 ? gh0 : gh1) - slot[kVGHi * kC + j]) +
                                      ((e < 2 ? gl0 : gl1) - slot[kVGLo * kC + j]))
                               : 0.f;
          dp[n][e] = in ? dp[n][e] * ((e < 2 ? po0 : po1) * ju) * gam : 0.f;
          dl[n][e] = in && j < i ? dl[n][e] * ((e < 2 ? ro0 : ro1) * ju) * gam : 0.f;
          const float kj = slot[kVKInv * kC + j];
          mx[0] = max(mx[0], mag(dp[n][e] * kj));
          mx[1] = max(mx[1], mag(dp[n][e] * (e < 2 ? qi0 : qi1)));
          mx[2] = max(mx[2], mag(dl[n][e] * kj));
          mx[3] = max(mx[3], mag(dl[n][e] * (e < 2 ? bk0 : bk1)));
        }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        mx[m] = warp_max(mx[m]);
        if (lane == 0) atomicMax(reinterpret_cast<unsigned*>(fs + kFMax) + m, mx[m]);
      }
      __syncthreads();  // also: every warp is done with S0 and D
      float f[4], inv[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) row_factor(reinterpret_cast<const unsigned*>(fs + kFMax)[m], f[m], inv[m]);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int col = wc * 32 + n * 8 + qd * 2;
        const float kj0 = slot[kVKInv * kC + col], kj1 = slot[kVKInv * kC + col + 1];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t off = tile_off<128>(e ? i1 : i0, col >> 3) + (col & 7) * 2;
          const float qi = e ? qi1 : qi0, bk = e ? bk1 : bk0;
          const float p0 = dp[n][2 * e], p1 = dp[n][2 * e + 1], l0 = dl[n][2 * e], l1 = dl[n][2 * e + 1];
          const float x[4][2] = {{p0 * kj0 * f[0], p1 * kj1 * f[0]},
                                 {p0 * qi * f[1], p1 * qi * f[1]},
                                 {l0 * kj0 * f[2], l1 * kj1 * f[2]},
                                 {l0 * bk * f[3], l1 * bk * f[3]}};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t hi, lo;
            split2(x[m][0], x[m][1], hi, lo);
            *reinterpret_cast<uint32_t*>(sm + C::O_S + 2 * m * kMatBytes + off) = hi;
            *reinterpret_cast<uint32_t*>(sm + C::O_S + (2 * m + 1) * kMatBytes + off) = lo;
          }
        }
      }
      __syncthreads();
      // products over the chunk's tokens
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint32_t mh = s_hi + 2 * m * kMatBytes, ml = mh + kMatBytes;
        const uint32_t bh_t = m == 1 ? qt_hi : kt_hi, bl_t = m == 1 ? qt_lo : kt_lo;
        uint32_t ah[4][4], al[4][4];
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          // rows i, summed j <= i; or rows j, summed i >= j by transposed loads
          const bool use = (m & 1) ? kt >= wr : kt <= wr;
          if (use) {
            if (m & 1) {
              ldsm4t(ah[kt], addr_at<128>(mh, kt * 16, wr * 2, lane));
              ldsm4t(al[kt], addr_at<128>(ml, kt * 16, wr * 2, lane));
            } else {
              ldsm4(ah[kt], addr_a<128>(mh, wr * 16, 2 * kt, lane));
              ldsm4(al[kt], addr_a<128>(ml, wr * 16, 2 * kt, lane));
            }
          } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) ah[kt][x] = al[kt][x] = 0;
          }
        }
#pragma unroll
        for (int np = 0; np < NT / 2; ++np) {
          float x[2][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) x[0][j] = x[1][j] = 0.f;
#pragma unroll
          for (int kt = 0; kt < 4; ++kt) {
            const bool use = (m & 1) ? kt >= wr : kt <= wr;
            if (!use) continue;
            const int piece = (wc * (DK / 2) + np * 16) / 8;
            uint32_t bb[4];
            ldsm4t(bb, addr_bt<RB>(bh_t, kt * 16, piece, lane));
            mma(x[0], ah[kt], bb[0], bb[1]);
            mma(x[1], ah[kt], bb[2], bb[3]);
            mma(x[0], al[kt], bb[0], bb[1]);
            mma(x[1], al[kt], bb[2], bb[3]);
            if constexpr (DT == kF32) {
              ldsm4t(bb, addr_bt<RB>(bl_t, kt * 16, piece, lane));
              mma(x[0], ah[kt], bb[0], bb[1]);
              mma(x[1], ah[kt], bb[2], bb[3]);
            }
          }
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float& dst = m == 0 ? dq[2 * np + t][j] : m == 2 ? z[2 * np + t][j] : dk[2 * np + t][j];
              dst = fmaf(inv[m], x[t][j], dst);
            }
        }
      }
    }

    // dK complete; dot products of each token's rows; sums over the heads
    float dots[3][2] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = wc * (DK / 2) + n * 8 + qd * 2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = e ? i1 : i0;
        const uint32_t off = tile_off<RB>(row, col >> 3) + (col & 7) * 2;
        float2 k2 = __half22float2(*reinterpret_cast<const __half2*>(sm + off));
        float2 q2 = __half22float2(*reinterpret_cast<const __half2*>(sm + C::TERMS * C::TILE + off));
        if constexpr (DT == kF32) {
          const float2 kl = __half22float2(*reinterpret_cast<const __half2*>(sm + C::TILE + off));
          const float2 ql = __half22float2(*reinterpret_cast<const __half2*>(sm + 3 * C::TILE + off));
          k2.x += kl.x, k2.y += kl.y, q2.x += ql.x, q2.y += ql.y;
        }
        const float be = e ? be1 : be0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int j = 2 * e + x;
          const float kv = x ? k2.y : k2.x, qv = x ? q2.y : q2.x;
          dk[n][j] = fmaf(be, z[n][j], dk[n][j]);
          dots[0][e] = fmaf(qv, dq[n][j], dots[0][e]);
          dots[1][e] = fmaf(kv, dk[n][j], dots[1][e]);
          dots[2][e] = fmaf(kv, z[n][j], dots[2][e]);
          tq[n][j] += dq[n][j];
          tk[n][j] += dk[n][j];
        }
      }
    }
#pragma unroll
    for (int d = 0; d < 3; ++d)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = dots[d][e];
        x += __shfl_xor_sync(kFullMask, x, 1);
        x += __shfl_xor_sync(kFullMask, x, 2);
        if (qd == 0) fs[kFPart + (wc * 3 + d) * kC + (e ? i1 : i0)] = x;
      }
    __syncthreads();
    if (tid < kC) {
      const int i = tid;
      const int64_t t = t0 + i;
      const float ki = slot[kVKInv * kC + i], qi = slot[kVQInv * kC + i], be = slot[kVBeta * kC + i];
      const float qdq = qi * (fs[kFPart + i] + fs[kFPart + 3 * kC + i]);
      const float kdk = ki * (fs[kFPart + kC + i] + fs[kFPart + 4 * kC + i]);
      const float kz = ki * (fs[kFPart + 2 * kC + i] + fs[kFPart + 5 * kC + i]);
      if (i < nt)
        static_cast<E*>(gr.dbeta)[b * gr.dbs[0] + t * gr.dbs[1] + h * gr.dbs[2]] = F::from_f(fs[kFVdr + i] + kz);
      float x = qdq - kdk + 2.f * be * kz;
      if (i == kC - 1) {
        float kl = 0.f, sdot = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) kl += fs[kFRed + k], sdot += fs[kFRed + 8 + k];
        const float ga = vecs[kHdGa];
        x += kl + (ga == 0.f ? 0.f : ga * sdot);
      }
      // sum towards the end of the token's sequence: within the warp, then the second warp's first
      const int sg = seg[i];
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const float y = __shfl_down_sync(kFullMask, x, m);
        const int sy = __shfl_down_sync(kFullMask, sg, m);
        if (lane + m < 32 && sy == sg) x += y;
      }
      fs[kFdG + i] = x;
    }
    __syncthreads();
    if (tid < nt) {
      const int i = tid;
      const int64_t t = t0 + i;
      float x = fs[kFdG + i];
      if (i < 32 && seg[32] == seg[i]) x += fs[kFdG + 32];
      // a sequence's first token decays nothing
      const bool first = i > 0 ? seg[i] != seg[i - 1] : seg[0] != 0 || (t == 0 && a.s0 == nullptr);
      gr.dg[b * gr.dgs[0] + t * gr.dgs[1] + h * gr.dgs[2]] = first ? 0.f : x;
    }
  }

  E* qo = static_cast<E*>(gr.dq) + b * gr.dqs[0] + hk * gr.dqs[2];
  E* ko = static_cast<E*>(gr.dk) + b * gr.dks[0] + hk * gr.dks[2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = wc * (DK / 2) + n * 8 + qd * 2 + (j & 1), row = j < 2 ? i0 : i1;
      if (row < nt && col < a.Dk) {
        qo[(t0 + row) * gr.dqs[1] + col * gr.dqs[3]] = F::from_f(tq[n][j]);
        ko[(t0 + row) * gr.dks[1] + col * gr.dks[3]] = F::from_f(tk[n][j]);
      }
    }
}

template <int DT, int DK>
cudaError_t launch(const GdrArgs& a, const GdrGrads& g, const GdrBwdWs& w, int nc, cudaStream_t s) {
  using C = Cfg<DT, DK>;
  static_assert(C::BYTES <= 232448, "shared memory of one block");
  const cudaError_t e =
      cudaFuncSetAttribute(gdr_bwd_grad_kernel<DT, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
  if (e != cudaSuccess) return e;
  return launch_pdl(gdr_bwd_grad_kernel<DT, DK>, static_cast<unsigned>(a.B * a.Hk * nc), kThreads, C::BYTES, s, a, g,
                    w, nc);
}

template <int DT>
cudaError_t launch_dt(const GdrArgs& a, const GdrGrads& g, const GdrBwdWs& w, int nc, cudaStream_t s) {
  return a.Dk <= 64 ? launch<DT, 64>(a, g, w, nc, s) : launch<DT, 128>(a, g, w, nc, s);
}

}  // namespace

cudaError_t launch_gdr_bwd_grad(const GdrArgs& a, const GdrGrads& g, Dtype dt, const GdrBwdWs& w, int nc,
                                cudaStream_t stream) {
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, g, w, nc, stream);
    case kF16: return launch_dt<kF16>(a, g, w, nc, stream);
    case kBF16: return launch_dt<kBF16>(a, g, w, nc, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ccv

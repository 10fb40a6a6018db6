// Gated delta rule, chunked: what a chunk needs that does not depend on the
// state (formulas in gdr_chunk.cuh), for all chunks at once.
//
// A block of four warps takes one chunk of one key head: it scales k and q to
// FP16 tiles, forms k k^T and q k^T with tensor instructions, and for each of
// the key head's value heads the factors, P, and T = (I + L)^-1.
//
// The inverse of the unit lower triangular matrix is made by blocks in FP32:
// the four 16 x 16 diagonal blocks by forward substitution (one warp each,
// a lane holds a column), then twice [A 0; C D]^-1 = [A' 0; -D' C A' D'].
// This is as stable as substitution and has 16 + 4 dependent steps instead of 64.
//
// The results leave as bulk copies of the shared-memory image that the scan
// reads back, already in its tile order.
#include "gdr_chunk.cuh"

namespace ccv {
namespace {

constexpr int kThreads = 128;
constexpr int kLd = 68;  // leading dimension of the FP32 matrices

template <int DT, int DK>
struct PrepSmem {
  static constexpr int TERMS = DT == kF32 ? 2 : 1;
  static constexpr int QK = qk_pack_bytes(DK, TERMS);
  static constexpr int MAT = kC * kLd * 4;
  static constexpr int BYTES = QK + kPackBytes + 2 * MAT + 5 * kC * 4 + 64;
};

// Rows of k or q to FP16 tiles, each row scaled by its power of two.
template <int DT, int DK>
__device__ __forceinline__ void load_rows(const void* base, const int64_t* st, int64_t b, int64_t h, int64_t t0,
                                          int nt, int64_t Dk, uint8_t* hi, uint8_t* lo, float* inv, unsigned& bad,
                                          bool vec) {
  using F = Fmt<DT>;
  using E = typename F::E;
  constexpr int RB = DK * 2;
  constexpr int PER = DK / 32;  // elements of one lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const E* p = static_cast<const E*>(base) + b * st[0] + h * st[2];
#pragma unroll 4
  for (int i = 0; i < kC / 4; ++i) {
    const int r = warp * (kC / 4) + i;
    float x[PER];
    const int c0 = lane * PER;
    const E* row = p + (t0 + r) * st[1];
    if (vec && r < nt) {  // PER elements of a lane in one load
      if constexpr (DT == kF32) {
        if constexpr (PER == 4) {
          const float4 v = *reinterpret_cast<const float4*>(row + c0);
          x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(row + c0);
          x[0] = v.x, x[1] = v.y;
        }
      } else {
        if constexpr (PER == 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(row + c0);
          x[0] = F::word_elem(v.x, 0), x[1] = F::word_elem(v.x, 1), x[2] = F::word_elem(v.y, 0),
          x[3] = F::word_elem(v.y, 1);
        } else {
          const uint32_t v = *reinterpret_cast<const uint32_t*>(row + c0);
          x[0] = F::word_elem(v, 0), x[1] = F::word_elem(v, 1);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        x[j] = (r < nt && c0 + j < Dk) ? F::to_f(row[(c0 + j) * st[3]]) : 0.f;
    }
    unsigned m = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) m = max(m, mag(x[j]));
    m = warp_max(m);
    bad |= m >= kInfBits;
    float f, iv;
    row_factor(m, f, iv);
    if (lane == 0) inv[r] = iv;
    const uint32_t off = tile_off<RB>(r, (c0 * 2) >> 4) + ((c0 * 2) & 15);
#pragma unroll
    for (int j = 0; j < PER; j += 2) {
      if constexpr (DT == kF32) {
        uint32_t a, c;
        split2(x[j] * f, x[j + 1] * f, a, c);
        *reinterpret_cast<uint32_t*>(hi + off + j * 2) = a;
        *reinterpret_cast<uint32_t*>(lo + off + j * 2) = c;
      } else {
        *reinterpret_cast<uint32_t*>(hi + off + j * 2) = h2(x[j] * f, x[j + 1] * f);
      }
    }
  }
}

// X = (I + Ls)^-1, both [64][kLd]; only X[i][j], j <= i, is defined after it.
__device__ __forceinline__ void invert(const float* Ls, float* X) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (lane < 16) {
    const float* Lb = Ls + (warp * 16) * kLd + warp * 16;
    float* Xb = X + (warp * 16) * kLd + warp * 16;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == lane ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) s = fmaf(-Lb[i * kLd + m], x[m], s);
      x[i] = s;
      Xb[i * kLd + lane] = s;
    }
  }
  __syncthreads();
  {  // 16 x 16 blocks (1,0) and (3,2); the scratch is the block above the diagonal
    const int p = warp >> 1, r = (warp & 1) * 8 + (lane >> 2), c = (lane & 3) * 4;
    const int r0 = 32 * p + 16, c0 = 32 * p;
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const float l = Ls[(r0 + r) * kLd + c0 + m];
      const float4 v = *reinterpret_cast<const float4*>(X + (c0 + m) * kLd + c0 + c);
      y[0] = fmaf(l, v.x, y[0]), y[1] = fmaf(l, v.y, y[1]), y[2] = fmaf(l, v.z, y[2]), y[3] = fmaf(l, v.w, y[3]);
    }
    *reinterpret_cast<float4*>(X + (c0 + r) * kLd + r0 + c) = make_float4(y[0], y[1], y[2], y[3]);
    __syncthreads();
    y[0] = y[1] = y[2] = y[3] = 0.f;
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const float l = X[(r0 + r) * kLd + r0 + m];
      const float4 v = *reinterpret_cast<const float4*>(X + (c0 + m) * kLd + r0 + c);
      y[0] = fmaf(-l, v.x, y[0]), y[1] = fmaf(-l, v.y, y[1]), y[2] = fmaf(-l, v.z, y[2]), y[3] = fmaf(-l, v.w, y[3]);
    }
    *reinterpret_cast<float4*>(X + (r0 + r) * kLd + c0 + c) = make_float4(y[0], y[1], y[2], y[3]);
    __syncthreads();
    // the scratch blocks are read as part of X below: they are zero there
    *reinterpret_cast<float4*>(X + (c0 + r) * kLd + r0 + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
  }
  {  // the 32 x 32 block
    const int r = tid >> 2, c = (tid & 3) * 8;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = 0.f;
#pragma unroll 8
    for (int m = 0; m < 32; ++m) {
      const float l = Ls[(32 + r) * kLd + m];
      const float4 v = *reinterpret_cast<const float4*>(X + m * kLd + c);
      const float4 w = *reinterpret_cast<const float4*>(X + m * kLd + c + 4);
      y[0] = fmaf(l, v.x, y[0]), y[1] = fmaf(l, v.y, y[1]), y[2] = fmaf(l, v.z, y[2]), y[3] = fmaf(l, v.w, y[3]);
      y[4] = fmaf(l, w.x, y[4]), y[5] = fmaf(l, w.y, y[5]), y[6] = fmaf(l, w.z, y[6]), y[7] = fmaf(l, w.w, y[7]);
    }
    *reinterpret_cast<float4*>(X + r * kLd + 32 + c) = make_float4(y[0], y[1], y[2], y[3]);
    *reinterpret_cast<float4*>(X + r * kLd + 36 + c) = make_float4(y[4], y[5], y[6], y[7]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = 0.f;
#pragma unroll 8
    for (int m = 0; m < 32; ++m) {
      const float l = X[(32 + r) * kLd + 32 + m];
      const float4 v = *reinterpret_cast<const float4*>(X + m * kLd + 32 + c);
      const float4 w = *reinterpret_cast<const float4*>(X + m * kLd + 36 + c);
      y[0] = fmaf(-l, v.x, y[0]), y[1] = fmaf(-l, v.y, y[1]), y[2] = fmaf(-l, v.z, y[2]), y[3] = fmaf(-l, v.w, y[3]);
      y[4] = fmaf(-l, w.x, y[4]), y[5] = fmaf(-l, w.y, y[5]), y[6] = fmaf(-l, w.z, y[6]), y[7] = fmaf(-l, w.w, y[7]);
    }
    *reinterpret_cast<float4*>(X + (32 + r) * kLd + c) = make_float4(y[0], y[1], y[2], y[3]);
    *reinterpret_cast<float4*>(X + (32 + r) * kLd + c + 4) = make_float4(y[4], y[5], y[6], y[7]);
    __syncthreads();
  }
}

template <int DT, int DK>
__global__ void __launch_bounds__(kThreads) gdr_prep_kernel(const GdrArgs a, uint8_t* qk_ws, uint8_t* pack_ws, int nc,
                                                            bool vec) {
  pdl_enter();
  using S = PrepSmem<DT, DK>;
  using F = Fmt<DT>;
  using E = typename F::E;
  constexpr int RB = DK * 2;
  constexpr int TILE = qk_tile_bytes(DK);
  extern __shared__ __align__(128) uint8_t sm[];
  uint8_t* k_hi = sm;
  uint8_t* k_lo = sm + TILE;  // FP32 inputs only
  uint8_t* q_hi = sm + S::TERMS * TILE;
  uint8_t* q_lo = q_hi + TILE;
  uint8_t* pack = sm + S::QK;
  float* vecs = reinterpret_cast<float*>(pack);
  float* slot = vecs + kVecHead;
  float* Ls = reinterpret_cast<float*>(pack + kPackBytes);
  float* X = Ls + kC * kLd;
  float* kinv = X + kC * kLd;
  float* qinv = kinv + kC;
  float* ghi = qinv + kC;
  float* glo = ghi + kC;
  int* seg = reinterpret_cast<int*>(glo + kC);
  unsigned* flag = reinterpret_cast<unsigned*>(seg + kC);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, qd = lane & 3;
  const int64_t id = blockIdx.x;
  const int64_t c = id % nc, bh = id / nc;
  const int64_t hk = bh % a.Hk, b = bh / a.Hk;
  const int64_t t0 = c * kC;
  const int nt = static_cast<int>(a.L - t0 < kC ? a.L - t0 : kC);
  const int64_t rep = a.Hv / a.Hk;

  unsigned bad_qk = 0;
  load_rows<DT, DK>(a.k, a.ks, b, hk, t0, nt, a.Dk, k_hi, k_lo, kinv, bad_qk, vec);
  load_rows<DT, DK>(a.q, a.qs, b, hk, t0, nt, a.Dk, q_hi, q_lo, qinv, bad_qk, vec);
  if (tid == 0) *flag = 0;
  fence_proxy_async_smem();
  __syncthreads();
  if (bad_qk) atomicOr(flag, 1u);
  if (tid == 0) {
    bulk_store(qk_ws + id * qk_pack_bytes(DK, S::TERMS), sm, qk_pack_bytes(DK, S::TERMS));
    bulk_commit();
  }

  // k k^T and q k^T: warp w makes rows 16w..16w+15, the column tiles up to the diagonal
  float kk[8][4], qq[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[i][j] = qq[i][j] = 0.f;
  const uint32_t kh = smem_u32(k_hi), kl = smem_u32(k_lo), qh = smem_u32(q_hi), ql = smem_u32(q_lo);
#pragma unroll
  for (int kt = 0; kt < DK / 16; ++kt) {
    uint32_t ak[4], aq[4], akl[4], aql[4];
    ldsm4(ak, addr_a<RB>(kh, warp * 16, 2 * kt, lane));
    ldsm4(aq, addr_a<RB>(qh, warp * 16, 2 * kt, lane));
    if constexpr (DT == kF32) {
      ldsm4(akl, addr_a<RB>(kl, warp * 16, 2 * kt, lane));
      ldsm4(aql, addr_a<RB>(ql, warp * 16, 2 * kt, lane));
    }
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      if (np > warp) continue;
      uint32_t bk[4];
      ldsm4(bk, addr_b<RB>(kh, np * 16, 2 * kt, lane));
      mma(kk[2 * np], ak, bk[0], bk[1]);
      mma(kk[2 * np + 1], ak, bk[2], bk[3]);
      mma(qq[2 * np], aq, bk[0], bk[1]);
      mma(qq[2 * np + 1], aq, bk[2], bk[3]);
      if constexpr (DT == kF32) {
        mma(kk[2 * np], akl, bk[0], bk[1]);
        mma(kk[2 * np + 1], akl, bk[2], bk[3]);
        mma(qq[2 * np], aql, bk[0], bk[1]);
        mma(qq[2 * np + 1], aql, bk[2], bk[3]);
        ldsm4(bk, addr_b<RB>(kl, np * 16, 2 * kt, lane));
        mma(kk[2 * np], ak, bk[0], bk[1]);
        mma(kk[2 * np + 1], ak, bk[2], bk[3]);
        mma(qq[2 * np], aq, bk[0], bk[1]);
        mma(qq[2 * np + 1], aq, bk[2], bk[3]);
      }
    }
  }
  const int i0 = warp * 16 + g, i1 = i0 + 8;  // the rows of this thread
  const float ki0 = kinv[i0], ki1 = kinv[i1], qi0 = qinv[i0], qi1 = qinv[i1];

  for (int64_t r = 0; r < rep; ++r) {
    const int64_t h = hk * rep + r;
    // cumulative decay and sequence starts: warp 0, two tokens a lane
    if (warp == 0) {
      float gv[2];
      int nw[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = 2 * lane + j;
        const int64_t t = t0 + i;
        gv[j] = i < nt ? a.g[b * a.gs[0] + t * a.gs[1] + h * a.gs[2]] : 0.f;
        nw[j] = (i < nt && a.seq != nullptr && t > 0 &&
                 a.seq[b * a.ss[0] + t * a.ss[1]] != a.seq[b * a.ss[0] + (t - 1) * a.ss[1]])
                    ? 1
                    : 0;
      }
      // inclusive scan of the pair sums; G is kept as hi + lo so that differences stay exact
      float hi = gv[0] + gv[1];
      float bb = hi - gv[0];
      float lo = (gv[0] - (hi - bb)) + (gv[1] - bb);
      int sn = nw[0] + nw[1];
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const float oh = __shfl_up_sync(kFullMask, hi, m), ol = __shfl_up_sync(kFullMask, lo, m);
        const int os = __shfl_up_sync(kFullMask, sn, m);
        if (lane >= m) {
          const float s = hi + oh, z = s - hi;
          lo += ol + ((hi - (s - z)) + (oh - z));
          hi = s;
          sn += os;
        }
      }
      // token 2 lane: the pair's sum without its second element
      const float s = hi - gv[1], z = s - hi;
      const float e = (hi - (s - z)) + (-gv[1] - z);
      ghi[2 * lane] = s;
      glo[2 * lane] = lo + e;
      ghi[2 * lane + 1] = hi;
      glo[2 * lane + 1] = lo;
      seg[2 * lane] = sn - nw[1];
      seg[2 * lane + 1] = sn;
    }
    if (tid == 0) bulk_wait_read();  // the package buffer is free again
    __syncthreads();

    if (tid < kC) {
      const int i = tid;
      const int64_t t = t0 + i;
      const float be = i < nt ? F::to_f(static_cast<const E*>(a.beta)[b * a.bs[0] + t * a.bs[1] + h * a.bs[2]]) : 0.f;
      const float gh = ghi[i], gl = glo[i];
      const float gi = seg[i] == 0 ? expf(gh + gl) : 0.f;
      const float gc = seg[i] == seg[kC - 1] ? expf((ghi[kC - 1] - gh) + (glo[kC - 1] - gl)) : 0.f;
      slot[kVKS * kC + i] = gi * kinv[i];
      slot[kVQS * kC + i] = a.scale * gi * qinv[i];
      slot[kVBeta * kC + i] = be;
      slot[kVU * kC + i] = gc * kinv[i];
      slot[kVGi * kC + i] = gi;
      slot[kVGc * kC + i] = gc;
      slot[kVKInv * kC + i] = kinv[i];
      slot[kVQInv * kC + i] = qinv[i];
      slot[kVGHi * kC + i] = gh;
      slot[kVGLo * kC + i] = gl;
      reinterpret_cast<int*>(slot)[kVSeg * kC + i] = seg[i];
      if (i == kC - 1) vecs[kHdGa] = gi;
      unsigned nf = (mag(be) >= kInfBits) | (mag(gi) >= kInfBits) | (mag(gc) >= kInfBits);
      // growing decays: the combined factors must be finite too
      nf |= (mag(gi * kinv[i]) >= kInfBits) | (mag(a.scale * gi * qinv[i]) >= kInfBits) |
            (mag(gc * kinv[i]) >= kInfBits);
      if (nf) atomicOr(flag, 2u);
    }
    __syncthreads();

    // Gam, L into shared memory, P split into its tile
    {
      const float gh0 = ghi[i0], gl0 = glo[i0], gh1 = ghi[i1], gl1 = glo[i1];
      const int s0 = seg[i0], s1 = seg[i1];
      const float b0 = slot[kVBeta * kC + i0] * ki0, b1 = slot[kVBeta * kC + i1] * ki1;
      float p[8][4];
      unsigned m0 = 0, m1 = 0;
#pragma unroll
      for (int nt8 = 0; nt8 < 8; ++nt8) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = nt8 * 8 + qd * 2 + e;
          p[nt8][e] = p[nt8][2 + e] = 0.f;
          if (nt8 * 8 <= warp * 16 + 15) {
            const float gj = ghi[j], lj = glo[j], kj = kinv[j];
            const int sj = seg[j];
            const float gam0 = (j <= i0 && sj == s0) ? expf((gh0 - gj) + (gl0 - lj)) : 0.f;
            const float gam1 = (j <= i1 && sj == s1) ? expf((gh1 - gj) + (gl1 - lj)) : 0.f;
            if (j < i0) Ls[i0 * kLd + j] = gam0 == 0.f ? 0.f : b0 * gam0 * kk[nt8][e] * kj;
            if (j < i1) Ls[i1 * kLd + j] = gam1 == 0.f ? 0.f : b1 * gam1 * kk[nt8][2 + e] * kj;
            if (gam0 != 0.f) p[nt8][e] = gam0 * qq[nt8][e] * kj * qi0;
            if (gam1 != 0.f) p[nt8][2 + e] = gam1 * qq[nt8][2 + e] * kj * qi1;
            m0 = max(m0, mag(p[nt8][e]));
            m1 = max(m1, mag(p[nt8][2 + e]));
          }
        }
      }
      m0 = quad_max(m0);
      m1 = quad_max(m1);
      if (m0 >= kInfBits || m1 >= kInfBits) atomicOr(flag, 2u);
      float f0, f1, v0, v1;
      row_factor(m0, f0, v0);
      row_factor(m1, f1, v1);
      if (qd == 0) {
        slot[kVP * kC + i0] = a.scale * v0;
        slot[kVP * kC + i1] = a.scale * v1;
        slot[kVPInv * kC + i0] = v0;
        slot[kVPInv * kC + i1] = v1;
      }
      uint8_t* ph = pack + kVecBytes + 2 * kMatBytes;
      uint8_t* pl = ph + kMatBytes;
#pragma unroll
      for (int nt8 = 0; nt8 < 8; ++nt8) {
        uint32_t hi, lo;
        split2(p[nt8][0] * f0, p[nt8][1] * f0, hi, lo);
        uint32_t off = tile_off<128>(i0, nt8) + qd * 4;
        *reinterpret_cast<uint32_t*>(ph + off) = hi;
        *reinterpret_cast<uint32_t*>(pl + off) = lo;
        split2(p[nt8][2] * f1, p[nt8][3] * f1, hi, lo);
        off = tile_off<128>(i1, nt8) + qd * 4;
        *reinterpret_cast<uint32_t*>(ph + off) = hi;
        *reinterpret_cast<uint32_t*>(pl + off) = lo;
      }
    }
    __syncthreads();
    invert(Ls, X);
    // T's rows scaled and split: a warp takes 16 rows, a lane two columns
    {
      uint8_t* th = pack + kVecBytes;
      uint8_t* tl = th + kMatBytes;
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int row = warp * 16 + i, col = 2 * lane;
        const float2 x = *reinterpret_cast<const float2*>(X + row * kLd + col);
        const float x0 = col <= row ? x.x : 0.f, x1 = col + 1 <= row ? x.y : 0.f;
        const unsigned m = warp_max(max(mag(x0), mag(x1)));
        if (m >= kInfBits && lane == 0) atomicOr(flag, 2u);
        float f, v;
        row_factor(m, f, v);
        if (lane == 0) slot[kVTInv * kC + row] = v;
        uint32_t hi, lo;
        split2(x0 * f, x1 * f, hi, lo);
        const uint32_t off = tile_off<128>(row, lane >> 2) + (lane & 3) * 4;
        *reinterpret_cast<uint32_t*>(th + off) = hi;
        *reinterpret_cast<uint32_t*>(tl + off) = lo;
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      vecs[kHdBad] = *flag ? 1.f : 0.f;
      *flag &= 1u;  // k and q are shared by the next head, its own factors are not
      fence_proxy_async_smem();
      bulk_store(pack_ws + ((b * a.Hv + h) * nc + c) * kPackBytes, pack, kPackBytes);
      bulk_commit();
    }
    __syncthreads();
  }
  if (tid == 0) bulk_wait_all();
}

template <int DT, int DK>
cudaError_t launch(const GdrArgs& a, uint8_t* qk_ws, uint8_t* pack_ws, int nc, cudaStream_t s) {
  using E = typename Fmt<DT>::E;
  constexpr int64_t PER = DK / 32;
  auto ok = [&](const void* p, const int64_t* st) {
    return st[3] == 1 && a.Dk == DK && reinterpret_cast<uintptr_t>(p) % (PER * sizeof(E)) == 0 && st[0] % PER == 0 &&
           st[1] % PER == 0 && st[2] % PER == 0;
  };
  const bool vec = ok(a.k, a.ks) && ok(a.q, a.qs);
  constexpr int smem = PrepSmem<DT, DK>::BYTES;
  const cudaError_t e =
      cudaFuncSetAttribute(gdr_prep_kernel<DT, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(gdr_prep_kernel<DT, DK>, static_cast<unsigned>(a.B * a.Hk * nc), kThreads, smem, s, a, qk_ws,
                    pack_ws, nc, vec);
}

template <int DT>
cudaError_t launch_dt(const GdrArgs& a, uint8_t* q, uint8_t* p, int nc, cudaStream_t s) {
  return a.Dk <= 64 ? launch<DT, 64>(a, q, p, nc, s) : launch<DT, 128>(a, q, p, nc, s);
}

}  // namespace

cudaError_t launch_gdr_prep(const GdrArgs& a, Dtype dt, uint8_t* qk_ws, uint8_t* pack_ws, int nc, cudaStream_t s) {
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, qk_ws, pack_ws, nc, s);
    case kF16: return launch_dt<kF16>(a, qk_ws, pack_ws, nc, s);
    case kBF16: return launch_dt<kBF16>(a, qk_ws, pack_ws, nc, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ccv

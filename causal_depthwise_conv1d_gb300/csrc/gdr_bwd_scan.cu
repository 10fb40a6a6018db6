// Gated delta rule, backward: the reverse scan over the chunks.
//
// With D the gradient of the state after a chunk (the given gradient of the
// final state, or zero, after the last), dO scaled by `scale`, X = beta gi dR:
//
//   dU = P^T dO + gc (K D),   dR = T^T dU,   dV = beta dR,
//   D <- ga D + Q^T (gi dO) - K^T X          (the gradient of the state before it)
//
// Laid out as the forward scan (gdr_scan.cu): a warp owns 16 value channels,
// everything is transposed, D^T stays in registers.  D before each step, dR
// and dO go to the workspace, as tiles that the gradients' matrix loads can
// take (gdr_chunk.cuh), with the products dR.v of this warp's channels.
//
// A chunk with a value that is not finite is taken token by token, as there.
//
// P^T and T^T are the tiles of the forward pass read by transposed matrix
// loads; the row factors of those tiles run along the summed index here and
// are multiplied into dO and dU.
//
// What bounds it: as in the forward scan, the chain of a chunk (3250 warp
// instructions a warp and chunk; tensor pipe 28 %, issue slots 23 % busy with
// four warps an SM, and the loop's code is larger than the instruction cache).
// 2 x 2048 tokens x 32 heads of 128 x 128, bf16: 231 us, 32 chunks of 7.2 us.
// Packed arithmetic between the products, which helps the forward scan,
// measured 250 us here, and the update of D as a rolled loop 239 us.
#include "gdr_chunk.cuh"

namespace ccv {
namespace {

__device__ unsigned g_fault;

// NW groups of 16 value channels a block, H warps each (as in the forward scan).
template <int DT, int DK, int NW, int H>
struct Cfg {
  static constexpr int TERMS = DT == kF32 ? 2 : 1;
  static constexpr int TILE = qk_tile_bytes(DK);
  static constexpr int QKB = qk_pack_bytes(DK, TERMS);
  static constexpr int STAGE = QKB + kPackBytes;
  static constexpr int ROW = DT == kF32 ? 64 : 32;
  static constexpr int GBYTES = kC * ROW;                     // dO of one warp
  static constexpr int OBYTES = DT == kF32 ? 0 : kC * 32;     // dV of one warp
  static constexpr int WARPS = NW * H;
  static constexpr int XBYTES = H == 2 ? 4096 : 0;            // a warp's share of K D for the other
  static constexpr int DIMG = 2 * img_state_bytes(DK) / H;    // this warp's part of D hi and D lo
  static constexpr int RIMG = 2 * kTokBytes;                  // dR hi and lo
  static constexpr int OIMG = TERMS * kTokBytes;              // dO
  static constexpr int PER_WARP = 2 * GBYTES + OBYTES + XBYTES + DIMG + RIMG + OIMG;
  // FP32 tiles leave room for one stage only
  static constexpr int STAGES = 2 * STAGE + WARPS * PER_WARP + 64 <= 232448 ? 2 : 1;
  static constexpr int BYTES = STAGES * STAGE + WARPS * PER_WARP + 64;
};

template <int DT>
__device__ __forceinline__ void fetch(const void* base, const int64_t* st, int64_t L, int64_t Dv, int64_t b, int64_t h,
                                      int64_t t0, int64_t v0, bool vec, uint8_t* buf, int lane) {
  using F = Fmt<DT>;
  using E = typename F::E;
  constexpr int ROW = DT == kF32 ? 64 : 32;
  constexpr int PIECES = ROW / 16;
  const E* p = static_cast<const E*>(base) + b * st[0] + h * st[2] + v0 * st[3];
  if (vec) {
#pragma unroll
    for (int i = 0; i < kC * PIECES / 32; ++i) {
      const int x = i * 32 + lane, r = x / PIECES, pc = x % PIECES;
      const bool in = t0 + r < L;
      cp_async16(buf + r * ROW + pc * 16, p + (in ? (t0 + r) * st[1] : 0) + pc * (16 / static_cast<int>(sizeof(E))), in);
    }
  } else {
    for (int x = lane; x < kC * 16; x += 32) {
      const int r = x >> 4, c = x & 15;
      E e = F::from_f(0.f);
      if (t0 + r < L && v0 + c < Dv) e = p[(t0 + r) * st[1] + c * st[3]];
      *reinterpret_cast<E*>(buf + r * ROW + c * sizeof(E)) = e;
    }
  }
  cp_async_commit();
}

// One chunk token by token, last token first, from the original inputs: the
// definition's own backward step on the warp's 16 rows of D^T.
//   D += q (scale dO)^T;   dR = D^T k;   dV = beta dR;   D <- a (D - k dV^T)
template <int DT, int NK, int H>
__device__ __noinline__ void token_by_token(const GdrArgs& a, const GdrGrads& gr, float (&d)[NK][4], int64_t b,
                                            int64_t h, int64_t t0, int64_t v0, float (&u)[8][4], int lane, int half,
                                            int pair, float* xb, const float* xo) {
  const int k0 = half * NK * 8;
  using F = Fmt<DT>;
  using E = typename F::E;
  const int g = lane >> 2, qd = lane & 3;
  const int64_t hk = h / (a.Hv / a.Hk);
  const E* kp = static_cast<const E*>(a.k) + b * a.ks[0] + hk * a.ks[2];
  const E* qp = static_cast<const E*>(a.q) + b * a.qs[0] + hk * a.qs[2];
  const int64_t r0 = v0 + g, r1 = v0 + g + 8;
  for (int i = kC - 1; i >= 0; --i) {
    const int64_t t = t0 + i;
    if (((i >> 1) & 3) == qd) u[i >> 3][i & 1] = u[i >> 3][2 + (i & 1)] = 0.f;
    if (t >= a.L) continue;
    const float dec = expf(a.g[b * a.gs[0] + t * a.gs[1] + h * a.gs[2]]);
    const float be = F::to_f(static_cast<const E*>(a.beta)[b * a.bs[0] + t * a.bs[1] + h * a.bs[2]]);
    const bool first =
        a.seq != nullptr && t > 0 && a.seq[b * a.ss[0] + t * a.ss[1]] != a.seq[b * a.ss[0] + (t - 1) * a.ss[1]];
    const E* op = static_cast<const E*>(gr.dout) + b * gr.dos[0] + t * gr.dos[1] + h * gr.dos[2];
    const float o0 = r0 < a.Dv ? a.scale * F::to_f(op[r0 * gr.dos[3]]) : 0.f;
    const float o1 = r1 < a.Dv ? a.scale * F::to_f(op[r1 * gr.dos[3]]) : 0.f;
    float p0 = 0.f, p1 = 0.f;
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t kd = k0 + 8 * n + 2 * qd + e;
        if (kd < a.Dk) {
          const float kv = F::to_f(kp[t * a.ks[1] + kd * a.ks[3]]), qv = F::to_f(qp[t * a.qs[1] + kd * a.qs[3]]);
          d[n][e] = fmaf(qv, o0, d[n][e]);
          d[n][2 + e] = fmaf(qv, o1, d[n][2 + e]);
          p0 = fmaf(kv, d[n][e], p0);
          p1 = fmaf(kv, d[n][2 + e], p1);
        }
      }
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
      p0 += __shfl_xor_sync(kFullMask, p0, m);
      p1 += __shfl_xor_sync(kFullMask, p1, m);
    }
    if constexpr (H == 2) {
      xb[lane] = p0;
      xb[32 + lane] = p1;
      pair_sync(pair);
      p0 += xo[lane], p1 += xo[32 + lane];
      pair_sync(pair);
    }
    const float w0 = be * p0, w1 = be * p1;
    if (((i >> 1) & 3) == qd) u[i >> 3][i & 1] = p0, u[i >> 3][2 + (i & 1)] = p1;
    if (qd == 0 && half == 0) {
      E* vp = static_cast<E*>(gr.dv) + b * gr.dvs[0] + t * gr.dvs[1] + h * gr.dvs[2];
      if (r0 < a.Dv) vp[r0 * gr.dvs[3]] = F::from_f(w0);
      if (r1 < a.Dv) vp[r1 * gr.dvs[3]] = F::from_f(w1);
    }
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t kd = k0 + 8 * n + 2 * qd + e;
        if (first) {
          d[n][e] = d[n][2 + e] = 0.f;
        } else if (kd < a.Dk) {
          const float kv = F::to_f(kp[t * a.ks[1] + kd * a.ks[3]]);
          d[n][e] = dec * fmaf(-kv, w0, d[n][e]);
          d[n][2 + e] = dec * fmaf(-kv, w1, d[n][2 + e]);
        }
      }
  }
}

template <int DT, int DK, int NW, int H>
__global__ void __launch_bounds__(32 * NW * H, 1)
    gdr_bwd_scan_kernel(const GdrArgs a, const GdrGrads gr, const GdrBwdWs w, int nc, int64_t head0, unsigned vtiles,
                        bool gvec, bool vvec, bool ovec) {
  pdl_enter();
  using C = Cfg<DT, DK, NW, H>;
  using F = Fmt<DT>;
  using E = typename F::E;
  constexpr int RB = DK * 2;
  constexpr int NK = DK / 8 / H;
  constexpr int NS = C::STAGES;
  extern __shared__ __align__(128) uint8_t sm[];
  uint8_t* gbuf0 = sm + NS * C::STAGE;
  uint8_t* obuf0 = gbuf0 + 2 * C::WARPS * C::GBYTES;  // dO, then v
  uint8_t* xbuf0 = obuf0 + C::WARPS * C::OBYTES;
  uint8_t* ibuf0 = xbuf0 + C::WARPS * C::XBYTES;
  constexpr int IMG = C::DIMG + C::RIMG + C::OIMG;
  uint64_t* full = reinterpret_cast<uint64_t*>(ibuf0 + C::WARPS * IMG);
  unsigned* left = reinterpret_cast<unsigned*>(full + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, qd = lane & 3;
  // indices below 2^31 (checked on the host): 32-bit divisions
  const unsigned Hv = static_cast<unsigned>(a.Hv), ubh = static_cast<unsigned>(head0) + blockIdx.x / vtiles;
  const unsigned ub = ubh / Hv, uh = ubh - ub * Hv;
  const int64_t bh = ubh, b = ub, h = uh, hk = uh / (Hv / static_cast<unsigned>(a.Hk));
  const int grp = warp / H, half = warp % H;
  const int64_t v0 = (static_cast<int64_t>(blockIdx.x % vtiles) * NW + grp) * 16;
  const int k0 = half * NK * 8;  // first key channel of this warp
  const int pair = grp + 1;      // its barrier
  float* xb = reinterpret_cast<float*>(xbuf0 + warp * C::XBYTES);
  const float* xo = reinterpret_cast<const float*>(xbuf0 + (warp ^ 1) * C::XBYTES);
  const uint8_t* qk = w.qk + (b * a.Hk + hk) * nc * qk_pack_bytes(DK, C::TERMS);
  const uint8_t* pkg = w.pack + bh * nc * kPackBytes;
  // step n takes chunk nc - 1 - n
  auto fill = [&](int n) {
    const int c = nc - 1 - n;
    uint8_t* dst = sm + (n % NS) * C::STAGE;
    uint64_t* bar = &full[n % NS];
    mbar_arrive_expect_tx(bar, C::STAGE);
    bulk_load(dst, qk + static_cast<int64_t>(c) * C::QKB, C::QKB, bar);
    bulk_load(dst + C::QKB, pkg + static_cast<int64_t>(c) * kPackBytes, kPackBytes, bar);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      left[s] = 0;
    }
    fence_barrier_init();
    for (int n = 0; n < NS && n < nc; ++n) fill(n);
  }
  __syncthreads();

  const bool active = v0 < a.Dv;
  uint8_t* gb = gbuf0 + warp * C::GBYTES;
  uint8_t* vb = gb + C::WARPS * C::GBYTES;
  uint8_t* ob = obuf0 + warp * C::OBYTES;
  uint8_t* ibuf = ibuf0 + warp * IMG;
  const uint32_t dimg = smem_u32(ibuf), rimg = dimg + C::DIMG, oimg = rimg + C::RIMG;
  const int ns = static_cast<int>((a.Dv + 15) / 16);
  const bool wgvec = gvec && v0 + 16 <= a.Dv, wvvec = vvec && v0 + 16 <= a.Dv, wovec = ovec && v0 + 16 <= a.Dv;

  float d[NK][4];
#pragma unroll
  for (int n = 0; n < NK; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t kd = k0 + 8 * n + 2 * qd + (j & 1), vc = v0 + g + (j >> 1) * 8;
      d[n][j] = (gr.ds1 != nullptr && kd < a.Dk && vc < a.Dv)
                    ? gr.ds1[b * gr.ds1s[0] + h * gr.ds1s[1] + kd * gr.ds1s[2] + vc * gr.ds1s[3]]
                    : 0.f;
    }
  auto fetch2 = [&](int64_t t0) {
    fetch<DT>(gr.dout, gr.dos, a.L, a.Dv, b, h, t0, v0, wgvec, gb, lane);
    fetch<DT>(a.v, a.vs, a.L, a.Dv, b, h, t0, v0, wvvec, vb, lane);
  };
  if (active && nc > 0)
    fetch2(static_cast<int64_t>(nc - 1) * kC);

  for (int n0 = 0; n0 < nc; ++n0) {
    const int s = n0 % NS, c = nc - 1 - n0;
    const int64_t t0 = static_cast<int64_t>(c) * kC;
    bool late = !mbar_wait(&full[s], (n0 / NS) & 1);
    if constexpr (H == 2) late = pair_any(pair, late);  // a pair gives up together
    if (late) {  // give up: no copy of this warp's, nor the other stage's, must outlive the block
      cp_async_wait_all();
      if (lane == 0) {
        atomicOr(&g_fault, kFaultConsumerWait);
        if (NS == 2 && n0 + 1 < nc && !mbar_wait(&full[s ^ 1], ((n0 + 1) / NS) & 1))
          atomicOr(&g_fault, kFaultDrainWait);
        bulk_wait_all();
      }
      return;
    }
    if (active) {
      const uint32_t kt_hi = smem_u32(sm + s * C::STAGE);
      const uint32_t kt_lo = kt_hi + C::TILE;
      const uint32_t qt_hi = kt_hi + C::TERMS * C::TILE;
      const uint32_t qt_lo = qt_hi + C::TILE;
      const float* vecs = reinterpret_cast<const float*>(sm + s * C::STAGE + C::QKB);
      const float* slot = vecs + kVecHead;
      const uint32_t th = kt_hi + C::QKB + kVecBytes, tl = th + kMatBytes;
      const uint32_t ph = kt_hi + C::QKB + kOffP, pl = ph + kMatBytes;
      const float ga = vecs[kHdGa];

      float a0 = 0.f, a1 = 0.f;
      uint8_t* gimg = w.img_b + ((bh * nc + c) * ns + v0 / 16) * ImgB::bytes(DK, C::TERMS);
      float* ginv = reinterpret_cast<float*>(gimg + ImgB::inv(DK, C::TERMS));
      if (lane == 0) bulk_wait_read();
      __syncwarp();
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        a0 = amax3(a0, d[n][0], d[n][1]);
        a1 = amax3(a1, d[n][2], d[n][3]);
      }
      const unsigned m0 = quad_max(__float_as_uint(a0)), m1 = quad_max(__float_as_uint(a1));
      bool bad = vecs[kHdBad] != 0.f || m0 >= kInfBits || m1 >= kInfBits;
      float f0, f1, di0, di1;
      row_factor(m0, f0, di0);
      row_factor(m1, f1, di1);
      const uint64_t p0 = pk(f0, f0), p1 = pk(f1, f1);

      // (K D)^T
      float u[8][4];
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) u[n][j] = 0.f;
#pragma unroll
      for (int kt = 0; kt < NK / 2; ++kt) {
        const int piece = k0 / 8 + 2 * kt;
        uint32_t hi[4], lo[4];
        split2f(d[2 * kt][0], d[2 * kt][1], p0, hi[0], lo[0]);
        split2f(d[2 * kt][2], d[2 * kt][3], p1, hi[1], lo[1]);
        split2f(d[2 * kt + 1][0], d[2 * kt + 1][1], p0, hi[2], lo[2]);
        split2f(d[2 * kt + 1][2], d[2 * kt + 1][3], p1, hi[3], lo[3]);
        {
          const uint32_t at = dimg + (kt >> 1) * kBlkBytes +
                              off64((lane & 7) + ((lane >> 3) & 1) * 8, (kt & 1) * 2 + (lane >> 4));
          stsm4(at, hi);
          stsm4(at + C::DIMG / 2, lo);
        }
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t bk[4];
          ldsm4(bk, addr_b<RB>(kt_hi, np * 16, piece, lane));
          mma(u[2 * np], hi, bk[0], bk[1]);
          mma(u[2 * np + 1], hi, bk[2], bk[3]);
          mma(u[2 * np], lo, bk[0], bk[1]);
          mma(u[2 * np + 1], lo, bk[2], bk[3]);
          if constexpr (DT == kF32) {
            ldsm4(bk, addr_b<RB>(kt_lo, np * 16, piece, lane));
            mma(u[2 * np], hi, bk[0], bk[1]);
            mma(u[2 * np + 1], hi, bk[2], bk[3]);
          }
        }
      }

      auto save_d = [&](float i0, float i1) {  // D's tiles are in the staging memory
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          bulk_store(gimg + half * (C::DIMG / 2), ibuf, C::DIMG / 2);
          bulk_store(gimg + img_state_bytes(DK) + half * (C::DIMG / 2), ibuf + C::DIMG / 2, C::DIMG / 2);
          bulk_commit();
        }
        if (qd == 0) {
#pragma unroll
          for (int y = 0; y < 2 / H; ++y) ginv[(half + y) * 16 + g] = i0, ginv[(half + y) * 16 + g + 8] = i1;
        }
      };
      save_d(di0, di1);

      // true values, and the other half's share
#pragma unroll
      for (int n = 0; n < 8; ++n) u[n][0] *= di0, u[n][1] *= di0, u[n][2] *= di1, u[n][3] *= di1;
      if constexpr (H == 2) {
        float4* x4 = reinterpret_cast<float4*>(xb);
        const float4* o4 = reinterpret_cast<const float4*>(xo);
#pragma unroll
        for (int n = 0; n < 8; ++n) x4[n * 32 + lane] = make_float4(u[n][0], u[n][1], u[n][2], u[n][3]);
        pair_sync(pair);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float4 o = o4[n * 32 + lane];
          u[n][0] += o.x, u[n][1] += o.y, u[n][2] += o.z, u[n][3] += o.w;
        }
      }

      // dO, read once; its two scaled forms follow from it
      float x[8][4];
      cp_async_wait_all();
      __syncwarp();
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        if constexpr (DT == kF32) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[2 * np + t][j] = *reinterpret_cast<const float*>(gb + (np * 16 + t * 8 + qd * 2 + (j & 1)) * C::ROW +
                                                                 (g + (j >> 1) * 8) * 4);
        } else {
          uint32_t r[4];
          ldsm4t(r, smem_u32(gb) + (np * 16 + (lane & 7) + ((lane >> 4) & 1) * 8) * C::ROW + ((lane >> 3) & 1) * 16);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[2 * np + t][j] = F::word_elem(r[2 * t + (j >> 1)], j & 1);
        }
      }
      float xv[8][4];  // v, for dR.v
      if (half == 0) {
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          if constexpr (DT == kF32) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                xv[2 * np + t][j] = *reinterpret_cast<const float*>(vb + (np * 16 + t * 8 + qd * 2 + (j & 1)) * C::ROW +
                                                                    (g + (j >> 1) * 8) * 4);
          } else {
            uint32_t r[4];
            ldsm4t(r, smem_u32(vb) + (np * 16 + (lane & 7) + ((lane >> 4) & 1) * 8) * C::ROW + ((lane >> 3) & 1) * 16);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int j = 0; j < 4; ++j) xv[2 * np + t][j] = F::word_elem(r[2 * t + (j >> 1)], j & 1);
          }
        }
      }
      __syncwarp();
      if (n0 + 1 < nc) fetch2(t0 - kC);

      uint32_t hi[4][4], lo[4][4];
      bool ignore = false;
      // a [64 tokens][16 v] tile from fragments of rows v
      auto put_tok = [&](uint32_t tile, const uint32_t (&r)[4][4]) {
#pragma unroll
        for (int np = 0; np < 4; ++np)
          stsm4t(tile + off32(np * 16 + (lane & 7) + ((lane >> 4) & 1) * 8, (lane >> 3) & 1), r[np]);
      };
      auto put_o = [&](auto kept) {  // dO's image
        if (half != 0) return;
        float i0, i1;
        split_rows<8, DT == kF32, kept.value>(x, hi, lo, i0, i1, ignore);
        put_tok(oimg, hi);
        if constexpr (DT == kF32) put_tok(oimg + kTokBytes, lo);
        if (qd == 0) ginv[48 + g] = i0, ginv[48 + g + 8] = i1;
      };
      put_o(std::false_type{});
      // after dR: its image and dR.v of this warp's channels, and all parts out;
      // `kept`: a chunk with values that are not finite
      auto save_r = [&](const float (&r)[8][4], auto kept) {
        if (half != 0) return;
        uint32_t rh[4][4], rl[4][4];
        float i0, i1;
        bool lost = false;
        split_rows<8, true, kept.value>(r, rh, rl, i0, i1, lost);
        if (!kept.value && lost) i0 = i1 = __uint_as_float(kLostBits);
        put_tok(rimg, rh);
        put_tok(rimg + kTokBytes, rl);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          bulk_store(gimg + ImgB::r(DK), ibuf + C::DIMG, C::RIMG + C::OIMG);
          bulk_commit();
        }
        if (qd == 0) ginv[32 + g] = i0, ginv[32 + g + 8] = i1;
        // sums over the 16 rows: two here, eight lanes by a halving exchange;
        // a lane ends with tokens 2 lane and 2 lane + 1
        float y[16];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) y[2 * n + e] = fmaf(r[n][e], xv[n][e], r[n][2 + e] * xv[n][2 + e]);
#pragma unroll
        for (int m = 8; m >= 2; m >>= 1)
#pragma unroll
          for (int j = 0; j < m; ++j) {
            const bool up = (lane & (2 * m)) != 0;
            const float mine = up ? y[m + j] : y[j], other = up ? y[j] : y[m + j];
            y[j] = mine + __shfl_xor_sync(kFullMask, other, 2 * m);
          }
        *reinterpret_cast<float2*>(ginv + 64 + 2 * lane) = make_float2(y[0], y[1]);
      };
      {  // dU^T = dO^T P + gc (K D)^T: 16-bit dO times powers of two is exact in hi
        float y[8][4], yi0, yi1;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float2 pi = *reinterpret_cast<const float2*>(slot + kVPInv * kC + n * 8 + qd * 2);
          y[n][0] = x[n][0] * pi.x, y[n][1] = x[n][1] * pi.y, y[n][2] = x[n][2] * pi.x, y[n][3] = x[n][3] * pi.y;
        }
        split_rows<8, DT == kF32>(y, hi, lo, yi0, yi1, bad);
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          float z[2][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) z[0][j] = z[1][j] = 0.f;
#pragma unroll
          for (int kt = np; kt < 4; ++kt) {
            uint32_t bp[4];
            ldsm4t(bp, addr_bt<128>(ph, kt * 16, 2 * np, lane));
            mma(z[0], hi[kt], bp[0], bp[1]);
            mma(z[1], hi[kt], bp[2], bp[3]);
            if constexpr (DT == kF32) {
              mma(z[0], lo[kt], bp[0], bp[1]);
              mma(z[1], lo[kt], bp[2], bp[3]);
            }
            ldsm4t(bp, addr_bt<128>(pl, kt * 16, 2 * np, lane));
            mma(z[0], hi[kt], bp[0], bp[1]);
            mma(z[1], hi[kt], bp[2], bp[3]);
          }
          const float s0 = a.scale * yi0, s1 = a.scale * yi1;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int n = 2 * np + t;
            const float2 cu = *reinterpret_cast<const float2*>(slot + kVU * kC + n * 8 + qd * 2);
            const float2 ti = *reinterpret_cast<const float2*>(slot + kVTInv * kC + n * 8 + qd * 2);
            // a factor of zero (another sequence) selects: a state with infinities must not leak
            const float k0 = cu.x == 0.f ? 0.f : cu.x * u[n][0], k1 = cu.y == 0.f ? 0.f : cu.y * u[n][1];
            const float k2 = cu.x == 0.f ? 0.f : cu.x * u[n][2], k3 = cu.y == 0.f ? 0.f : cu.y * u[n][3];
            u[n][0] = ti.x * fmaf(s0, z[t][0], k0);
            u[n][1] = ti.y * fmaf(s0, z[t][1], k1);
            u[n][2] = ti.x * fmaf(s1, z[t][2], k2);
            u[n][3] = ti.y * fmaf(s1, z[t][3], k3);
          }
        }
      }
      // dR^T = dU^T T (the factors of T's rows are in dU now)
      float ui0, ui1;
      split_rows<8, true>(u, hi, lo, ui0, ui1, bad);
      // (with two warps: also the barrier after which the exchange buffers may be written again)
      bad = H == 2 ? pair_any(pair, bad) : __any_sync(kFullMask, bad) != 0;
      if (bad) {
        float tmp[NK][4];  // a copy: D itself has to stay in registers
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) tmp[n][j] = d[n][j];
        {  // D's and dO's images again
          if (lane == 0) bulk_wait_all();
          __syncwarp();
          float i0, i1;
          keep_state(tmp, dimg, C::DIMG / 2, lane, i0, i1);
          save_d(i0, i1);
          put_o(std::true_type{});
        }
        float ut[8][4];
        token_by_token<DT, NK, H>(a, gr, tmp, b, h, t0, v0, ut, lane, half, pair, xb, xo);
        save_r(ut, std::true_type{});
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) d[n][j] = tmp[n][j];
      } else {
      {
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          float z[2][2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) z[0][i][j] = z[1][i][j] = 0.f;
#pragma unroll
          for (int kt = np; kt < 4; ++kt) {
            uint32_t bt[4];
            ldsm4t(bt, addr_bt<128>(th, kt * 16, 2 * np, lane));
            mma(z[0][0], hi[kt], bt[0], bt[1]);
            mma(z[0][1], hi[kt], bt[2], bt[3]);
            mma(z[1][0], lo[kt], bt[0], bt[1]);
            mma(z[1][1], lo[kt], bt[2], bt[3]);
            ldsm4t(bt, addr_bt<128>(tl, kt * 16, 2 * np, lane));
            mma(z[1][0], hi[kt], bt[0], bt[1]);
            mma(z[1][1], hi[kt], bt[2], bt[3]);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            u[2 * np + t][0] = (z[0][t][0] + z[1][t][0]) * ui0;
            u[2 * np + t][1] = (z[0][t][1] + z[1][t][1]) * ui0;
            u[2 * np + t][2] = (z[0][t][2] + z[1][t][2]) * ui1;
            u[2 * np + t][3] = (z[0][t][3] + z[1][t][3]) * ui1;
          }
        }
      }
      save_r(u, std::false_type{});
      // dV out
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        float y[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int n = 2 * np + t;
          const float2 be = *reinterpret_cast<const float2*>(slot + kVBeta * kC + n * 8 + qd * 2);
          y[t][0] = u[n][0] * be.x, y[t][1] = u[n][1] * be.y, y[t][2] = u[n][2] * be.x, y[t][3] = u[n][3] * be.y;
        }
        if (H == 2 && (np >> 1) != half) continue;  // the other warp's tokens
        if (DT != kF32 && wovec) {
          if constexpr (DT != kF32) {
            const uint32_t r[4] = {F::pack2(y[0][0], y[0][1]), F::pack2(y[0][2], y[0][3]), F::pack2(y[1][0], y[1][1]),
                                   F::pack2(y[1][2], y[1][3])};
            stsm4t(smem_u32(ob) + (np * 16 + (lane & 7) + ((lane >> 4) & 1) * 8) * 32 + ((lane >> 3) & 1) * 16, r);
          }
        } else {
          E* op = static_cast<E*>(gr.dv) + b * gr.dvs[0] + h * gr.dvs[2];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int64_t tok = t0 + np * 16 + t * 8 + qd * 2 + (j & 1), vc = v0 + g + (j >> 1) * 8;
              if (tok < a.L && vc < a.Dv) op[tok * gr.dvs[1] + vc * gr.dvs[3]] = F::from_f(y[t][j]);
            }
        }
      }
      if (DT != kF32 && wovec) {
        __syncwarp();
        E* op = static_cast<E*>(gr.dv) + b * gr.dvs[0] + h * gr.dvs[2] + v0;
#pragma unroll
        for (int i = 0; i < 4 / H; ++i) {
          const int y = (half * 2 + i) * 32 + lane, r = y >> 1, pc = y & 1;
          const uint4 v = lds128(ob + r * 32 + pc * 16);
          if (t0 + r < a.L) *reinterpret_cast<uint4*>(op + (t0 + r) * gr.dvs[1] + pc * 8) = v;
        }
        __syncwarp();
      }

      // D <- ga D + Q^T (gi scale dO) - K^T (beta gi dR), one product after the other
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        float y[8][4], yi0, yi1;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          if (part == 0) {
            const float2 cq = *reinterpret_cast<const float2*>(slot + kVQS * kC + n * 8 + qd * 2);
            y[n][0] = x[n][0] * cq.x, y[n][1] = x[n][1] * cq.y, y[n][2] = x[n][2] * cq.x, y[n][3] = x[n][3] * cq.y;
          } else {
            const float2 ck = *reinterpret_cast<const float2*>(slot + kVKS * kC + n * 8 + qd * 2);
            const float2 be = *reinterpret_cast<const float2*>(slot + kVBeta * kC + n * 8 + qd * 2);
            const float fx = -be.x * ck.x, fy = -be.y * ck.y;
            y[n][0] = u[n][0] * fx, y[n][1] = u[n][1] * fy, y[n][2] = u[n][2] * fx, y[n][3] = u[n][3] * fy;
          }
        }
        split_rows<8, true>(y, hi, lo, yi0, yi1, ignore);
        const uint32_t th_ = part == 0 ? qt_hi : kt_hi, tl_ = part == 0 ? qt_lo : kt_lo;
#pragma unroll
        for (int n4 = 0; n4 < NK / 4; ++n4) {
          float z[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) z[i][j] = 0.f;
#pragma unroll
          for (int kt = 0; kt < 4; ++kt) {
            uint32_t bk[2][4];
            ldsm4t(bk[0], addr_bt<RB>(th_, kt * 16, k0 / 8 + n4 * 4, lane));
            ldsm4t(bk[1], addr_bt<RB>(th_, kt * 16, k0 / 8 + n4 * 4 + 2, lane));
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(z[i], hi[kt], bk[i >> 1][(i & 1) * 2], bk[i >> 1][(i & 1) * 2 + 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(z[i], lo[kt], bk[i >> 1][(i & 1) * 2], bk[i >> 1][(i & 1) * 2 + 1]);
            if constexpr (DT == kF32) {
              ldsm4t(bk[0], addr_bt<RB>(tl_, kt * 16, k0 / 8 + n4 * 4, lane));
              ldsm4t(bk[1], addr_bt<RB>(tl_, kt * 16, k0 / 8 + n4 * 4 + 2, lane));
#pragma unroll
              for (int i = 0; i < 4; ++i) mma(z[i], hi[kt], bk[i >> 1][(i & 1) * 2], bk[i >> 1][(i & 1) * 2 + 1]);
            }
          }
          const float keep = part == 0 ? ga : 1.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = n4 * 4 + i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float old = keep == 0.f ? 0.f : keep * d[n][j];
              d[n][j] = fmaf(j < 2 ? yi0 : yi1, z[i][j], old);
            }
          }
        }
      }
      }
    }
    __syncwarp();
    if (lane == 0) {
      unsigned n;
      asm volatile("atom.acq_rel.cta.shared.add.u32 %0, [%1], 1;" : "=r"(n) : "r"(smem_u32(&left[s])) : "memory");
      if (n == C::WARPS - 1) {
        left[s] = 0;
        if (n0 + NS < nc) fill(n0 + NS);
      }
    }
  }
  if (lane == 0) bulk_wait_all();
  if (gr.ds0 != nullptr) {
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t kd = k0 + 8 * n + 2 * qd + (j & 1), vc = v0 + g + (j >> 1) * 8;
        if (kd < a.Dk && vc < a.Dv)
          gr.ds0[b * gr.ds0s[0] + h * gr.ds0s[1] + kd * gr.ds0s[2] + vc * gr.ds0s[3]] = d[n][j];
      }
  }
}

template <int DT, int DK, int NW, int H>
cudaError_t launch(const GdrArgs& a, const GdrGrads& g, const GdrBwdWs& w, int nc, int64_t head0, int64_t heads,
                   cudaStream_t s) {
  using C = Cfg<DT, DK, NW, H>;
  static_assert(C::BYTES <= 232448, "shared memory of one block");
  using E = typename Fmt<DT>::E;
  constexpr int64_t V = 16 / sizeof(E);
  auto al = [&](const void* p, const int64_t* st) {
    return st[3] == 1 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && st[0] % V == 0 && st[1] % V == 0 && st[2] % V == 0;
  };
  const unsigned vtiles = static_cast<unsigned>((a.Dv + 16 * NW - 1) / (16 * NW));
  const cudaError_t e =
      cudaFuncSetAttribute(gdr_bwd_scan_kernel<DT, DK, NW, H>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
  if (e != cudaSuccess) return e;
  return launch_pdl(gdr_bwd_scan_kernel<DT, DK, NW, H>, static_cast<unsigned>(heads * vtiles), 32 * C::WARPS,
                    C::BYTES, s, a, g, w, nc, head0, vtiles, al(g.dout, g.dos), al(a.v, a.vs), al(g.dv, g.dvs));
}

template <int DT, int DK>
cudaError_t launch_nw(const GdrArgs& a, const GdrGrads& g, const GdrBwdWs& w, int nc, const Device& dev,
                      cudaStream_t s) {
  // As in the forward scan; the tiles that go to the workspace leave no room
  // for eight groups a block.
  constexpr int H2 = DT == kF32 ? 1 : 2;
  const int64_t heads = a.B * a.Hv, groups = (a.Dv + 15) / 16, sms = dev.sm_count;
  const int64_t small = (groups + 1) / 2, large = (groups + 3) / 4;  // blocks of a head
  if (heads * small <= sms) return launch<DT, DK, 2, H2>(a, g, w, nc, 0, heads, s);
  // heads of a last round that would leave half of the SMs idle take the small blocks
  const int64_t round = sms / large, rest = round > 0 ? heads % round : 0;
  if (heads > round && rest > 0 && rest * small <= sms) {
    const cudaError_t e = launch<DT, DK, 4, 1>(a, g, w, nc, 0, heads - rest, s);
    return e != cudaSuccess ? e : launch<DT, DK, 2, H2>(a, g, w, nc, heads - rest, rest, s);
  }
  return launch<DT, DK, 4, 1>(a, g, w, nc, 0, heads, s);
}

template <int DT>
cudaError_t launch_dt(const GdrArgs& a, const GdrGrads& g, const GdrBwdWs& w, int nc, const Device& dev,
                      cudaStream_t s) {
  return a.Dk <= 64 ? launch_nw<DT, 64>(a, g, w, nc, dev, s) : launch_nw<DT, 128>(a, g, w, nc, dev, s);
}

}  // namespace

cudaError_t launch_gdr_bwd_scan(const GdrArgs& a, const GdrGrads& g, Dtype dt, const GdrBwdWs& w, int nc,
                                const Device& dev, cudaStream_t stream) {
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, g, w, nc, dev, stream);
    case kF16: return launch_dt<kF16>(a, g, w, nc, dev, stream);
    case kBF16: return launch_dt<kBF16>(a, g, w, nc, dev, stream);
  }
  return cudaErrorInvalidValue;
}

unsigned read_and_clear_fault_gdr_bwd() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_fault, sizeof(v)) != cudaSuccess) return ~0u;
  if (v != 0 && cudaMemcpyToSymbol(g_fault, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace ccv

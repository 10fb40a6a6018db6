// Gated delta rule, chunked: the scan that carries the state over the chunks
// (formulas and precision in gdr_chunk.cuh).
//
// Everything is kept transposed: a warp owns 16 columns of the state (value
// channels) as S^T, 16 rows of accumulator fragments over all Dk key
// channels.  Then every product of a chunk has the warp's own fragments as
// its A operand and a tile that all warps share as its B operand,
//
//   (K S)^T = S^T K^T,   U^T = R^T T^T,   O^T = .. + U^T P^T,   S^T += U'^T K,
//
// an accumulator fragment is an A fragment of the next product, and no warp
// waits for another: the state never leaves registers.  The shared tiles (k,
// q, T, P and the factors of one chunk) come by bulk copies two chunks deep;
// the warp that is the last to leave a stage refills it, so no warp waits for
// another and none is set aside for the copies.  v is fetched by each warp for
// itself.
//
// With few heads a group of 16 channels takes two warps (H = 2), each with half
// of the key channels: both form their share of K S, exchange it through
// shared memory, take the triangular system both (its result is an operand of
// both halves of the state), and split the output by tokens.  A chunk's chain
// is then about 0.6 as long.
//
// What bounds it: the chain of one chunk after the other, in which a warp
// alternates between tensor instructions (16-bit mma.sync, measured at 8 cycles
// each a quarter SM) and the splitting of their results into the next operands
// (2324 warp instructions a warp and chunk of 128 x 128, bf16).  With eight
// warps a block the tensor pipe is 55 % and the issue slots 31 % busy; a second
// block does not fit beside 255 registers a thread (two warps a block, three
// blocks an SM: spills, 611 us for 597).  A head's columns are spread over as
// many blocks as it takes to fill the SMs; a chunk then takes 7.2 us in blocks
// of eight groups, 4.8 us in blocks of four and 3.1 us in blocks of two groups
// with two warps each.  8192 tokens x 32 heads: 399 us, 128 chunks of 3.1 us;
// 8 x 2048 tokens x 40 heads: 459 us for the 304 heads that fill whole rounds
// and 103 us for the other 16, in small blocks.  All operands of the output have
// both terms, for bf16 too: with one (11 bits) these took 361, 410 and 93 us, and
// one output in ten was another number than the exact value rounded.
//
// A chunk with a value that is not finite (in its inputs or in the state) is
// taken token by token from the original inputs instead, so that nothing
// reaches tokens before it, or past a new sequence, through a product with 0.
#include "gdr_chunk.cuh"

namespace ccv {
namespace {

__device__ unsigned g_fault;

// NW groups of 16 value channels a block, H warps each.
template <int DT, int DK, int NW, int H, bool SAVE>
struct ScanCfg {
  static constexpr int TERMS = DT == kF32 ? 2 : 1;             // of k and q
  static constexpr int TILE = qk_tile_bytes(DK);
  static constexpr int QKB = SAVE ? TERMS * TILE : 2 * TERMS * TILE;  // k alone, or k and q
  static constexpr int MATB = (SAVE ? 2 : 4) * kMatBytes;
  static constexpr int STAGE = QKB + kVecBytes + MATB;
  static constexpr int VROW = DT == kF32 ? 64 : 32;            // bytes of a warp's 16 channels of one token
  static constexpr int VBYTES = kC * VROW;
  static constexpr int OBYTES = (DT == kF32 || SAVE) ? 0 : kC * 32;
  static constexpr int WARPS = NW * H;
  static constexpr int SIMG = SAVE ? 2 * img_state_bytes(DK) / H : 0;  // this warp's part of S hi and S lo
  static constexpr int UIMG = SAVE ? 2 * kTokBytes / H : 0;             // U hi and lo, or one of them
  static constexpr int XBYTES = H == 2 ? (SAVE ? 4096 : 6144) : 0;  // a warp's share of K S (and Q S) for the other
  static constexpr int BYTES = 2 * STAGE + WARPS * (VBYTES + OBYTES + XBYTES + SIMG + UIMG) + 64;
};

// This warp's v of one chunk into its buffer; rows past the sequence and
// channels past Dv are zero.
template <int DT>
__device__ __forceinline__ void fetch_v(const GdrArgs& a, int64_t b, int64_t h, int64_t t0, int64_t v0, bool vec,
                                        uint8_t* buf, int lane) {
  using F = Fmt<DT>;
  using E = typename F::E;
  constexpr int VROW = DT == kF32 ? 64 : 32;
  constexpr int PIECES = VROW / 16;
  const E* p = static_cast<const E*>(a.v) + b * a.vs[0] + h * a.vs[2] + v0 * a.vs[3];
  if (vec) {
#pragma unroll
    for (int i = 0; i < kC * PIECES / 32; ++i) {
      const int x = i * 32 + lane, r = x / PIECES, pc = x % PIECES;
      const bool in = t0 + r < a.L;
      const E* src = p + (in ? (t0 + r) * a.vs[1] : 0) + pc * (16 / static_cast<int>(sizeof(E)));
      cp_async16(buf + r * VROW + pc * 16, src, in);
    }
  } else {
    for (int x = lane; x < kC * 16; x += 32) {
      const int r = x >> 4, c = x & 15;
      E e = F::from_f(0.f);
      if (t0 + r < a.L && v0 + c < a.Dv) e = p[(t0 + r) * a.vs[1] + c * a.vs[3]];
      *reinterpret_cast<E*>(buf + r * VROW + c * sizeof(E)) = e;
    }
  }
  cp_async_commit();
}

// One chunk token by token, from the original inputs, on the warp's 16 rows
// of S^T (rows g and g + 8 of this thread, key channels 8 i + 2 qd + {0, 1}).
// Two warps of a pair add their sums through xb (own) and xo (the other's).
template <int DT, int NK, int H, bool SAVE>
__device__ __noinline__ void token_by_token(const GdrArgs& a, float (&st)[NK][4], int64_t b, int64_t h, int64_t t0,
                                            int64_t v0, float (&u)[8][4], int lane, int half, int pair, float* xb,
                                            const float* xo) {
  using F = Fmt<DT>;
  using E = typename F::E;
  const int g = lane >> 2, qd = lane & 3;
  const int64_t hk = h / (a.Hv / a.Hk);
  const E* kp = static_cast<const E*>(a.k) + b * a.ks[0] + hk * a.ks[2];
  const E* qp = static_cast<const E*>(a.q) + b * a.qs[0] + hk * a.qs[2];
  const int64_t r0 = v0 + g, r1 = v0 + g + 8;
  const int k0 = half * NK * 8;
  for (int n = 0; n < 8; ++n)
    for (int j = 0; j < 4; ++j) u[n][j] = 0.f;
  for (int i = 0; i < kC && t0 + i < a.L; ++i) {
    const int64_t t = t0 + i;
    float dec = expf(a.g[b * a.gs[0] + t * a.gs[1] + h * a.gs[2]]);
    const float be = F::to_f(static_cast<const E*>(a.beta)[b * a.bs[0] + t * a.bs[1] + h * a.bs[2]]);
    if (a.seq != nullptr && t > 0 && a.seq[b * a.ss[0] + t * a.ss[1]] != a.seq[b * a.ss[0] + (t - 1) * a.ss[1]]) {
      dec = 0.f;
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) st[n][j] = 0.f;
    }
    float p0 = 0.f, p1 = 0.f, o0 = 0.f, o1 = 0.f, qk = 0.f;
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t kd = k0 + 8 * n + 2 * qd + e;
        const float kv = kd < a.Dk ? F::to_f(kp[t * a.ks[1] + kd * a.ks[3]]) : 0.f;
        const float qv = kd < a.Dk ? F::to_f(qp[t * a.qs[1] + kd * a.qs[3]]) : 0.f;
        if (kd < a.Dk) {
          p0 = fmaf(kv, st[n][e], p0);
          p1 = fmaf(kv, st[n][2 + e], p1);
          o0 = fmaf(qv, st[n][e], o0);
          o1 = fmaf(qv, st[n][2 + e], o1);
        }
        qk = fmaf(kv, qv, qk);
      }
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
      p0 += __shfl_xor_sync(kFullMask, p0, m);
      p1 += __shfl_xor_sync(kFullMask, p1, m);
      o0 += __shfl_xor_sync(kFullMask, o0, m);
      o1 += __shfl_xor_sync(kFullMask, o1, m);
      qk += __shfl_xor_sync(kFullMask, qk, m);
    }
    if constexpr (H == 2) {
      const float x[5] = {p0, p1, o0, o1, qk};
#pragma unroll
      for (int j = 0; j < 5; ++j) xb[j * 32 + lane] = x[j];
      pair_sync(pair);
      p0 += xo[lane], p1 += xo[32 + lane], o0 += xo[64 + lane], o1 += xo[96 + lane], qk += xo[128 + lane];
      pair_sync(pair);
    }
    const E* vp = static_cast<const E*>(a.v) + b * a.vs[0] + t * a.vs[1] + h * a.vs[2];
    const float x0 = r0 < a.Dv ? F::to_f(vp[r0 * a.vs[3]]) : 0.f, x1 = r1 < a.Dv ? F::to_f(vp[r1 * a.vs[3]]) : 0.f;
    const float u0 = be * (x0 - dec * p0), u1 = be * (x1 - dec * p1);
    if constexpr (SAVE) {
      if (((i >> 1) & 3) == qd) u[i >> 3][i & 1] = u0, u[i >> 3][2 + (i & 1)] = u1;
    } else if (qd == 0 && half == 0) {
        E* op = static_cast<E*>(a.out) + b * a.os[0] + t * a.os[1] + h * a.os[2];
        if (r0 < a.Dv) op[r0 * a.os[3]] = F::from_f(a.scale * fmaf(qk, u0, dec * o0));
        if (r1 < a.Dv) op[r1 * a.os[3]] = F::from_f(a.scale * fmaf(qk, u1, dec * o1));
    }
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t kd = k0 + 8 * n + 2 * qd + e;
        const float kv = kd < a.Dk ? F::to_f(kp[t * a.ks[1] + kd * a.ks[3]]) : 0.f;
        if (kd < a.Dk) {
          st[n][e] = fmaf(kv, u0, dec * st[n][e]);
          st[n][2 + e] = fmaf(kv, u1, dec * st[n][2 + e]);
        }
      }
  }
}

template <int DT, int DK, int NW, int H, bool SAVE>
__global__ void __launch_bounds__(32 * NW * H, 1)
    gdr_scan_kernel(const GdrArgs a, const uint8_t* qk_ws, const uint8_t* pack_ws, uint8_t* img, int nc, int64_t head0,
                    unsigned vtiles, bool vvec, bool ovec) {
  pdl_enter();
  using C = ScanCfg<DT, DK, NW, H, SAVE>;
  using F = Fmt<DT>;
  using E = typename F::E;
  constexpr int RB = DK * 2;
  constexpr int NK = DK / 8 / H;  // key channel tiles of a warp
  extern __shared__ __align__(128) uint8_t sm[];
  uint8_t* vbuf0 = sm + 2 * C::STAGE;
  uint8_t* obuf0 = vbuf0 + C::WARPS * C::VBYTES;
  uint8_t* xbuf0 = obuf0 + C::WARPS * C::OBYTES;
  uint8_t* ibuf0 = xbuf0 + C::WARPS * C::XBYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(ibuf0 + C::WARPS * (C::SIMG + C::UIMG));
  unsigned* left = reinterpret_cast<unsigned*>(full + 2);  // warps that have left a stage

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

  const uint8_t* qk = qk_ws + (b * a.Hk + hk) * nc * qk_pack_bytes(DK, C::TERMS);
  const uint8_t* pkg = pack_ws + bh * nc * kPackBytes;
  auto fill = [&](int c) {
    uint8_t* dst = sm + (c & 1) * C::STAGE;
    uint64_t* bar = &full[c & 1];
    constexpr uint32_t kVec = SAVE ? kVecBytes : kVecFwdBytes;
    const uint8_t* pc = pkg + static_cast<int64_t>(c) * kPackBytes;
    mbar_arrive_expect_tx(bar, C::QKB + kVec + C::MATB);
    bulk_load(dst, qk + static_cast<int64_t>(c) * qk_pack_bytes(DK, C::TERMS), C::QKB, bar);
    bulk_load(dst + C::QKB, pc, kVec, bar);
    bulk_load(dst + C::QKB + kVecBytes, pc + kVecBytes, C::MATB, bar);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&full[s], 1);
      left[s] = 0;
    }
    fence_barrier_init();
    for (int c = 0; c < 2 && c < nc; ++c) fill(c);
  }
  __syncthreads();

  const bool active = v0 < a.Dv;
  uint8_t* vb = vbuf0 + warp * C::VBYTES;
  uint8_t* ob = obuf0 + warp * C::OBYTES;
  uint8_t* ibuf = ibuf0 + warp * (C::SIMG + C::UIMG);
  const uint32_t simg = smem_u32(ibuf), uimg = simg + C::SIMG;
  const bool wvec = vvec && v0 + 16 <= a.Dv, wovec = ovec && v0 + 16 <= a.Dv;

  float st[NK][4];
#pragma unroll
  for (int n = 0; n < NK; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t kd = k0 + 8 * n + 2 * qd + (j & 1), vc = v0 + g + (j >> 1) * 8;
      st[n][j] = (a.s0 != nullptr && kd < a.Dk && vc < a.Dv)
                     ? a.s0[b * a.s0s[0] + h * a.s0s[1] + kd * a.s0s[2] + vc * a.s0s[3]]
                     : 0.f;
    }
  if (active && nc > 0) fetch_v<DT>(a, b, h, 0, v0, wvec, vb, lane);

  for (int c = 0; c < nc; ++c) {
    const int s = c & 1;
    const int64_t t0 = static_cast<int64_t>(c) * kC;
    bool late = !mbar_wait(&full[s], (c >> 1) & 1);
    if constexpr (H == 2) late = pair_any(pair, late);  // a pair gives up together
    if (late) {
      // give up: no copy of this warp's, nor the other stage's, must outlive the block
      cp_async_wait_all();
      if (lane == 0) {
        atomicOr(&g_fault, kFaultConsumerWait);
        if (c + 1 < nc && !mbar_wait(&full[s ^ 1], ((c + 1) >> 1) & 1)) atomicOr(&g_fault, kFaultDrainWait);
        if constexpr (SAVE) bulk_wait_all();
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
      // SAVE: this slice's image of the chunk, and the staging of its parts
      const int ns = static_cast<int>((a.Dv + 15) / 16);
      uint8_t* gimg = SAVE ? img + ((bh * nc + c) * ns + v0 / 16) * ImgF::bytes(DK) : nullptr;
      if constexpr (SAVE) {
        if (lane == 0) bulk_wait_read();
        __syncwarp();
      }
      bool bad = vecs[kHdBad] != 0.f;

      // U's image; `kept`: a chunk with values that are not finite.  Of two warps one keeps hi, the other lo.
      auto save_u = [&](const float (&x)[8][4], auto kept) {
        uint32_t uh[4][4], ul[4][4];
        float i0, i1;
        bool lost = false;
        split_rows<8, true, kept.value>(x, uh, ul, i0, i1, lost);
        if (!kept.value && lost) i0 = i1 = __uint_as_float(kLostBits);
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          // tokens 16 np..: fragments of rows v are read back as rows of tokens
          const uint32_t at = uimg + off32(np * 16 + (lane & 7) + ((lane >> 4) & 1) * 8, (lane >> 3) & 1);
          if (H == 1 || half == 0) stsm4t(at, uh[np]);
          if (H == 1) stsm4t(at + kTokBytes, ul[np]);
          if (H == 2 && half == 1) stsm4t(at, ul[np]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          bulk_store(gimg + ImgF::u(DK) + half * kTokBytes, ibuf + C::SIMG, C::UIMG);
          bulk_commit();
        }
        if (qd == 0 && half == 0) {
          float* inv = reinterpret_cast<float*>(gimg + ImgF::inv(DK)) + 32;
          inv[g] = i0, inv[g + 8] = i1;
        }
      };
      auto save_state = [&](float i0, float i1) {  // its tiles are in the staging memory
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          bulk_store(gimg + half * (C::SIMG / 2), ibuf, C::SIMG / 2);
          bulk_store(gimg + img_state_bytes(DK) + half * (C::SIMG / 2), ibuf + C::SIMG / 2, C::SIMG / 2);
          bulk_commit();
        }
        if (qd == 0) {
          float* inv = reinterpret_cast<float*>(gimg + ImgF::inv(DK));
#pragma unroll
          for (int x = 0; x < 2 / H; ++x) inv[(half + x) * 16 + g] = i0, inv[(half + x) * 16 + g + 8] = i1;
        }
      };
      // the state's row factors
      float a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        a0 = amax3(a0, st[n][0], st[n][1]);
        a1 = amax3(a1, st[n][2], st[n][3]);
      }
      const unsigned m0 = quad_max(__float_as_uint(a0)), m1 = quad_max(__float_as_uint(a1));
      bad = bad || m0 >= kInfBits || m1 >= kInfBits;
      float f0, f1, si0, si1;
      row_factor(m0, f0, si0);
      row_factor(m1, f1, si1);
      const uint64_t p0 = pk(f0, f0), p1 = pk(f1, f1);
      // (K S)^T and (Q S)^T
      float ks[8][4], qs[8][4];
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) ks[n][j] = qs[n][j] = 0.f;
#pragma unroll
      for (int kt = 0; kt < NK / 2; ++kt) {
        const int piece = k0 / 8 + 2 * kt;
        uint32_t hi[4], lo[4];
        split2f(st[2 * kt][0], st[2 * kt][1], p0, hi[0], lo[0]);
        split2f(st[2 * kt][2], st[2 * kt][3], p1, hi[1], lo[1]);
        split2f(st[2 * kt + 1][0], st[2 * kt + 1][1], p0, hi[2], lo[2]);
        split2f(st[2 * kt + 1][2], st[2 * kt + 1][3], p1, hi[3], lo[3]);
        if constexpr (SAVE) {
          const uint32_t at = simg + (kt >> 1) * kBlkBytes +
                              off64((lane & 7) + ((lane >> 3) & 1) * 8, (kt & 1) * 2 + (lane >> 4));
          stsm4(at, hi);
          stsm4(at + C::SIMG / 2, lo);
        }
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t bk[4];
          ldsm4(bk, addr_b<RB>(kt_hi, np * 16, piece, lane));
          mma(ks[2 * np], hi, bk[0], bk[1]);
          mma(ks[2 * np + 1], hi, bk[2], bk[3]);
          mma(ks[2 * np], lo, bk[0], bk[1]);
          mma(ks[2 * np + 1], lo, bk[2], bk[3]);
          if constexpr (DT == kF32) {
            ldsm4(bk, addr_b<RB>(kt_lo, np * 16, piece, lane));
            mma(ks[2 * np], hi, bk[0], bk[1]);
            mma(ks[2 * np + 1], hi, bk[2], bk[3]);
          }
          if constexpr (!SAVE) {
            ldsm4(bk, addr_b<RB>(qt_hi, np * 16, piece, lane));
            mma(qs[2 * np], hi, bk[0], bk[1]);
            mma(qs[2 * np + 1], hi, bk[2], bk[3]);
            mma(qs[2 * np], lo, bk[0], bk[1]);
            mma(qs[2 * np + 1], lo, bk[2], bk[3]);
            if constexpr (DT == kF32) {
              ldsm4(bk, addr_b<RB>(qt_lo, np * 16, piece, lane));
              mma(qs[2 * np], hi, bk[0], bk[1]);
              mma(qs[2 * np + 1], hi, bk[2], bk[3]);
            }
          }
        }
      }

      if constexpr (SAVE) save_state(si0, si1);
      // true values, and the other half's share; O: this warp's tokens are 16 np0.. and 16 np1..
      const int np0 = H == 2 ? half : 0, np1 = H == 2 ? 3 - half : 0;
      float qo[H == 2 ? 4 : 1][4];
      if constexpr (H == 2) {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          set_pair(ks[n], 0, fmul2(pair_of(ks[n], 0), both(si0)));
          set_pair(ks[n], 1, fmul2(pair_of(ks[n], 1), both(si1)));
          if constexpr (!SAVE) {
            set_pair(qs[n], 0, fmul2(pair_of(qs[n], 0), both(si0)));
            set_pair(qs[n], 1, fmul2(pair_of(qs[n], 1), both(si1)));
          }
        }
      }
      // what is left of the state's factors to be taken out (with two warps: nothing)
      const uint64_t ks0 = both(H == 2 ? -1.f : -si0), ks1 = both(H == 2 ? -1.f : -si1);
      const uint64_t qs0 = both(H == 2 ? 1.f : si0), qs1 = both(H == 2 ? 1.f : si1);
      if constexpr (H == 2) {
        float4* x4 = reinterpret_cast<float4*>(xb);
        const float4* o4 = reinterpret_cast<const float4*>(xo);
#pragma unroll
        for (int n = 0; n < 8; ++n) x4[n * 32 + lane] = make_float4(ks[n][0], ks[n][1], ks[n][2], ks[n][3]);
        if constexpr (!SAVE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // tiles 0, 1, 6, 7 are the first half's tokens, 2..5 the second's
            const int lo_t = i < 2 ? i : i + 4, hi_t = i + 2;
            float send[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              send[j] = half == 0 ? qs[hi_t][j] : qs[lo_t][j];
              qo[i][j] = half == 0 ? qs[lo_t][j] : qs[hi_t][j];
            }
            x4[(8 + i) * 32 + lane] = make_float4(send[0], send[1], send[2], send[3]);
          }
        }
        pair_sync(pair);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float4 o = o4[n * 32 + lane];
          ks[n][0] += o.x, ks[n][1] += o.y, ks[n][2] += o.z, ks[n][3] += o.w;
        }
        if constexpr (!SAVE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 o = o4[(8 + i) * 32 + lane];
            // the second half's tokens are 16 np0 = 16 (tiles 2, 3) and 16 np1 = 32 (tiles 4, 5)
            qo[i][0] += o.x, qo[i][1] += o.y, qo[i][2] += o.z, qo[i][3] += o.w;
          }
        }
      }

      // R = beta (V - gi K S)
      cp_async_wait_all();
      __syncwarp();
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        float x[2][4];
        if constexpr (DT == kF32) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[t][j] = *reinterpret_cast<const float*>(vb + (np * 16 + t * 8 + qd * 2 + (j & 1)) * C::VROW +
                                                        (g + (j >> 1) * 8) * 4);
        } else {
          uint32_t r[4];
          ldsm4t(r, smem_u32(vb) + (np * 16 + (lane & 7) + ((lane >> 4) & 1) * 8) * C::VROW + ((lane >> 3) & 1) * 16);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[t][j] = F::word_elem(r[2 * t + (j >> 1)], j & 1);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int n = 2 * np + t;
          const uint64_t cf = ld_pair(slot + kVKS * kC + n * 8 + qd * 2), be = ld_pair(slot + kVBeta * kC + n * 8 + qd * 2);
          const uint64_t c0 = fmul2(cf, ks0), c1 = H == 2 ? c0 : fmul2(cf, ks1);
          set_pair(ks[n], 0, fmul2(be, ffma2(c0, pair_of(ks[n], 0), pair_of(x[t], 0))));
          set_pair(ks[n], 1, fmul2(be, ffma2(c1, pair_of(ks[n], 1), pair_of(x[t], 1))));
        }
      }
      uint32_t hi[4][4], lo[4][4];
      float ri0, ri1;
      split_rows<8, true>(ks, hi, lo, ri0, ri1, bad);
      // (with two warps: also the barrier after which the exchange buffers may be written again)
      bad = H == 2 ? pair_any(pair, bad) : __any_sync(kFullMask, bad) != 0;

      if (bad) {
        float tmp[NK][4];  // a copy: the state itself has to stay in registers
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) tmp[n][j] = st[n][j];
        if constexpr (SAVE) {  // the state's image again
          if (lane == 0) bulk_wait_all();
          __syncwarp();
          float i0, i1;
          keep_state(tmp, simg, C::SIMG / 2, lane, i0, i1);
          save_state(i0, i1);
        }
        float ut[8][4];
        token_by_token<DT, NK, H, SAVE>(a, tmp, b, h, t0, v0, ut, lane, half, pair, xb, xo);
        if constexpr (SAVE) save_u(ut, std::true_type{});
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) st[n][j] = tmp[n][j];
        __syncwarp();
        if (c + 1 < nc) fetch_v<DT>(a, b, h, t0 + kC, v0, wvec, vb, lane);
      } else {
        __syncwarp();
        if (c + 1 < nc) fetch_v<DT>(a, b, h, t0 + kC, v0, wvec, vb, lane);
        // U^T = R^T T^T, T lower triangular
        float u[8][4];
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          float x[2][2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[0][i][j] = x[1][i][j] = 0.f;
#pragma unroll
          for (int kt = 0; kt <= np; ++kt) {
            uint32_t bt[4];
            ldsm4(bt, addr_b<128>(th, np * 16, 2 * kt, lane));
            mma(x[0][0], hi[kt], bt[0], bt[1]);
            mma(x[0][1], hi[kt], bt[2], bt[3]);
            mma(x[1][0], lo[kt], bt[0], bt[1]);
            mma(x[1][1], lo[kt], bt[2], bt[3]);
            ldsm4(bt, addr_b<128>(tl, np * 16, 2 * kt, lane));
            mma(x[1][0], hi[kt], bt[0], bt[1]);
            mma(x[1][1], hi[kt], bt[2], bt[3]);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint64_t ti = ld_pair(slot + kVTInv * kC + (2 * np + t) * 8 + qd * 2);
            set_pair(u[2 * np + t], 0,
                     fmul2(fadd2(pair_of(x[0][t], 0), pair_of(x[1][t], 0)), fmul2(ti, both(ri0))));
            set_pair(u[2 * np + t], 1,
                     fmul2(fadd2(pair_of(x[0][t], 1), pair_of(x[1][t], 1)), fmul2(ti, both(ri1))));
          }
        }
        if constexpr (SAVE) {
          save_u(u, std::false_type{});
        } else {
          // O^T = scale (gi (Q S)^T + U^T P^T)
          float ui0, ui1;
          bool ignore = false;
          split_rows<8, true>(u, hi, lo, ui0, ui1, ignore);
#pragma unroll
          for (int i = 0; i < 4 / H; ++i) {
            const int np = H == 1 ? i : i == 0 ? np0 : np1;
            float x[2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[0][j] = x[1][j] = 0.f;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
              if (kt > np) continue;
              uint32_t bp[4];
              ldsm4(bp, addr_b<128>(ph, np * 16, 2 * kt, lane));
              mma(x[0], hi[kt], bp[0], bp[1]);
              mma(x[1], hi[kt], bp[2], bp[3]);
              mma(x[0], lo[kt], bp[0], bp[1]);
              mma(x[1], lo[kt], bp[2], bp[3]);
              ldsm4(bp, addr_b<128>(pl, np * 16, 2 * kt, lane));
              mma(x[0], hi[kt], bp[0], bp[1]);
              mma(x[1], hi[kt], bp[2], bp[3]);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int n = 2 * np + t;
              const float(&qv)[4] = H == 1 ? qs[2 * i + t] : qo[H == 2 ? 2 * i + t : 0];
              const uint64_t cq = ld_pair(slot + kVQS * kC + n * 8 + qd * 2), cp = ld_pair(slot + kVP * kC + n * 8 + qd * 2);
              set_pair(x[t], 0, ffma2(fmul2(cp, both(ui0)), pair_of(x[t], 0), fmul2(fmul2(cq, qs0), pair_of(qv, 0))));
              set_pair(x[t], 1, ffma2(fmul2(cp, both(ui1)), pair_of(x[t], 1), fmul2(fmul2(cq, qs1), pair_of(qv, 1))));
            }
            if (DT != kF32 && wovec) {
              if constexpr (DT != kF32) {
                const uint32_t r[4] = {F::pack2(x[0][0], x[0][1]), F::pack2(x[0][2], x[0][3]),
                                       F::pack2(x[1][0], x[1][1]), F::pack2(x[1][2], x[1][3])};
                stsm4t(smem_u32(ob) + (np * 16 + (lane & 7) + ((lane >> 4) & 1) * 8) * 32 + ((lane >> 3) & 1) * 16, r);
              }
            } else {
              E* op = static_cast<E*>(a.out) + b * a.os[0] + h * a.os[2];
#pragma unroll
              for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int64_t tok = t0 + np * 16 + t * 8 + qd * 2 + (j & 1), vc = v0 + g + (j >> 1) * 8;
                  if (tok < a.L && vc < a.Dv) op[tok * a.os[1] + vc * a.os[3]] = F::from_f(x[t][j]);
                }
            }
          }
          if (DT != kF32 && wovec) {
            __syncwarp();
            E* op = static_cast<E*>(a.out) + b * a.os[0] + h * a.os[2] + v0;
#pragma unroll
            for (int i = 0; i < 4 / H; ++i) {
              const int x = (H == 1 ? i : i == 0 ? np0 : np1) * 32 + lane, r = x >> 1, pc = x & 1;
              const uint4 w = lds128(ob + r * 32 + pc * 16);
              if (t0 + r < a.L) *reinterpret_cast<uint4*>(op + (t0 + r) * a.os[1] + pc * 8) = w;
            }
          }
        }
        // S^T <- ga S^T + (gc U)^T K
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const uint64_t cu = ld_pair(slot + kVU * kC + n * 8 + qd * 2);
          set_pair(u[n], 0, fmul2(cu, pair_of(u[n], 0)));
          set_pair(u[n], 1, fmul2(cu, pair_of(u[n], 1)));
        }
        float ui0, ui1;
        bool ignore = false;
        split_rows<8, true>(u, hi, lo, ui0, ui1, ignore);
#pragma unroll
        for (int n4 = 0; n4 < NK / 4; ++n4) {
          float x[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll
          for (int kt = 0; kt < 4; ++kt) {
            uint32_t bk[2][4];
            ldsm4t(bk[0], addr_bt<RB>(kt_hi, kt * 16, k0 / 8 + n4 * 4, lane));
            ldsm4t(bk[1], addr_bt<RB>(kt_hi, kt * 16, k0 / 8 + n4 * 4 + 2, lane));
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(x[i], hi[kt], bk[i >> 1][(i & 1) * 2], bk[i >> 1][(i & 1) * 2 + 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(x[i], lo[kt], bk[i >> 1][(i & 1) * 2], bk[i >> 1][(i & 1) * 2 + 1]);
            if constexpr (DT == kF32) {
              ldsm4t(bk[0], addr_bt<RB>(kt_lo, kt * 16, k0 / 8 + n4 * 4, lane));
              ldsm4t(bk[1], addr_bt<RB>(kt_lo, kt * 16, k0 / 8 + n4 * 4 + 2, lane));
#pragma unroll
              for (int i = 0; i < 4; ++i) mma(x[i], hi[kt], bk[i >> 1][(i & 1) * 2], bk[i >> 1][(i & 1) * 2 + 1]);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = n4 * 4 + i;
            set_pair(st[n], 0, ffma2(both(ui0), pair_of(x[i], 0), fmul2(both(ga), pair_of(st[n], 0))));
            set_pair(st[n], 1, ffma2(both(ui1), pair_of(x[i], 1), fmul2(both(ga), pair_of(st[n], 1))));
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) {
      unsigned n;
      asm volatile("atom.acq_rel.cta.shared.add.u32 %0, [%1], 1;" : "=r"(n) : "r"(smem_u32(&left[s])) : "memory");
      if (n == C::WARPS - 1) {  // every warp has left the stage
        left[s] = 0;
        if (c + 2 < nc) fill(c + 2);
      }
    }
  }
  if (SAVE && lane == 0) bulk_wait_all();
  if (a.s1 != nullptr) {
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t kd = k0 + 8 * n + 2 * qd + (j & 1), vc = v0 + g + (j >> 1) * 8;
        if (kd < a.Dk && vc < a.Dv)
          a.s1[b * a.s1s[0] + h * a.s1s[1] + kd * a.s1s[2] + vc * a.s1s[3]] = st[n][j];
      }
  }
}

// Heads head0 .. head0 + heads - 1 of the [B, Hv].
struct Heads {
  int64_t head0, heads;
};

template <int DT, int DK, int NW, int H, bool SAVE>
cudaError_t launch(const GdrArgs& a, const uint8_t* qk, const uint8_t* pkg, uint8_t* img, int nc, Heads hd,
                   cudaStream_t s) {
  using C = ScanCfg<DT, DK, NW, H, SAVE>;
  static_assert(C::BYTES <= 232448, "shared memory of one block");
  using E = typename Fmt<DT>::E;
  constexpr int64_t V = 16 / sizeof(E);
  auto al = [&](const void* p, const int64_t* st) {
    return st[3] == 1 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && st[0] % V == 0 && st[1] % V == 0 && st[2] % V == 0;
  };
  const unsigned vtiles = static_cast<unsigned>((a.Dv + 16 * NW - 1) / (16 * NW));
  const cudaError_t e = cudaFuncSetAttribute(gdr_scan_kernel<DT, DK, NW, H, SAVE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
  if (e != cudaSuccess) return e;
  return launch_pdl(gdr_scan_kernel<DT, DK, NW, H, SAVE>, static_cast<unsigned>(hd.heads * vtiles), 32 * C::WARPS,
                    C::BYTES, s, a, qk, pkg, img, nc, hd.head0, vtiles, al(a.v, a.vs), !SAVE && al(a.out, a.os));
}

template <int DT, int DK, bool SAVE>
cudaError_t launch_nw(const GdrArgs& a, const uint8_t* qk, const uint8_t* pkg, uint8_t* img, int nc, Heads hd,
                      const Device& dev, cudaStream_t s) {
  // Blocks of few channels while that still puts no more than one on an SM.
  // Two warps a group only where one each would leave half the quarters of an
  // SM idle (32 heads, 8192 tokens: 662 -> 493 us with all kernels; with 64
  // heads, four groups a block, 119 -> 145 us in the state-keeping scan).
  const int64_t groups = (a.Dv + 15) / 16, sms = dev.sm_count;
  if constexpr (DT == kF32) {  // two terms of k and q: the stages leave room for one warp a group, four groups
    if (hd.heads * ((groups + 1) / 2) <= sms) return launch<DT, DK, 2, 1, SAVE>(a, qk, pkg, img, nc, hd, s);
    return launch<DT, DK, 4, 1, SAVE>(a, qk, pkg, img, nc, hd, s);
  } else {
    if (hd.heads * ((groups + 1) / 2) <= sms) return launch<DT, DK, 2, 2, SAVE>(a, qk, pkg, img, nc, hd, s);
    if (hd.heads * ((groups + 3) / 4) <= sms) return launch<DT, DK, 4, 1, SAVE>(a, qk, pkg, img, nc, hd, s);
    // More than one block an SM: full rounds of whole heads, and the heads of
    // a last round that would not fill the SMs spread over smaller blocks
    // behind them (a chunk takes 7.2, 4.8 or 3.1 us by the three shapes; 8 x 2048
    // tokens x 40 heads 970 -> 870 us).
    const int64_t rest = hd.heads % sms;
    if (hd.heads > sms && groups <= 8 && rest > 0 && rest * ((groups + 3) / 4) <= sms) {
      const cudaError_t e =
          launch<DT, DK, 8, 1, SAVE>(a, qk, pkg, img, nc, Heads{hd.head0, hd.heads - rest}, s);
      if (e != cudaSuccess) return e;
      return launch_nw<DT, DK, SAVE>(a, qk, pkg, img, nc, Heads{hd.head0 + hd.heads - rest, rest}, dev, s);
    }
    return launch<DT, DK, 8, 1, SAVE>(a, qk, pkg, img, nc, hd, s);
  }
}

template <int DT, int DK>
cudaError_t launch_k(const GdrArgs& a, const uint8_t* qk, const uint8_t* pk, uint8_t* img, int nc,
                     const Device& dev, cudaStream_t s) {
  return img != nullptr ? launch_nw<DT, DK, true>(a, qk, pk, img, nc, Heads{0, a.B * a.Hv}, dev, s)
                       : launch_nw<DT, DK, false>(a, qk, pk, img, nc, Heads{0, a.B * a.Hv}, dev, s);
}

template <int DT>
cudaError_t launch_dt(const GdrArgs& a, const uint8_t* qk, const uint8_t* pk, uint8_t* img, int nc,
                      const Device& dev, cudaStream_t s) {
  return a.Dk <= 64 ? launch_k<DT, 64>(a, qk, pk, img, nc, dev, s)
                    : launch_k<DT, 128>(a, qk, pk, img, nc, dev, s);
}

}  // namespace

cudaError_t launch_gdr_scan(const GdrArgs& a, Dtype dt, const uint8_t* qk_ws, const uint8_t* pack_ws, uint8_t* img,
                            int nc, const Device& dev, cudaStream_t stream) {
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, qk_ws, pack_ws, img, nc, dev, stream);
    case kF16: return launch_dt<kF16>(a, qk_ws, pack_ws, img, nc, dev, stream);
    case kBF16: return launch_dt<kBF16>(a, qk_ws, pack_ws, img, nc, dev, stream);
  }
  return cudaErrorInvalidValue;
}

uint64_t gdr_qk_bytes(const GdrArgs& a, Dtype dt, int nc) {
  return static_cast<uint64_t>(a.B * a.Hk) * nc * qk_pack_bytes(a.Dk <= 64 ? 64 : 128, dt == kF32 ? 2 : 1);
}

uint64_t gdr_pack_bytes(const GdrArgs& a, int nc) { return static_cast<uint64_t>(a.B * a.Hv) * nc * kPackBytes; }

unsigned read_and_clear_fault_gdr() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_fault, sizeof(v)) != cudaSuccess) return ~0u;
  if (v != 0 && cudaMemcpyToSymbol(g_fault, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace ccv

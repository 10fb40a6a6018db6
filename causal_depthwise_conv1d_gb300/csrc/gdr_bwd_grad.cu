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
// are summed here one after the other, in a fixed order.
//
// The scans left their parts as FP16 tiles (hi and lo, every value channel
// scaled by its own power of two), a slice of 16 channels at a time: a block
// streams the slices through a ring of bulk copies and does nothing per slice
// but matrix loads and products.  A slice is one step of 16 of the sum over
// the channels, so the channels' factors are multiplied into the A operand
// (powers of two at most 1, relative to the product's largest; what falls
// below 2^-24 of it is zero), and <S0, D> is the trace of a product.
//
// What bounds it: no unit alone.  Of 265 us (2 x 2048 tokens x 32 heads on 16 key
// heads, 128 x 128, bf16) the tensor pipe is busy 35 % (products of two FP32
// operands take three instructions) and the issue slots 38 %: a chunk and head
// takes 56 thousand warp instructions, and one block of sixteen warps fills the
// registers of an SM, so its phases follow one another.  Of some 34 thousand
// cycles a head, the slices take 17, the matrices A and B 4, the products with
// them 4, and the rest is the factors before the slices and the sums after them.
// What measured faster: factors and first slices of the next head on their way
// while this one is finished, dQ and dK leaving as whole rows (308 -> 281 us),
// sums of independent products in turn (281 -> 266 us), nothing for tiles above
// the diagonal (263 us; eight warps instead of sixteen cost 5 us more).  That
// values which are not finite stay where they are costs 2 us.
#include "gdr_chunk.cuh"

namespace ccv {
namespace {

__device__ unsigned g_fault;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;  // 4 groups of 16 tokens x 4 quarters of the columns
// Two bits a warp: its group of tokens.  In this order each quarter of the SM
// has two or three of the ten warps whose tiles of the 64 x 64 matrices are not
// all above the diagonal.
constexpr unsigned kRowOf = 0x9c9339e4u;

template <typename E>
struct alignas(2 * sizeof(E)) Pair {
  E x, y;
};

// Products over the value channels, each with its own factors.
enum { kOS0 = 0, kOS1, kRS0, kRS1, kUD0, kUD1, kSD0, kSD1, kOU, kRU, kProducts };

template <int DT, int DK, bool REP>
struct Cfg {
  static constexpr int TERMS = DT == kF32 ? 2 : 1;
  static constexpr int TILE = qk_tile_bytes(DK);
  static constexpr int QKB = qk_pack_bytes(DK, TERMS);
  static constexpr int STAGE = ImgF::bytes(DK) + ImgB::bytes(DK, TERMS);
  static constexpr int STAGES = DT == kF32 ? 2 : 4;
  static constexpr int RING = STAGES * STAGE > 8 * kMatBytes ? STAGES * STAGE : 8 * kMatBytes;  // later: A and B
  static constexpr int OROW = DK * (DT == kF32 ? 4 : 2);  // a row of dQ or dK on its way out, in the ring's memory
  static_assert(2 * kC * OROW <= RING, "dQ and dK in the ring");
  static constexpr int TOTAL = REP ? 2 * kC * DK * 4 : 0;  // dQ and dK of the heads so far
  static constexpr int O_RING = QKB + kVecBytes;
  static constexpr int O_TOTAL = O_RING + RING;
  static constexpr int O_MULT = O_TOTAL + TOTAL;           // half [kProducts][kGdrBwdDv]
  static constexpr int O_F = O_MULT + kProducts * kGdrBwdDv * 2;
  static constexpr int BYTES = O_F + 1536 * 4;
};

// Float scratch.
enum { kFVdr = 0, kFPart = 64 /* [4][3][64] */, kFdG = 832, kFRed = 896 /* [2][kWarps] */, kFMax = 928 /* 4 unsigned */,
       kFRef = 932 /* kProducts ints */, kFBar = 944 /* barriers and counters, 8-byte aligned */ };

__device__ __forceinline__ uint32_t hmul(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// An A operand times factors of its summed index: lo for the first eight, hi for the others.
__device__ __forceinline__ void scaled(uint32_t (&r)[4], const uint32_t (&a)[4], uint32_t m_lo, uint32_t m_hi) {
  r[0] = hmul(a[0], m_lo);
  r[1] = hmul(a[1], m_lo);
  r[2] = hmul(a[2], m_hi);
  r[3] = hmul(a[3], m_hi);
}

// d (two column tiles) += (hi + lo of a) (hi + lo of b), without lo lo; LO: a has a lo part.
template <bool LO>
__device__ __forceinline__ void mma3(float (*d)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                     const uint32_t (&bh)[4], const uint32_t (&bl)[4]) {
  mma(d[0], ah, bh[0], bh[1]);
  mma(d[1], ah, bh[2], bh[3]);
  mma(d[0], ah, bl[0], bl[1]);
  mma(d[1], ah, bl[2], bl[3]);
  if constexpr (LO) {
    mma(d[0], al, bh[0], bh[1]);
    mma(d[1], al, bh[2], bh[3]);
  }
}

// The exponent of a row that was lost (kLostBits): more than any product's.
constexpr int kLost = 1024;

// Multiply by 2^e for any int e that a sum of two float exponents can be; NaN for a lost row's.
struct Pow2 {
  float a, b;
  __device__ __forceinline__ explicit Pow2(int e) {
    const int h = e >> 1, r = e - h;
    a = __uint_as_float(e >= kLost / 2 ? 0x7fffffffu : static_cast<unsigned>(max(1, min(254, h + 127))) << 23);
    b = __uint_as_float(static_cast<unsigned>(max(1, min(254, r + 127))) << 23);
  }
  __device__ __forceinline__ float operator()(float x) const { return x * a * b; }
};

template <int DT, int DK, bool REP>
__global__ void __launch_bounds__(kThreads, 1)
    gdr_bwd_grad_kernel(const GdrArgs a, const GdrGrads gr, const GdrBwdWs w, int nc, bool vec) {
  pdl_enter();
  using C = Cfg<DT, DK, REP>;
  using F = Fmt<DT>;
  using E = typename F::E;
  constexpr int RB = DK * 2;
  constexpr int NT = DK / 32;  // column tiles of 8 of one warp (a quarter of DK)
  constexpr bool OLO = DT == kF32;
  extern __shared__ __align__(128) uint8_t sm[];
  float* fs = reinterpret_cast<float*>(sm + C::O_F);
  uint64_t* full = reinterpret_cast<uint64_t*>(fs + kFBar);
  unsigned* left = reinterpret_cast<unsigned*>(full + C::STAGES);
  int* ref = reinterpret_cast<int*>(fs + kFRef);
  uint16_t* mult = reinterpret_cast<uint16_t*>(sm + C::O_MULT);
  const float* vecs = reinterpret_cast<const float*>(sm + C::QKB);
  const float* slot = vecs + kVecHead;
  const int* seg = reinterpret_cast<const int*>(slot + kVSeg * kC);
  const uint32_t base = smem_u32(sm);
  const uint32_t kt_hi = base, kt_lo = base + C::TILE, qt_hi = base + C::TERMS * C::TILE, qt_lo = qt_hi + C::TILE;
  const uint32_t mats = base + C::O_RING;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, qd = lane & 3;
  const int wc = warp >> 2, half = wc >> 1, wr = kRowOf >> (2 * warp) & 3;
  const int i0 = wr * 16 + g, i1 = i0 + 8;
  // indices below 2^31 (checked on the host): 32-bit divisions
  const int64_t id = blockIdx.x;
  const unsigned uc = blockIdx.x % static_cast<unsigned>(nc), ubk = blockIdx.x / static_cast<unsigned>(nc);
  const int64_t c = uc, hk = ubk % static_cast<unsigned>(a.Hk), b = ubk / static_cast<unsigned>(a.Hk);
  const int64_t t0 = c * kC;
  const int nt = static_cast<int>(a.L - t0 < kC ? a.L - t0 : kC);
  const int64_t rep = static_cast<unsigned>(a.Hv) / static_cast<unsigned>(a.Hk);
  const int ns = static_cast<int>((a.Dv + 15) / 16);
  constexpr int BF = ImgF::bytes(DK), BB = ImgB::bytes(DK, C::TERMS);

  int64_t ch = (b * a.Hv + hk * rep) * nc + c;
  auto fill = [&](int64_t ch, int sl, int n) {  // slice sl of this chunk and head as the block's n-th copy
    uint8_t* dst = sm + C::O_RING + (n % C::STAGES) * C::STAGE;
    uint64_t* bar = &full[n % C::STAGES];
    mbar_arrive_expect_tx(bar, C::STAGE);
    bulk_load(dst, w.img_f + (ch * ns + sl) * BF, BF, bar);
    bulk_load(dst + BF, w.img_b + (ch * ns + sl) * BB, BB, bar);
  };
  // What a head needs before its slices, one element a thread: the channel's
  // seven factors, a piece of the vector part, a share of dR.v.  Brought to the
  // L2 cache a head ahead.
  static_assert(kGdrBwdDv <= kThreads && kVecBytes / 16 <= kThreads, "one element a thread");
  const bool channel = tid < ns * 16;
  float fac[7], vdr;
  uint4 vpiece;
  auto fetch = [&](int64_t ch) {
    const uint8_t* imf = w.img_f + ch * ns * BF + ImgF::inv(DK);
    const uint8_t* imb = w.img_b + ch * ns * BB + ImgB::inv(DK, C::TERMS);
    if (channel) {
      const float* pf = reinterpret_cast<const float*>(imf + (tid >> 4) * BF) + (tid & 15);
      const float* pb = reinterpret_cast<const float*>(imb + (tid >> 4) * BB) + (tid & 15);
#pragma unroll
      for (int i = 0; i < 3; ++i) fac[i] = pf[16 * i];
#pragma unroll
      for (int i = 0; i < 4; ++i) fac[3 + i] = pb[16 * i];
    }
    if (tid < kVecBytes / 16) vpiece = reinterpret_cast<const uint4*>(w.pack + ch * kPackBytes)[tid];
    auto share = [&](int sl) { return reinterpret_cast<const float*>(imb + sl * BB)[64 + tid % kC]; };
    vdr = tid / kC < ns ? share(tid / kC) : 0.f;  // not added to anything here: nothing waits for it
    for (int sl = tid / kC + kThreads / kC; sl < ns; sl += kThreads / kC) vdr += share(sl);
  };
  auto ahead = [&](int64_t ch) {
    const int y = tid - ns * 6;  // two lines of factors of the one image, four of the other, the vector part
    const uint8_t* p = nullptr;
    if (tid < ns * 2)
      p = w.img_f + (ch * ns + (tid >> 1)) * BF + ImgF::inv(DK) + (tid & 1) * 128;
    else if (tid < ns * 6)
      p = w.img_b + (ch * ns + ((tid - ns * 2) >> 2)) * BB + ImgB::inv(DK, C::TERMS) + ((tid - ns * 2) & 3) * 128;
    else if (y < kVecBytes / 128)
      p = w.pack + ch * kPackBytes + y * 128;
    if (p != nullptr) asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
  };
  auto start = [&](int64_t ch, int n) {  // the head's maxima and first slices
    if (tid < 4) reinterpret_cast<unsigned*>(fs + kFMax)[tid] = 0;
    if (tid < kProducts) ref[tid] = -1000;
    if (warp == kWarps - 1 && lane < C::STAGES && lane < ns) fill(ch, lane, n + lane);
  };
  if (warp == kWarps - 1 && lane < C::STAGES) {
    mbar_init(&full[lane], 1);
    left[lane] = 0;
    fence_barrier_init();
  }
  start(ch, 0);
  {  // k and q tiles
    const uint4* src = reinterpret_cast<const uint4*>(w.qk + id * C::QKB);
    uint4* dst = reinterpret_cast<uint4*>(sm);
#pragma unroll 8
    for (int i = tid; i < C::QKB / 16; i += kThreads) dst[i] = src[i];
  }
  float4* total = reinterpret_cast<float4*>(sm + C::O_TOTAL);  // this thread's tiles at [tile][tid]
  int n_copy = 0;  // copies consumed so far

  for (int64_t r = 0; r < rep; ++r, ch += nc) {
    const int64_t h = hk * rep + r;
    fetch(ch);
    if (r + 1 < rep) ahead(ch + nc);
    __syncthreads();  // the last head's factors and sums have been read
    if (tid < kVecBytes / 16) reinterpret_cast<uint4*>(sm + C::QKB)[tid] = vpiece;
    fs[kFPart + tid] = vdr;
    // exponents of the channels' factors; each product's largest
    int e[kProducts];
    if (warp * 32 < ns * 16) {
      int x[7];
#pragma unroll
      for (int i = 0; i < 7; ++i) {
        const unsigned f = __float_as_uint(fac[i]);
        x[i] = f == kLostBits ? kLost : static_cast<int>(f >> 23) - 127;
      }
      const int s0 = x[0], s1 = x[1], u = x[2], d0 = x[3], d1 = x[4], rr = x[5], o = x[6];
      e[kOS0] = o + s0, e[kOS1] = o + s1, e[kRS0] = rr + s0, e[kRS1] = rr + s1, e[kUD0] = u + d0, e[kUD1] = u + d1;
      e[kSD0] = s0 + d0, e[kSD1] = s1 + d1, e[kOU] = o + u, e[kRU] = rr + u;
#pragma unroll
      for (int p = 0; p < kProducts; ++p) {
        const int m = __reduce_max_sync(kFullMask, channel ? e[p] : -1000);
        if (lane == 0) atomicMax(&ref[p], m);
      }
    }
    __syncthreads();
    if (channel) {
#pragma unroll
      for (int p = 0; p < kProducts; ++p) {
        const int d = e[p] - ref[p];
        mult[p * kGdrBwdDv + tid] = d >= -14 ? (d + 15) << 10 : d >= -24 ? 1 << (d + 24) : 0;
      }
    }
    if (tid < kC) {  // dR.v: the shares in order
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < kThreads / kC; ++i) x += fs[kFPart + i * kC + tid];
      fs[kFVdr + tid] = x;
    }
    __syncthreads();

    float dq[NT][4], z[NT][4], dk[NT][4], dp[2][4], dl[2][4], tr[2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) dq[n][j] = z[n][j] = dk[n][j] = 0.f;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) dp[n][j] = dl[n][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) tr[0][j] = tr[1][j] = 0.f;

    for (int sl = 0; sl < ns; ++sl, ++n_copy) {
      const int s = n_copy % C::STAGES;
      if (!mbar_wait(&full[s], (n_copy / C::STAGES) & 1)) {
        // give up: wait for the copies still in flight as well
        if (lane == 0) {
          atomicOr(&g_fault, kFaultConsumerWait);
          for (int k = 1; k < C::STAGES && sl + k < ns; ++k)
            mbar_wait(&full[(n_copy + k) % C::STAGES], ((n_copy + k) / C::STAGES) & 1);
        }
        return;
      }
      const uint32_t f0 = base + C::O_RING + s * C::STAGE, b0 = f0 + BF;
      const uint32_t s_hi = f0, s_lo = s_hi + img_state_bytes(DK), u_hi = f0 + ImgF::u(DK), u_lo = u_hi + kTokBytes;
      const uint32_t d_hi = b0, d_lo = d_hi + img_state_bytes(DK), r_hi = b0 + ImgB::r(DK), r_lo = r_hi + kTokBytes;
      const uint32_t o_hi = b0 + ImgB::o(DK), o_lo = o_hi + kTokBytes;
      auto factors = [&](int p, uint32_t& lo, uint32_t& hi) {
        const uint32_t* m = reinterpret_cast<const uint32_t*>(mult + p * kGdrBwdDv + sl * 16);
        lo = m[qd];
        hi = m[4 + qd];
      };
      const uint32_t at = off32(wr * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
      uint32_t oh[4], ol[4], rh[4], rl[4], m0, m1;
      ldsm4(oh, o_hi + at);
      if constexpr (OLO) ldsm4(ol, o_lo + at);
      ldsm4(rh, r_hi + at);
      ldsm4(rl, r_lo + at);
      if (wc <= wr) {  // dO U^T and dR U^T, the column tiles up to the diagonal
        uint32_t xo[4], xl[4], yh[4], yl[4];
        factors(kOU, m0, m1);
        scaled(xo, oh, m0, m1);
        if constexpr (OLO) scaled(xl, ol, m0, m1);
        factors(kRU, m0, m1);
        scaled(yh, rh, m0, m1);
        scaled(yl, rl, m0, m1);
        uint32_t bh[4], bl[4];
        const uint32_t bt = off32(wc * 16 + (lane & 7) + ((lane >> 4) & 1) * 8, (lane >> 3) & 1);
        ldsm4(bh, u_hi + bt);
        ldsm4(bl, u_lo + bt);
        mma3<OLO>(dp, xo, xl, bh, bl);
        mma3<true>(dl, yh, yl, bh, bl);
      }
      uint32_t uh[4], ul[4];
      ldsm4(uh, u_hi + at);
      ldsm4(ul, u_lo + at);
      factors(kOS0 + half, m0, m1);
      scaled(oh, oh, m0, m1);
      if constexpr (OLO) scaled(ol, ol, m0, m1);
      factors(kRS0 + half, m0, m1);
      scaled(rh, rh, m0, m1);
      scaled(rl, rl, m0, m1);
      factors(kUD0 + half, m0, m1);
      scaled(uh, uh, m0, m1);
      scaled(ul, ul, m0, m1);
      const int rowt = (lane & 7) + ((lane >> 3) & 1) * 8, pct = lane >> 4;
#pragma unroll
      for (int np = 0; np < NT / 2; ++np) {
        const int n0 = wc * (DK / 4) + np * 16;
        const uint32_t bt = (n0 >> 5) * kBlkBytes + off64(rowt, ((n0 & 31) >> 3) + pct);
        uint32_t bh[4], bl[4];
        ldsm4t(bh, s_hi + bt);
        ldsm4t(bl, s_lo + bt);
        // two pairs of sums in turn: a sum's next instruction is four away
        mma(dq[2 * np], oh, bh[0], bh[1]);
        mma(dq[2 * np + 1], oh, bh[2], bh[3]);
        mma(z[2 * np], rh, bh[0], bh[1]);
        mma(z[2 * np + 1], rh, bh[2], bh[3]);
        mma(dq[2 * np], oh, bl[0], bl[1]);
        mma(dq[2 * np + 1], oh, bl[2], bl[3]);
        mma(z[2 * np], rh, bl[0], bl[1]);
        mma(z[2 * np + 1], rh, bl[2], bl[3]);
        if constexpr (OLO) {
          mma(dq[2 * np], ol, bh[0], bh[1]);
          mma(dq[2 * np + 1], ol, bh[2], bh[3]);
        }
        mma(z[2 * np], rl, bh[0], bh[1]);
        mma(z[2 * np + 1], rl, bh[2], bh[3]);
        if (np == wr) {  // <S0, D>: one row group for each tile pair; the diagonal of D S0^T
          uint32_t ah[4], al[4];
          const uint32_t tt = (n0 >> 5) * kBlkBytes +
                              off64((lane & 7) + ((lane >> 4) & 1) * 8, ((n0 & 31) >> 3) + ((lane >> 3) & 1));
          ldsm4t(ah, d_hi + tt);
          ldsm4t(al, d_lo + tt);
          factors(kSD0 + half, m0, m1);
          scaled(ah, ah, m0, m1);
          scaled(al, al, m0, m1);
          mma3<true>(tr, ah, al, bh, bl);
        }
        ldsm4t(bh, d_hi + bt);
        ldsm4t(bl, d_lo + bt);
        mma3<true>(&dk[2 * np], uh, ul, bh, bl);
      }
      __syncwarp();
      if (lane == 0) {
        unsigned n;
        asm volatile("atom.acq_rel.cta.shared.add.u32 %0, [%1], 1;" : "=r"(n) : "r"(smem_u32(&left[s])) : "memory");
        if (n == kWarps - 1) {  // every warp has left the stage
          left[s] = 0;
          if (sl + C::STAGES < ns) fill(ch, sl + C::STAGES, n_copy + C::STAGES);
        }
      }
    }

    // true values of the products with the states
    const float be0 = slot[kVBeta * kC + i0], be1 = slot[kVBeta * kC + i1];
    float klast = 0.f;  // sum of k.(gc U D^T) over this thread's elements
    {
      const float gi0 = slot[kVGi * kC + i0], gi1 = slot[kVGi * kC + i1];
      const float gc0 = slot[kVGc * kC + i0], gc1 = slot[kVGc * kC + i1];
      const Pow2 po(ref[kOS0 + half]), pr(ref[kRS0 + half]), pd(ref[kUD0 + half]);
      const float q0 = a.scale * gi0, q1 = a.scale * gi1;
      const float ki0 = gc0 == 0.f ? 0.f : slot[kVKInv * kC + i0], ki1 = gc1 == 0.f ? 0.f : slot[kVKInv * kC + i1];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int col = wc * (DK / 4) + n * 8 + qd * 2;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float gi = e ? gi1 : gi0, gc = e ? gc1 : gc0, qf = e ? q1 : q0;
          const uint32_t off = tile_off<RB>(e ? i1 : i0, col >> 3) + (col & 7) * 2;
          float2 k2 = __half22float2(*reinterpret_cast<const __half2*>(sm + off));
          if constexpr (DT == kF32) {
            const float2 l2 = __half22float2(*reinterpret_cast<const __half2*>(sm + C::TILE + off));
            k2.x += l2.x, k2.y += l2.y;
          }
          float part = 0.f;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int j = 2 * e + x;
            // factors of zero (another sequence) select
            dq[n][j] = gi == 0.f ? 0.f : po(dq[n][j]) * qf;
            z[n][j] = gi == 0.f ? 0.f : -(pr(z[n][j]) * gi);
            dk[n][j] = gc == 0.f ? 0.f : pd(dk[n][j]) * gc;
            part = fmaf(x ? k2.y : k2.x, dk[n][j], part);
          }
          klast = fmaf(e ? ki1 : ki0, part, klast);
        }
      }
    }
    // the diagonal of tr: row g (g + 8) of tile 0 (1) is column 2 qd + e
    float sd = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (2 * qd + e == g) sd += tr[0][e] + tr[1][2 + e];
    sd = Pow2(ref[kSD0 + half])(sd);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      klast += __shfl_xor_sync(kFullMask, klast, m);
      sd += __shfl_xor_sync(kFullMask, sd, m);
    }
    if (lane == 0) fs[kFRed + warp] = klast, fs[kFRed + kWarps + warp] = sd;

    // A and B with the factors of the products they enter; one power of two a matrix
    float mx[4] = {0.f, 0.f, 0.f, 0.f};
    {
      const float gh0 = slot[kVGHi * kC + i0], gl0 = slot[kVGLo * kC + i0];
      const float gh1 = slot[kVGHi * kC + i1], gl1 = slot[kVGLo * kC + i1];
      const int s0 = seg[i0], s1 = seg[i1];
      const Pow2 pu(ref[kOU]), pr(ref[kRU]);
      const float qi0 = slot[kVQInv * kC + i0], qi1 = slot[kVQInv * kC + i1];
      const float bk0 = be0 * slot[kVKInv * kC + i0], bk1 = be1 * slot[kVKInv * kC + i1];
      const bool lower = wc <= wr;  // the tiles above the diagonal are never read
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (!lower) break;
        const int j0 = wc * 16 + n * 8 + qd * 2;
        const float2 gj = *reinterpret_cast<const float2*>(slot + kVGHi * kC + j0);
        const float2 lj = *reinterpret_cast<const float2*>(slot + kVGLo * kC + j0);
        const float2 kj = *reinterpret_cast<const float2*>(slot + kVKInv * kC + j0);
        const int2 sj = *reinterpret_cast<const int2*>(seg + j0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + (e & 1), i = e < 2 ? i0 : i1;
          const bool in = j <= i && ((e & 1) ? sj.y : sj.x) == (e < 2 ? s0 : s1);
          const float gam = exp2f(((e < 2 ? gh0 : gh1) - ((e & 1) ? gj.y : gj.x)) +
                                       ((e < 2 ? gl0 : gl1) - ((e & 1) ? lj.y : lj.x)));
          dp[n][e] = in ? pu(dp[n][e]) * (a.scale * gam) : 0.f;
          dl[n][e] = in && j < i ? -(pr(dl[n][e]) * gam) : 0.f;
        }
        mx[0] = amax3(amax3(mx[0], dp[n][0] * kj.x, dp[n][1] * kj.y), dp[n][2] * kj.x, dp[n][3] * kj.y);
        mx[1] = amax3(amax3(mx[1], dp[n][0] * qi0, dp[n][1] * qi0), dp[n][2] * qi1, dp[n][3] * qi1);
        mx[2] = amax3(amax3(mx[2], dl[n][0] * kj.x, dl[n][1] * kj.y), dl[n][2] * kj.x, dl[n][3] * kj.y);
        mx[3] = amax3(amax3(mx[3], dl[n][0] * bk0, dl[n][1] * bk0), dl[n][2] * bk1, dl[n][3] * bk1);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const unsigned x = warp_max(__float_as_uint(mx[m]));
        if (lane == 0) atomicMax(reinterpret_cast<unsigned*>(fs + kFMax) + m, x);
      }
      // rows i0 (e = 0) or i1, columns of tile n: the entries with the four products' factors
      auto entries = [&](int n, int e, float (&x)[4][2]) {
        const float2 kj = *reinterpret_cast<const float2*>(slot + kVKInv * kC + wc * 16 + n * 8 + qd * 2);
        const float qi = e ? qi1 : qi0, bk = e ? bk1 : bk0;
        const float p0 = dp[n][2 * e], p1 = dp[n][2 * e + 1], l0 = dl[n][2 * e], l1 = dl[n][2 * e + 1];
        // selected: a factor that is not finite stays in its sequence and below the diagonal
        auto by = [](float x, float f) { return x == 0.f ? 0.f : x * f; };
        x[0][0] = by(p0, kj.x), x[0][1] = by(p1, kj.y), x[1][0] = by(p0, qi), x[1][1] = by(p1, qi);
        x[2][0] = by(l0, kj.x), x[2][1] = by(l1, kj.y), x[3][0] = by(l0, bk), x[3][1] = by(l1, bk);
      };
      unsigned* top = reinterpret_cast<unsigned*>(fs + kFMax);
      __syncthreads();  // also: every warp is done with the ring
      if (max(max(top[0], top[1]), max(top[2], top[3])) >= kInfBits) {  // the largest finite ones (finite_max)
        __syncthreads();
        if (tid < 4) top[tid] = 0;
        __syncthreads();
        unsigned fin[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (!lower) continue;
            float x[4][2];
            entries(n, e, x);
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
              for (int j = 0; j < 2; ++j) fin[m] = max(fin[m], mag(x[m][j]) < kInfBits ? mag(x[m][j]) : 0u);
          }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const unsigned x = warp_max(fin[m]);
          if (lane == 0) atomicMax(&top[m], x);
        }
        __syncthreads();
      }
      float f[4], inv[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) row_factor(top[m], f[m], inv[m]);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (!lower) break;
        const int col = wc * 16 + n * 8 + qd * 2;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t off = tile_off<128>(e ? i1 : i0, col >> 3) + (col & 7) * 2;
          float x[4][2];
          entries(n, e, x);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t hi, lo;
            split2f(x[m][0], x[m][1], pk(f[m], f[m]), hi, lo);
            *reinterpret_cast<uint32_t*>(sm + C::O_RING + 2 * m * kMatBytes + off) = hi;
            *reinterpret_cast<uint32_t*>(sm + C::O_RING + (2 * m + 1) * kMatBytes + off) = lo;
          }
        }
      }
      __syncthreads();
      // products over the chunk's tokens
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint32_t mh = mats + 2 * m * kMatBytes, ml = mh + kMatBytes;
        const uint32_t bh_t = m == 1 ? qt_hi : kt_hi, bl_t = m == 1 ? qt_lo : kt_lo;
        float x[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) x[n][j] = 0.f;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          // rows i, summed j <= i; or rows j, summed i >= j by transposed loads
          if ((m & 1) ? kt < wr : kt > wr) continue;
          uint32_t ah[4], al[4];
          if (m & 1) {
            ldsm4t(ah, addr_at<128>(mh, kt * 16, wr * 2, lane));
            ldsm4t(al, addr_at<128>(ml, kt * 16, wr * 2, lane));
          } else {
            ldsm4(ah, addr_a<128>(mh, wr * 16, 2 * kt, lane));
            ldsm4(al, addr_a<128>(ml, wr * 16, 2 * kt, lane));
          }
#pragma unroll
          for (int np = 0; np < NT / 2; ++np) {
            const int piece = (wc * (DK / 4) + np * 16) / 8;
            uint32_t bb[4];
            ldsm4t(bb, addr_bt<RB>(bh_t, kt * 16, piece, lane));
            mma(x[2 * np], ah, bb[0], bb[1]);
            mma(x[2 * np + 1], ah, bb[2], bb[3]);
            mma(x[2 * np], al, bb[0], bb[1]);
            mma(x[2 * np + 1], al, bb[2], bb[3]);
            if constexpr (DT == kF32) {
              ldsm4t(bb, addr_bt<RB>(bl_t, kt * 16, piece, lane));
              mma(x[2 * np], ah, bb[0], bb[1]);
              mma(x[2 * np + 1], ah, bb[2], bb[3]);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float& dst = m == 0 ? dq[n][j] : m == 2 ? z[n][j] : dk[n][j];
            dst = fmaf(inv[m], x[n][j], dst);
          }
      }
    }

    // dK complete; dot products of each token's rows
    float dots[3][2] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = wc * (DK / 4) + n * 8 + qd * 2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t off = tile_off<RB>(e ? i1 : i0, col >> 3) + (col & 7) * 2;
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
    // sums over the heads, and out with the last
    if constexpr (REP) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (r > 0) {
          const float4 x = total[n * kThreads + tid], y = total[(NT + n) * kThreads + tid];
          dq[n][0] += x.x, dq[n][1] += x.y, dq[n][2] += x.z, dq[n][3] += x.w;
          dk[n][0] += y.x, dk[n][1] += y.y, dk[n][2] += y.z, dk[n][3] += y.w;
        }
        if (r + 1 < rep) {
          total[n * kThreads + tid] = make_float4(dq[n][0], dq[n][1], dq[n][2], dq[n][3]);
          total[(NT + n) * kThreads + tid] = make_float4(dk[n][0], dk[n][1], dk[n][2], dk[n][3]);
        }
      }
    }
    const bool last = r + 1 == rep;
    __syncthreads();  // the dot products are there; the matrices have been read
    if (!last) {
      if (warp == kWarps - 1) fence_proxy_async_smem();  // the ring held matrices written by threads
      start(ch + nc, n_copy);
    } else {  // dQ and dK through the ring's memory, to leave as whole rows
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = (wc * (DK / 4) + n * 8 + qd * 2) * static_cast<int>(sizeof(E));
          uint8_t* o = sm + C::O_RING + tile_off<C::OROW>(e ? i1 : i0, at >> 4) + (at & 15);
          Pair<E> x{F::from_f(dq[n][2 * e]), F::from_f(dq[n][2 * e + 1])};
          *reinterpret_cast<Pair<E>*>(o) = x;
          x = {F::from_f(dk[n][2 * e]), F::from_f(dk[n][2 * e + 1])};
          *reinterpret_cast<Pair<E>*>(o + kC * C::OROW) = x;
        }
    }
    if (tid < kC) {
      const int i = tid;
      const int64_t t = t0 + i;
      const float ki = slot[kVKInv * kC + i], qi = slot[kVQInv * kC + i], be = slot[kVBeta * kC + i];
      auto dot = [&](int d) {  // the four quarters in order
        const float* p = fs + kFPart + d * kC + i;
        return (p[0] + p[3 * kC]) + (p[6 * kC] + p[9 * kC]);
      };
      const float qdq = qi * dot(0), kdk = ki * dot(1), kz = ki * dot(2);
      if (i < nt)
        static_cast<E*>(gr.dbeta)[b * gr.dbs[0] + t * gr.dbs[1] + h * gr.dbs[2]] = F::from_f(fs[kFVdr + i] + kz);
      float x = qdq - kdk + 2.f * be * kz;
      if (i == kC - 1) {
        float kl = 0.f, sdot = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) kl += fs[kFRed + k], sdot += fs[kFRed + kWarps + k];
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
    if (last) {
      constexpr int PIECES = C::OROW / 16;
      E* const base_o[2] = {static_cast<E*>(gr.dq) + b * gr.dqs[0] + hk * gr.dqs[2],
                            static_cast<E*>(gr.dk) + b * gr.dks[0] + hk * gr.dks[2]};
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int64_t* st = o ? gr.dks : gr.dqs;
        const uint8_t* src = sm + C::O_RING + o * kC * C::OROW;
        for (int x = tid; x < kC * PIECES; x += kThreads) {
          const int row = x / PIECES, piece = x % PIECES;
          if (row >= nt) break;
          E* dst = base_o[o] + (t0 + row) * st[1];
          const int col = piece * F::VEC;
          const uint4 y = *reinterpret_cast<const uint4*>(src + tile_off<C::OROW>(row, piece));
          if (vec) {
            if (col < a.Dk) *reinterpret_cast<uint4*>(dst + col) = y;
          } else {
            E e[F::VEC];
            memcpy(e, &y, 16);
#pragma unroll
            for (int j = 0; j < F::VEC; ++j)
              if (col + j < a.Dk) dst[(col + j) * st[3]] = e[j];
          }
        }
      }
    }
  }
}

template <int DT, int DK, bool REP>
cudaError_t launch(const GdrArgs& a, const GdrGrads& g, const GdrBwdWs& w, int nc, cudaStream_t s) {
  using C = Cfg<DT, DK, REP>;
  static_assert(C::BYTES <= 232448, "shared memory of one block");
  const cudaError_t e =
      cudaFuncSetAttribute(gdr_bwd_grad_kernel<DT, DK, REP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
  if (e != cudaSuccess) return e;
  constexpr int64_t V = Fmt<DT>::VEC;
  auto ok = [&](const void* p, const int64_t* st) {
    return st[3] == 1 && a.Dk % V == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && st[0] % V == 0 &&
           st[1] % V == 0 && st[2] % V == 0;
  };
  const bool vec = ok(g.dq, g.dqs) && ok(g.dk, g.dks);
  return launch_pdl(gdr_bwd_grad_kernel<DT, DK, REP>, static_cast<unsigned>(a.B * a.Hk * nc), kThreads, C::BYTES, s, a,
                    g, w, nc, vec);
}

template <int DT>
cudaError_t launch_dt(const GdrArgs& a, const GdrGrads& g, const GdrBwdWs& w, int nc, cudaStream_t s) {
  if (a.Hv == a.Hk) return a.Dk <= 64 ? launch<DT, 64, false>(a, g, w, nc, s) : launch<DT, 128, false>(a, g, w, nc, s);
  return a.Dk <= 64 ? launch<DT, 64, true>(a, g, w, nc, s) : launch<DT, 128, true>(a, g, w, nc, s);
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

uint64_t gdr_img_f_bytes(int64_t Dk) { return ImgF::bytes(Dk <= 64 ? 64 : 128); }
uint64_t gdr_img_b_bytes(int64_t Dk, Dtype dt) { return ImgB::bytes(Dk <= 64 ? 64 : 128, dt == kF32 ? 2 : 1); }

unsigned read_and_clear_fault_gdr_grad() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_fault, sizeof(v)) != cudaSuccess) return ~0u;
  if (v != 0 && cudaMemcpyToSymbol(g_fault, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace ccv

// Gated delta rule, chunked: what a chunk needs that does not depend on the
// state (formulas in gdr_chunk.cuh), for all chunks at once.
//
// A block of eight warps takes one chunk of one key head: it scales k and q to
// FP16 tiles, forms k k^T and q k^T with tensor instructions, and for each of
// the key head's value heads the factors, P, and T = (I + L)^-1.
//
// The inverse of the unit lower triangular matrix is made by blocks in FP32:
// the four 16 x 16 diagonal blocks by forward substitution (one warp each,
// a lane holds a column), then twice [A 0; C D]^-1 = [A' 0; -D' C A' D'].
// This is as stable as substitution and has 16 + 4 dependent steps instead of 64.
// The block products run on tf32 tensor instructions, every operand as the sum
// of two tf32 values (22 bits; the exponent range of FP32, so nothing is scaled)
// and FP32 sums; on the FP32 units, whose operands all come from shared memory,
// the 92 us below were 107.
//
// What bounds it: the steps of one block follow one another between barriers,
// so shared memory is kept small enough for four blocks an SM (the inverse and
// L lie where k and q were, and T where L was; 64 registers).  The issue slots
// are then 56 % busy, the load/store path 47 %, the integer pipe 38 %.  4096
// chunks and heads of 128 channels on half as many key heads (8192 tokens x 32
// heads) take 92 us, 2048 take 48 us, 10240 with a key head each 281 us.  Blocks
// of four warps were 2.8 times as slow as three blocks of eight an SM, which
// were 1.1 times as slow as four.  The scan of the decays runs while k and q are
// on their way (5 us more beside the other warps' wait for it).
//
// The results leave as bulk copies of the shared-memory image that the scan
// reads back, already in its tile order.
#include "gdr_chunk.cuh"

namespace ccv {
namespace {

constexpr int kThreads = 256;
constexpr int kLd = 68;  // leading dimension of L and X
constexpr float kFarDecay = 16384.f;  // of log 2: a decay by more is this one

template <int DT, int DK>
struct PrepSmem {
  static constexpr int TERMS = DT == kF32 ? 2 : 1;
  static constexpr int QK = qk_pack_bytes(DK, TERMS);
  static constexpr int MAT = kC * kLd * 4;
  static constexpr int FIRST = QK > 2 * MAT ? QK : 2 * MAT;  // k and q, then X and L, and T over L
  static constexpr int BYTES = FIRST + kVecBytes + 2 * kMatBytes + 6 * kC * 4 + 64;
};

// Eight rows of k or q a warp to FP16 tiles, each row scaled by its power of
// two; eight elements a lane.
template <int DT, int DK>
struct RowLoad {
  using F = Fmt<DT>;
  using E = typename F::E;
  static constexpr int LPR = DK / 8;        // lanes of one row
  static constexpr int RPP = 32 / LPR;      // rows of one pass
  static constexpr int PASSES = 8 / RPP;
  static constexpr int W = DT == kF32 ? 2 : 1;  // 16-byte words of a lane
  uint4 raw[PASSES][W];

  __device__ __forceinline__ void load(const void* base, const int64_t* st, int64_t b, int64_t h, int64_t t0, int nt,
                                       int64_t Dk, bool vec) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const E* p = static_cast<const E*>(base) + b * st[0] + h * st[2];
    const int c0 = (lane % LPR) * 8;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = warp * 8 + i * RPP + lane / LPR;
#pragma unroll
      for (int w = 0; w < W; ++w) raw[i][w] = make_uint4(0, 0, 0, 0);
      if (r < nt) {
        const E* row = p + (t0 + r) * st[1];
        if (vec) {
#pragma unroll
          for (int w = 0; w < W; ++w) raw[i][w] = __ldg(reinterpret_cast<const uint4*>(row + c0 + w * F::VEC));
        } else {
#pragma unroll
          for (int w = 0; w < W; ++w) {
            E e[F::VEC];
#pragma unroll
            for (int j = 0; j < F::VEC; ++j) {
              const int c = c0 + w * F::VEC + j;
              e[j] = c < Dk ? row[c * st[3]] : static_cast<E>(0);
            }
            raw[i][w] = vec_from_bits<DT>(e);
          }
        }
      }
    }
  }

  // A row with a value that is not finite is stored as zeros with the factor NaN.
  // Entries of the matrices that its token enters become NaN by the factor; zeros
  // of them, above the diagonal or across a new sequence, meet no infinity here.
  __device__ __forceinline__ void store(uint8_t* hi, uint8_t* lo, float* inv, bool& bad) const {
    constexpr int RB = DK * 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = (lane % LPR) * 8;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = warp * 8 + i * RPP + lane / LPR;
      float x[8];
#pragma unroll
      for (int w = 0; w < W; ++w) unpack16<DT>(raw[i][w], x + w * F::VEC);
      float mf = 0.f;
#pragma unroll
      for (int j = 0; j < 8; j += 2) mf = amax3(mf, x[j], x[j + 1]);
      unsigned m = __float_as_uint(mf);
#pragma unroll
      for (int k = 1; k < LPR; k <<= 1) m = max(m, __shfl_xor_sync(kFullMask, m, k));
      const bool lost = m >= kInfBits;
      bad = bad || lost;
      float f, iv;
      row_factor(m, f, iv);
      if (lost) iv = __uint_as_float(0x7fffffffu);
      if (lane % LPR == 0) inv[r] = iv;
      const uint32_t off = tile_off<RB>(r, c0 >> 3);
      uint32_t h[4], l[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (DT == kF32)
          split2(x[2 * j] * f, x[2 * j + 1] * f, h[j], l[j]);
        else
          h[j] = h2(x[2 * j] * f, x[2 * j + 1] * f);
        if (lost) h[j] = l[j] = 0u;
      }
      *reinterpret_cast<uint4*>(hi + off) = make_uint4(h[0], h[1], h[2], h[3]);
      if constexpr (DT == kF32) *reinterpret_cast<uint4*>(lo + off) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
};

// An FP32 value as a sum of two tf32 values (11 bits each).
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d += a (8 columns m of 16 rows) times the values at `row` (two of a row, of
// the summed index), both split: the summed index of an operand's registers
// runs 0, 2, 4, 6 and 1, 3, 5, 7, so that an accumulator tile is the next
// product's operand as it is.
__device__ __forceinline__ void step_tf32(float (&d)[4], const float (&a)[4], const float* row) {
  const float2 bv = *reinterpret_cast<const float2*>(row);
  uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) split_tf32(a[i], ah[i], al[i]);
  split_tf32(bv.x, bh[0], bl[0]);
  split_tf32(bv.y, bh[1], bl[1]);
  mma_tf32(d, al, bh[0], bh[1]);
  mma_tf32(d, ah, bl[0], bl[1]);
  mma_tf32(d, ah, bh[0], bh[1]);
}

// The same with the left operand from 8 rows of x (a thread's two rows and two columns).
__device__ __forceinline__ void step_rows(float (&d)[4], const float* x, const float* row) {
  const float a[4] = {x[0], x[8], x[kLd], x[kLd + 8]};
  step_tf32(d, a, row);
}

__device__ __forceinline__ void store_neg(float* x, const float (&d)[4]) {
  x[0] = -d[0];
  x[kLd] = -d[1];
  x[8] = -d[2];
  x[kLd + 8] = -d[3];
}

// X = (I + L)^-1; only X[i][j], j <= i, is defined after it.  The blocks below
// the diagonal are -D' (C A'), made transposed, (A'^T C^T) D'^T: a 16 x 8
// accumulator tile is then an operand of the second product.  The 32 x 32
// product in brackets goes through the block above the diagonal, negated.
__device__ __forceinline__ void invert(const float* L, float* X) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp < 4 && lane < 16) {
    const float* Lb = L + warp * 16 * (kLd + 1);
    float* Xb = X + warp * 16 * (kLd + 1) + lane;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == lane ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 l = *reinterpret_cast<const float4*>(Lb + i * kLd + m);
        s = fmaf(-l.x, x[m], s);
        if (m + 1 < i) s = fmaf(-l.y, x[m + 1], s);
        if (m + 2 < i) s = fmaf(-l.z, x[m + 2], s);
        if (m + 3 < i) s = fmaf(-l.w, x[m + 3], s);
      }
      x[i] = s;
      Xb[i * kLd] = s;
    }
  }
  __syncthreads();
  const int g = lane >> 2, q2 = (lane & 3) * 2;
  if (warp < 4) {  // 16 x 16 blocks (1,0) and (3,2), half of the rows a warp
    const int n = warp & 1, c0 = (warp >> 1) * 32, r0 = c0 + 16;
    float m[2][4] = {}, d[4] = {};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        step_rows(m[t], X + (c0 + 8 * s + q2) * kLd + c0 + g, L + (r0 + 8 * t + g) * kLd + c0 + 8 * s + q2);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s > n) continue;  // D' is lower triangular
      const float a[4] = {m[s][0], m[s][2], m[s][1], m[s][3]};
      step_tf32(d, a, X + (r0 + 8 * n + g) * kLd + r0 + 8 * s + q2);
    }
    store_neg(X + (r0 + 8 * n + q2) * kLd + c0 + g, d);
  }
  __syncthreads();
  {  // the 32 x 32 block: 16 columns and 8 rows a warp
    const int c0 = (warp & 1) * 16, n = warp >> 1;
    float d[4] = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (8 * s < c0) continue;  // A' is lower triangular
      step_rows(d, X + (8 * s + q2) * kLd + c0 + g, L + (32 + 8 * n + g) * kLd + 8 * s + q2);
    }
    store_neg(X + (8 * n + q2) * kLd + 32 + c0 + g, d);
    __syncthreads();
    d[0] = d[1] = d[2] = d[3] = 0.f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s > n) continue;
      step_rows(d, X + (8 * s + q2) * kLd + 32 + c0 + g, X + (32 + 8 * n + g) * kLd + 32 + 8 * s + q2);
    }
    // minus the negated product
    float* x = X + (32 + 8 * n + q2) * kLd + c0 + g;
    x[0] = d[0];
    x[kLd] = d[1];
    x[8] = d[2];
    x[kLd + 8] = d[3];
    __syncthreads();
  }
}

template <int DT, int DK>
__global__ void __launch_bounds__(kThreads, DT == kF32 ? 2 : 4)
    gdr_prep_kernel(const GdrArgs a, uint8_t* qk_ws, uint8_t* pack_ws, int nc, bool vec) {
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
  float* X = reinterpret_cast<float*>(sm);  // once k and q are done with
  uint8_t* pack = sm + S::FIRST;
  float* vecs = reinterpret_cast<float*>(pack);
  float* slot = vecs + kVecHead;
  float* L = X + kC * kLd;
  uint8_t* th = reinterpret_cast<uint8_t*>(L);  // once the inverse is done
  uint8_t* tl = th + kMatBytes;
  uint8_t* ph = pack + kVecBytes;
  uint8_t* pl = ph + kMatBytes;
  float* kinv = reinterpret_cast<float*>(pl + kMatBytes);
  float* qinv = kinv + kC;
  float* ghi = qinv + kC;
  float* glo = ghi + kC;
  int* seg = reinterpret_cast<int*>(glo + kC);
  unsigned* pmax = reinterpret_cast<unsigned*>(seg + kC);
  unsigned* flag = pmax + kC;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, qd = lane & 3;
  const int wr = warp & 3, wc = warp >> 2;  // 16 rows and 32 columns of the 64 x 64 matrices
  // indices below 2^31 (checked on the host): 32-bit divisions
  const int64_t id = blockIdx.x;
  const unsigned uc = blockIdx.x % static_cast<unsigned>(nc), ubh = blockIdx.x / static_cast<unsigned>(nc);
  const unsigned uhk = ubh % static_cast<unsigned>(a.Hk), ub = ubh / static_cast<unsigned>(a.Hk);
  const int64_t c = uc, hk = uhk, b = ub;
  const int64_t t0 = c * kC;
  const int nt = static_cast<int>(a.L - t0 < kC ? a.L - t0 : kC);
  const int64_t rep = static_cast<unsigned>(a.Hv) / static_cast<unsigned>(a.Hk);

  // warp 0 has the gates: two tokens a lane
  float gv[2] = {0.f, 0.f}, bv[2] = {0.f, 0.f};
  int nw[2] = {0, 0};
  auto gates = [&](int64_t h) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t t = t0 + 2 * lane + j;
      gv[j] = t < a.L ? a.g[b * a.gs[0] + t * a.gs[1] + h * a.gs[2]] : 0.f;
      bv[j] = t < a.L ? F::to_f(static_cast<const E*>(a.beta)[b * a.bs[0] + t * a.bs[1] + h * a.bs[2]]) : 0.f;
    }
  };
  // Warp 0: the inclusive scan of the pair sums of g log2 e; G is kept as hi +
  // lo so that differences stay exact.  Then the next head's gates.
  auto decays = [&](int64_t h) {
    // A factor that far below FP32's range is zero (minus infinity's too; a select
    // keeps NaN).  64 of them come to 2^20, so that the second term of a sum
    // has room for what the other tokens add.
    auto low = [](float x) { return x < -kFarDecay ? -kFarDecay : x; };
    const float a0 = low(gv[0] * kLog2e), a1 = low(gv[1] * kLog2e);
    float hi = a0 + a1;
    const float bb = hi - a0;
    float lo = (a0 - (hi - bb)) + (a1 - bb);
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
    const float s = hi - a1, z = s - hi;
    const float2 gh = make_float2(s, hi), gl = make_float2(lo + ((hi - (s - z)) + (-a1 - z)), lo);
    const int2 sg = make_int2(sn - nw[1], sn);
    reinterpret_cast<float2*>(ghi)[lane] = gh;
    reinterpret_cast<float2*>(glo)[lane] = gl;
    reinterpret_cast<int2*>(seg)[lane] = sg;
    reinterpret_cast<float2*>(slot + kVGHi * kC)[lane] = gh;
    reinterpret_cast<float2*>(slot + kVGLo * kC)[lane] = gl;
    reinterpret_cast<int2*>(slot + kVSeg * kC)[lane] = sg;
    reinterpret_cast<float2*>(slot + kVBeta * kC)[lane] = make_float2(bv[0], bv[1]);
    if (h + 1 < (hk + 1) * rep) gates(h + 1);
  };
  if (warp == 0) {
    gates(hk * rep);
    if (a.seq != nullptr) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t t = t0 + 2 * lane + j;
        nw[j] = (t < a.L && t > 0 && a.seq[b * a.ss[0] + t * a.ss[1]] != a.seq[b * a.ss[0] + (t - 1) * a.ss[1]]) ? 1 : 0;
      }
    }
  }
  bool bad_qk = false;
  {
    RowLoad<DT, DK> lk, lq;
    lk.load(a.k, a.ks, b, hk, t0, nt, a.Dk, vec);
    if constexpr (DT != kF32) lq.load(a.q, a.qs, b, hk, t0, nt, a.Dk, vec);
    if (warp == 0) decays(hk * rep);  // the first head's, while k and q are on their way
    lk.store(k_hi, k_lo, kinv, bad_qk);
    if constexpr (DT == kF32) lq.load(a.q, a.qs, b, hk, t0, nt, a.Dk, vec);
    lq.store(q_hi, q_lo, qinv, bad_qk);
  }
  if (tid == 0) *flag = 0;
  fence_proxy_async_smem();
  __syncthreads();
  if (bad_qk) atomicOr(flag, 1u);
  if (tid == 0) {
    bulk_store(qk_ws + id * S::QK, sm, S::QK);
    bulk_commit();
  }

  // k k^T and q k^T, the column tiles up to the diagonal
  float kk[4][4], qq[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[i][j] = qq[i][j] = 0.f;
  const uint32_t kh = smem_u32(k_hi), kl = smem_u32(k_lo), qh = smem_u32(q_hi), ql = smem_u32(q_lo);
  if (wc * 2 <= wr) {
#pragma unroll
    for (int kt = 0; kt < DK / 16; ++kt) {
      uint32_t ak[4], aq[4], akl[4], aql[4];
      ldsm4(ak, addr_a<RB>(kh, wr * 16, 2 * kt, lane));
      ldsm4(aq, addr_a<RB>(qh, wr * 16, 2 * kt, lane));
      if constexpr (DT == kF32) {
        ldsm4(akl, addr_a<RB>(kl, wr * 16, 2 * kt, lane));
        ldsm4(aql, addr_a<RB>(ql, wr * 16, 2 * kt, lane));
      }
#pragma unroll
      for (int np = 0; np < 2; ++np) {
        if (wc * 2 + np > wr) continue;
        uint32_t bk[4];
        ldsm4(bk, addr_b<RB>(kh, wc * 32 + np * 16, 2 * kt, lane));
        mma(kk[2 * np], ak, bk[0], bk[1]);
        mma(kk[2 * np + 1], ak, bk[2], bk[3]);
        mma(qq[2 * np], aq, bk[0], bk[1]);
        mma(qq[2 * np + 1], aq, bk[2], bk[3]);
        if constexpr (DT == kF32) {
          mma(kk[2 * np], akl, bk[0], bk[1]);
          mma(kk[2 * np + 1], akl, bk[2], bk[3]);
          mma(qq[2 * np], aql, bk[0], bk[1]);
          mma(qq[2 * np + 1], aql, bk[2], bk[3]);
          ldsm4(bk, addr_b<RB>(kl, wc * 32 + np * 16, 2 * kt, lane));
          mma(kk[2 * np], ak, bk[0], bk[1]);
          mma(kk[2 * np + 1], ak, bk[2], bk[3]);
          mma(qq[2 * np], aq, bk[0], bk[1]);
          mma(qq[2 * np + 1], aq, bk[2], bk[3]);
        }
      }
    }
  }
  const int i0 = wr * 16 + g, i1 = i0 + 8;  // the rows of this thread
  {  // true values
    const float ki0 = kinv[i0], ki1 = kinv[i1], qi0 = qinv[i0], qi1 = qinv[i1];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float kj = kinv[wc * 32 + n * 8 + qd * 2 + (e & 1)];
        kk[n][e] *= (e < 2 ? ki0 : ki1) * kj;
        qq[n][e] *= (e < 2 ? qi0 : qi1) * kj;
      }
  }

  for (int64_t r = 0; r < rep; ++r) {
    const int64_t h = hk * rep + r;
    if (tid < kC) pmax[tid] = 0;
    if (tid == 0) bulk_wait_read();  // the tiles and the package are free again
    if (warp == 0 && r > 0) decays(h);
    __syncthreads();

    if (wc == 1 && wr < 2) {  // these two warps have no tile below the diagonal: the tokens' factors
      const int i = wr * 32 + lane;
      const float gh = ghi[i], gl = glo[i], bv = slot[kVBeta * kC + i];
      const float gi = seg[i] == 0 ? exp2f(gh + gl) : 0.f;
      const float gc = seg[i] == seg[kC - 1] ? exp2f((ghi[kC - 1] - gh) + (glo[kC - 1] - gl)) : 0.f;
      const float ki = kinv[i], qi = qinv[i];
      const float cks = gi * ki, cqs = a.scale * gi * qi, cu = gc * ki;
      slot[kVKS * kC + i] = cks;
      slot[kVQS * kC + i] = cqs;
      slot[kVU * kC + i] = cu;
      slot[kVGi * kC + i] = gi;
      slot[kVGc * kC + i] = gc;
      slot[kVKInv * kC + i] = ki;
      slot[kVQInv * kC + i] = qi;
      if (i == kC - 1) vecs[kHdGa] = gi;
      // growing decays: the combined factors must be finite too
      if (mag(bv) >= kInfBits || mag(gi) >= kInfBits || mag(gc) >= kInfBits || mag(cks) >= kInfBits ||
          mag(cqs) >= kInfBits || mag(cu) >= kInfBits)
        atomicOr(flag, 2u);
    }

    // Gam; L into shared memory; P
    float p[4][4];
    {
      const float gh0 = ghi[i0], gl0 = glo[i0], gh1 = ghi[i1], gl1 = glo[i1];
      const int s0 = seg[i0], s1 = seg[i1];
      const float b0 = slot[kVBeta * kC + i0], b1 = slot[kVBeta * kC + i1];
      float m0 = 0.f, m1 = 0.f;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) p[n][e] = 0.f;
        if (wc * 32 + n * 8 > wr * 16 + 15) continue;
        const int j0 = wc * 32 + n * 8 + qd * 2;
        const float2 gj = *reinterpret_cast<const float2*>(ghi + j0), lj = *reinterpret_cast<const float2*>(glo + j0);
        const int2 sj = *reinterpret_cast<const int2*>(seg + j0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + (e & 1), i = e < 2 ? i0 : i1;
          const bool in = j <= i && ((e & 1) ? sj.y : sj.x) == (e < 2 ? s0 : s1);
          const float gam = exp2f(((e < 2 ? gh0 : gh1) - ((e & 1) ? gj.y : gj.x)) +
                                       ((e < 2 ? gl0 : gl1) - ((e & 1) ? lj.y : lj.x)));
          // selected, not multiplied: nothing crosses the diagonal or a new sequence
          p[n][e] = in ? gam * qq[n][e] : 0.f;
          if (j < i) L[i * kLd + j] = in ? (e < 2 ? b0 : b1) * gam * kk[n][e] : 0.f;
        }
        m0 = amax3(m0, p[n][0], p[n][1]);
        m1 = amax3(m1, p[n][2], p[n][3]);
      }
      const unsigned u0 = quad_max(__float_as_uint(m0)), u1 = quad_max(__float_as_uint(m1));
      if (qd == 0) {
        atomicMax(&pmax[i0], u0);
        atomicMax(&pmax[i1], u1);
      }
    }
    __syncthreads();
    {
      const unsigned u0 = pmax[i0], u1 = pmax[i1];
      if (u0 >= kInfBits || u1 >= kInfBits) atomicOr(flag, 2u);
      float f0, f1, v0, v1;
      row_factor(u0, f0, v0);
      row_factor(u1, f1, v1);
      if (qd == 0 && wc == 0) {
        slot[kVP * kC + i0] = a.scale * v0;
        slot[kVP * kC + i1] = a.scale * v1;
        slot[kVPInv * kC + i0] = v0;
        slot[kVPInv * kC + i1] = v1;
      }
      const uint64_t w0 = pk(f0, f0), w1 = pk(f1, f1);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t hi, lo;
        split2f(p[n][0], p[n][1], w0, hi, lo);
        uint32_t off = tile_off<128>(i0, wc * 4 + n) + qd * 4;
        *reinterpret_cast<uint32_t*>(ph + off) = hi;
        *reinterpret_cast<uint32_t*>(pl + off) = lo;
        split2f(p[n][2], p[n][3], w1, hi, lo);
        off = tile_off<128>(i1, wc * 4 + n) + qd * 4;
        *reinterpret_cast<uint32_t*>(ph + off) = hi;
        *reinterpret_cast<uint32_t*>(pl + off) = lo;
      }
    }
    invert(L, X);
    // T's rows scaled and split: eight rows a warp, two at a time, four columns a lane
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = warp * 8 + i * 2 + (lane >> 4), col = (lane & 15) * 4;
      const float4 y = *reinterpret_cast<const float4*>(X + row * kLd + col);
      float x[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j > row) x[j] = 0.f;
      unsigned m = __float_as_uint(amax3(amax3(0.f, x[0], x[1]), x[2], x[3]));
#pragma unroll
      for (int k = 1; k < 16; k <<= 1) m = max(m, __shfl_xor_sync(kFullMask, m, k));
      if (m >= kInfBits) atomicOr(flag, 2u);
      float f, v;
      row_factor(m, f, v);
      if ((lane & 15) == 0) slot[kVTInv * kC + row] = v;
      const uint64_t w = pk(f, f);
      uint2 hi, lo;
      split2f(x[0], x[1], w, hi.x, lo.x);
      split2f(x[2], x[3], w, hi.y, lo.y);
      const uint32_t off = tile_off<128>(row, (lane & 15) >> 1) + (lane & 1) * 8;
      *reinterpret_cast<uint2*>(th + off) = hi;
      *reinterpret_cast<uint2*>(tl + off) = lo;
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      vecs[kHdBad] = *flag ? 1.f : 0.f;
      *flag &= 1u;  // k and q are shared by the next head, its own factors are not
      fence_proxy_async_smem();
      uint8_t* dst = pack_ws + ((b * a.Hv + h) * nc + c) * kPackBytes;
      bulk_store(dst, pack, kVecBytes);
      bulk_store(dst + kVecBytes, th, 2 * kMatBytes);
      bulk_store(dst + kOffP, ph, 2 * kMatBytes);
      bulk_commit();
    }
  }
  if (tid == 0) bulk_wait_all();
}

template <int DT, int DK>
cudaError_t launch(const GdrArgs& a, uint8_t* qk_ws, uint8_t* pack_ws, int nc, cudaStream_t s) {
  constexpr int64_t V = Fmt<DT>::VEC;
  auto ok = [&](const void* p, const int64_t* st) {
    return st[3] == 1 && a.Dk == DK && reinterpret_cast<uintptr_t>(p) % 16 == 0 && st[0] % V == 0 && st[1] % V == 0 &&
           st[2] % V == 0;
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

cudaError_t launch_gdr_prep(const GdrArgs& a, Dtype dt, uint8_t* qk_ws, uint8_t* pack_ws, int nc,
                            cudaStream_t s) {
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, qk_ws, pack_ws, nc, s);
    case kF16: return launch_dt<kF16>(a, qk_ws, pack_ws, nc, s);
    case kBF16: return launch_dt<kBF16>(a, qk_ws, pack_ws, nc, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ccv

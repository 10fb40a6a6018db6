// Shared by the chunked kernels of the gated delta rule.
//
// A sequence is cut into chunks of C = 64 tokens.  With G_i the cumulative
// log decay inside the chunk, Gam_ij = exp(G_i - G_j) for j <= i (0 where a
// new sequence begins between them), S0 the state before the chunk:
//
//   L_ij = beta_i Gam_ij k_i.k_j (j < i),   T = (I + L)^-1,   P_ij = Gam_ij q_i.k_j (j <= i)
//   E = V - gi (K S0),   U = T (beta E),   O = scale (gi (Q S0) + P U),   S1 = ga S0 + K^T (gc U)
//
// with gi_i = exp(G_i), gc_i = exp(G_last - G_i), ga = exp(G_last) (0 across a
// new sequence).  One kernel (gdr_prep.cu) makes what does not depend on the
// state, for all chunks at once; another (gdr_scan.cu) carries the state.
//
// Precision.  The state and all sums are FP32.  The products run on FP16
// tensor instructions with FP32 accumulation; an FP32 operand x enters as two
// FP16 numbers, hi = fp16(s x) and lo = fp16(s x - hi), where s is the power
// of two that brings the largest magnitude of x's row (the index that is not
// summed over) to [2^14, 2^15).  hi + lo holds 22 bits of the row's largest
// element, and 2^28 below it still 11 bits.  16-bit inputs are exact in hi,
// so a product with q or k takes two instructions (hi and lo of the other
// factor), a product of two FP32 operands three (lo lo is below 2^-22).  The
// row factors are powers of two and are taken out exactly in FP32.
#pragma once

#include <type_traits>

#include "ccv_common.cuh"
#include "ccv_tma.cuh"
#include "mix_internal.h"

namespace ccv {

constexpr int kC = kGdrChunk;

// Per-chunk factors in FP32: a head of kVecHead floats, then arrays of 64.
constexpr int kVecHead = 16;
enum VecHead { kHdGa = 0, kHdBad = 1 };
enum VecSlot {
  kVKS = 0,     // gi / k's factor: true gi (K S0) from the scaled product
  kVQS = 1,     // scale gi / q's factor
  kVP = 2,      // scale / P's row factor
  kVBeta = 3,
  kVTInv = 4,   // 1 / T's row factor
  kVU = 5,      // gc / k's factor
  kVGi = 6,     // the remaining slots serve the backward pass
  kVGc = 7,
  kVKInv = 8,   // 1 / k's row factor
  kVQInv = 9,
  kVPInv = 10,
  kVGHi = 11,   // G in units of log 2, as a sum of two floats
  kVGLo = 12,
  kVSeg = 13,   // number of sequence starts in the chunk up to the token (as an integer)
  kVSlots = 14
};
constexpr int kVecBytes = 4096;
constexpr int kVecFwdBytes = (kVecHead + 6 * kC) * 4;  // what the forward scan reads
static_assert((kVecHead + kVSlots * kC) * 4 <= kVecBytes, "vector part");
constexpr int kMatBytes = kC * kC * 2;                     // one FP16 64 x 64 matrix
constexpr int kOffP = kVecBytes + 2 * kMatBytes;
constexpr int kPackBytes = kOffP + 2 * kMatBytes;          // factors, T hi, T lo, P hi, P lo

// Bytes of the [64, DK] FP16 tiles of k and q of one chunk and key head
// (hi, and lo for FP32 inputs): k hi, (k lo,) q hi, (q lo).
__host__ __device__ constexpr int qk_tile_bytes(int DK) { return kC * DK * 2; }
__host__ __device__ constexpr int qk_pack_bytes(int DK, int terms) { return 2 * terms * qk_tile_bytes(DK); }

// What the backward pass keeps of a chunk, per group ("slice") of 16 value
// channels, as FP16 tiles ready for matrix loads: the state before the chunk
// and U from the forward scan, D, dR and dO from the reverse scan, each row of
// a value channel scaled by its power of two and split in hi and lo (dO of
// 16-bit inputs is exact in hi).  S and D: blocks of 32 key channels, [16 v][32
// k]; U, dR, dO: [64 tokens][16 v].  The inverse row factors follow; S and D
// have one for each half of the key channels (a scan with two warps a slice
// has two).
constexpr int kSliceV = 16;
constexpr int kBlkBytes = kSliceV * 32 * 2;
constexpr int kTokBytes = kC * kSliceV * 2;
__host__ __device__ constexpr int img_state_bytes(int DK) { return DK / 32 * kBlkBytes; }  // hi, or lo
struct ImgF {  // S hi, S lo, U hi, U lo, 1/factors of S [2][16], of U [16]
  static __host__ __device__ constexpr int u(int DK) { return 2 * img_state_bytes(DK); }
  static __host__ __device__ constexpr int inv(int DK) { return u(DK) + 2 * kTokBytes; }
  static __host__ __device__ constexpr int bytes(int DK) { return inv(DK) + 256; }
};
struct ImgB {  // D hi, D lo, dR hi, dR lo, dO hi, (dO lo,) 1/factors of D [2][16], dR, dO, then dR.v of 64 tokens
  static __host__ __device__ constexpr int r(int DK) { return 2 * img_state_bytes(DK); }
  static __host__ __device__ constexpr int o(int DK) { return r(DK) + 2 * kTokBytes; }
  static __host__ __device__ constexpr int inv(int DK, int terms) { return o(DK) + terms * kTokBytes; }
  static __host__ __device__ constexpr int bytes(int DK, int terms) { return inv(DK, terms) + 512; }
};
// Rows of 64 and 32 bytes whose 16-byte pieces are placed so that eight rows
// at one piece lie in different banks.
__device__ __forceinline__ uint32_t off64(int row, int piece) {
  return static_cast<uint32_t>(row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
}
__device__ __forceinline__ uint32_t off32(int row, int piece) {
  return static_cast<uint32_t>(row * 32 + ((piece ^ ((row >> 2) & 1)) << 4));
}

// Tiles are rows of RB bytes in 16-byte pieces; piece p of row r lies at
// p ^ (r & 7), so the eight rows of a matrix load touch all banks.
template <int RB>
__device__ __forceinline__ uint32_t tile_off(int row, int piece) {
  return static_cast<uint32_t>(row * RB + ((piece ^ (row & 7)) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

__device__ __forceinline__ void stsm4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

// B operand of two column tiles (n0, n0 + 8) and 16 summed indices: rows of
// the tile are columns of B (summed index along the row).
template <int RB>
__device__ __forceinline__ uint32_t addr_b(uint32_t tile, int n0, int piece, int lane) {
  return tile + tile_off<RB>(n0 + (lane & 7) + ((lane >> 4) & 1) * 8, piece + ((lane >> 3) & 1));
}

// The same where rows of the tile are the summed index (transposed load).
template <int RB>
__device__ __forceinline__ uint32_t addr_bt(uint32_t tile, int k0, int piece, int lane) {
  return tile + tile_off<RB>(k0 + (lane & 7) + ((lane >> 3) & 1) * 8, piece + (lane >> 4));
}

// A operand: 16 rows of the tile from r0, 16 summed indices along the row.
template <int RB>
__device__ __forceinline__ uint32_t addr_a(uint32_t tile, int r0, int piece, int lane) {
  return tile + tile_off<RB>(r0 + (lane & 7) + ((lane >> 3) & 1) * 8, piece + (lane >> 4));
}

// A operand where rows of the tile are the summed index (transposed load):
// 16 columns from piece's first, 16 rows from k0.
template <int RB>
__device__ __forceinline__ uint32_t addr_at(uint32_t tile, int k0, int piece, int lane) {
  return tile + tile_off<RB>(k0 + (lane & 7) + ((lane >> 4) & 1) * 8, piece + ((lane >> 3) & 1));
}

// d += a b for 16 x 8 x 16, FP16 operands, FP32 sums.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// hi = fp16(x, y), lo = fp16(x - hi, y - hi).
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = h2(x - f.x, y - f.y);
}

// The same of (x, y) times f, packed arithmetic.
__device__ __forceinline__ void split2f(float x, float y, uint64_t f, uint32_t& hi, uint32_t& lo) {
  const uint64_t v = fmul2(pk(x, y), f);
  float a, b;
  upk(v, a, b);
  const __half2 h = __floats2half2_rn(a, b);
  const float2 e = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  upk(ffma2(pk(e.x, e.y), pk(-1.f, -1.f), v), a, b);
  lo = h2(a, b);
}

// Elements 0, 1 (row g) or 2, 3 (row g + 8) of an accumulator tile as a pair.
__device__ __forceinline__ uint64_t pair_of(const float (&x)[4], int row) { return pk(x[2 * row], x[2 * row + 1]); }
__device__ __forceinline__ void set_pair(float (&x)[4], int row, uint64_t v) { upk(v, x[2 * row], x[2 * row + 1]); }
__device__ __forceinline__ uint64_t both(float x) { return pk(x, x); }
__device__ __forceinline__ uint64_t ld_pair(const float* p) {
  const float2 x = *reinterpret_cast<const float2*>(p);
  return pk(x.x, x.y);
}

// max(m, |x|, |y|), NaN where one of them is.
__device__ __forceinline__ float amax3(float m, float x, float y) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(x), "f"(y));
  return d;
}

__device__ __forceinline__ unsigned mag(float x) { return __float_as_uint(x) & 0x7fffffffu; }

constexpr unsigned kInfBits = 0x7f800000u;  // magnitudes from here on are not finite

// Power of two that brings a finite magnitude to [2^14, 2^15), and its inverse
// (2^126 and 2^-126 where the magnitude is zero or smaller than any product needs).
__device__ __forceinline__ void row_factor(unsigned m, float& f, float& inv) {
  const unsigned e = max(15u, min(254u, m >> 23));
  f = __uint_as_float((268u - e) << 23);
  inv = __uint_as_float((e - 14u) << 23);
}

__device__ __forceinline__ unsigned quad_max(unsigned m) {
  m = max(m, __shfl_xor_sync(kFullMask, m, 1));
  return max(m, __shfl_xor_sync(kFullMask, m, 2));
}

__device__ __forceinline__ unsigned warp_max(unsigned m) {
  return __reduce_max_sync(kFullMask, m);
}

// What the backward pass keeps of a chunk with values that are not finite: each
// row is scaled by the largest of its finite ones, so that these stay what they
// are and only sums that the others enter are lost.  That largest of rows g and g + 8:
template <int NT>
__device__ __forceinline__ void finite_max(const float (&x)[NT][4], unsigned& m0, unsigned& m1) {
  unsigned m[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned u = mag(x[i][j]);
      m[j >> 1] = max(m[j >> 1], u < kInfBits ? u : 0u);
    }
  m0 = quad_max(m[0]);
  m1 = quad_max(m[1]);
}

// 16 x 64 accumulator fragments (8 column tiles) as A operands of the next
// product: each row scaled by its factor and split.  Returns the inverse
// factors of rows g and g + 8; `bad` is set where a value is not finite.
// KEPT: by their finite values (finite_max).
template <int NT, bool LO, bool KEPT = false>
__device__ __forceinline__ void split_rows(const float (&x)[NT][4], uint32_t (&hi)[NT / 2][4],
                                           uint32_t (&lo)[NT / 2][4], float& inv0, float& inv1, bool& bad) {
  float a0 = 0.f, a1 = 0.f;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    a0 = amax3(a0, x[i][0], x[i][1]);
    a1 = amax3(a1, x[i][2], x[i][3]);
  }
  unsigned m0 = quad_max(__float_as_uint(a0)), m1 = quad_max(__float_as_uint(a1));
  bad = bad || m0 >= kInfBits || m1 >= kInfBits;
  if constexpr (KEPT) finite_max(x, m0, m1);
  float f0, f1;
  row_factor(m0, f0, inv0);
  row_factor(m1, f1, inv1);
  const uint64_t p0 = pk(f0, f0), p1 = pk(f1, f1);
#pragma unroll
  for (int i = 0; i < NT / 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (LO) {
        split2f(x[2 * i + j][0], x[2 * i + j][1], p0, hi[i][2 * j], lo[i][2 * j]);
        split2f(x[2 * i + j][2], x[2 * i + j][3], p1, hi[i][2 * j + 1], lo[i][2 * j + 1]);
      } else {
        hi[i][2 * j] = h2(x[2 * i + j][0] * f0, x[2 * i + j][1] * f0);
        hi[i][2 * j + 1] = h2(x[2 * i + j][2] * f1, x[2 * i + j][3] * f1);
      }
    }
}

// A warp's rows of S^T or D^T as kept for the backward pass, in a chunk with
// values that are not finite: hi to `tile`, lo behind it by `lo_at`.
template <int NK>
__device__ __noinline__ void keep_state(const float (&x)[NK][4], uint32_t tile, uint32_t lo_at, int lane, float& inv0,
                                        float& inv1) {
  uint32_t hi[NK / 2][4], lo[NK / 2][4];
  bool ignore = false;
  split_rows<NK, true, true>(x, hi, lo, inv0, inv1, ignore);
#pragma unroll
  for (int kt = 0; kt < NK / 2; ++kt) {
    const uint32_t at = tile + (kt >> 1) * kBlkBytes + off64((lane & 7) + ((lane >> 3) & 1) * 8, (kt & 1) * 2 + (lane >> 4));
    stsm4(at, hi[kt]);
    stsm4(at + lo_at, lo[kt]);
  }
}

// The inverse factor of a row that overflowed although nothing that enters it
// is infinite: the gradients that it enters become NaN.
constexpr unsigned kLostBits = kInfBits;

// Barriers of one pair of warps (id from 1).
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, 64, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool in) {
  // a false predicate copies nothing and fills the piece with zeros
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

}  // namespace ccv

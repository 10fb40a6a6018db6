// Tiles of the recurrence's sequence kernels: 64 tokens x 64 channels, cut
// into the warps' runs of tokens; a lane owns two adjacent channels.
//
// A run of tokens maps the state h before it to A h + H; a run that holds a
// sequence's start gives H whatever h is, which A's sign bit marks (decays are
// not negative), so that an infinite state does not cross it as 0 * inf.
//
// Carrying the state from tile to tile.  Tiles are taken from a counter in
// the order of time, so the tiles before a taken one belong to blocks that
// already run, and a block works its tiles off in that order: the earliest
// unfinished tile never waits.  A tile has a slot of 16 bytes for each lane,
// empty at first; it gets the tile's (A, H), and then the state after it, which
// is DEFINED as A h + H for the state h before it.  Whoever needs a state folds
// the pairs from the last state on, so the chain of operations is the same
// wherever that fold starts, and results do not depend on timing.  A slot is
// read and written whole (128-bit relaxed accesses), so nothing needs a fence:
// with flags beside the values, released and acquired, 8192 tokens x 5120
// channels took 327 us instead of 99 (and 83 with what came after).
#pragma once

#include <cuda.h>

#include "ccv_tma.cuh"
#include "glr.cuh"
#include "rec_pairs.cuh"
#include "tensor_map.h"
#include "tma_store.cuh"

namespace ccv {

constexpr int kGlrT = kGlrChunk;  // tokens of a tile
constexpr int kGlrC = 64;         // channels of a tile
static_assert(kGlrT == 64 && kGlrC == 64, "reset masks are two words, a lane has two channels");

// Few tiles along the time: a block carries the state itself, with no memset and
// no slots.  1024 channels in bf16, forward (backward): 128 tokens 5.8 us against
// 10.2 (14.1 against 19.5), 256 tokens 8.2 against 11.2 (14.6 against 18.9), 512
// tokens 14.4 against 9.6 (23.6 against 17.2).
constexpr int kGlrSerial = 4;

// Workspace of the chain: ticket and slots [tile][lane]; all bits set before
// the launch.
struct GlrChain {
  unsigned* ticket;
  uint4* slots;
};

inline uint64_t glr_chain_bytes(uint64_t tiles) { return 256 + tiles * 512; }
inline GlrChain glr_chain(void* ws) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  return {reinterpret_cast<unsigned*>(p), reinterpret_cast<uint4*>(p + 256)};
}

// A tile's place, found once by the thread that starts its copies.
struct GlrPlace {
  int tile, level, col, b, c0;
};

// What the tile kernels get beside their arguments: sizes in 32 bits.
struct GlrTiles {
  int ncols;   // columns: batch rows x channel tiles
  int nct;     // channel tiles of a row
  uint64_t ncols_inv, nct_inv;  // 2^63 / n rounded up, for t / n of 0 <= t < 2^31
  int levels;  // tiles along the time
  int total;   // ncols * levels
  bool pair;   // outputs may be stored in pairs
  bool one;    // a block for every tile: a block takes one
  bool serial; // a block takes the tiles of a column in turn: no chain
};

// Tiles in the order of a block's work without a chain: its columns one after
// the other, each from the first tile on.
__device__ __forceinline__ int glr_serial_tile(const GlrTiles& g, int k) {
  const int64_t col = blockIdx.x + static_cast<int64_t>(k / g.levels) * gridDim.x;
  return col < g.ncols ? k % g.levels * g.ncols + static_cast<int>(col) : g.total;
}

// t / n, exact: the rounding adds less than t / 2^63 to a quotient whose fraction is at most 1 - 1 / n.
__device__ __forceinline__ int glr_div(int t, uint64_t inv) {
  return static_cast<int>(__umul64hi(static_cast<uint64_t>(t) << 1, inv));
}

constexpr float kMinusZero = -0.0f;
__device__ __forceinline__ bool glr_cut(float A) { return __float_as_uint(A) == 0x80000000u; }
__device__ __forceinline__ float glr_map(float A, float H, float h) { return glr_cut(A) ? H : fmaf(A, h, H); }
// (A, H) after (A0, H0)
__device__ __forceinline__ void glr_join(float A, float H, float& A0, float& H0) {
  H0 = glr_map(A, H, H0);
  A0 = glr_cut(A) || glr_cut(A0) ? kMinusZero : __fmul_rn(A, A0);
}
// Maps of a run of tokens for two channels, from the product A of its decays (start: a sequence starts in it).  The mark of
// a start is no factor of A: a later decay that is NaN would replace it.
__device__ __forceinline__ float4 glr_run(uint64_t A, uint64_t H, bool start) {
  float a, b, u, v;
  upk(A, a, b), upk(H, u, v);
  return start ? make_float4(kMinusZero, u, kMinusZero, v) : make_float4(glr_positive(a), u, glr_positive(b), v);
}

// A slot's first word: empty, or a state (in the second and fourth word), or
// the decay of a pair.  (Both are NaNs with a sign; a decay that is one is
// stored without it.)
constexpr unsigned kSlotEmpty = 0xffffffffu, kSlotState = 0xfffffffeu;

__device__ __forceinline__ uint4 ld_slot(const uint4* p) {
  uint64_t lo, hi;
  asm volatile(
      "{\n\t.reg .b128 v;\n\tld.relaxed.gpu.global.b128 v, [%2];\n\tmov.b128 {%0, %1}, v;\n\t}"
      : "=l"(lo), "=l"(hi)
      : "l"(p)
      : "memory");
  return make_uint4(static_cast<unsigned>(lo), static_cast<unsigned>(lo >> 32), static_cast<unsigned>(hi),
                    static_cast<unsigned>(hi >> 32));
}
__device__ __forceinline__ void st_slot(uint4* p, uint4 v) {
  const uint64_t lo = v.x | static_cast<uint64_t>(v.y) << 32, hi = v.z | static_cast<uint64_t>(v.w) << 32;
  asm volatile("{\n\t.reg .b128 v;\n\tmov.b128 v, {%1, %2};\n\tst.relaxed.gpu.global.b128 [%0], v;\n\t}" ::"l"(p),
               "l"(lo), "l"(hi)
               : "memory");
}
__device__ __forceinline__ uint4* glr_slot(const GlrChain& c, int tile, int lane) {
  return c.slots + static_cast<int64_t>(tile) * 32 + lane;
}
__device__ __forceinline__ void glr_put_pair(const GlrChain& c, int tile, int lane, float4 m) {
  const unsigned a = __float_as_uint(m.x);
  st_slot(glr_slot(c, tile, lane), make_uint4(a >= kSlotState ? 0x7fffffffu : a, __float_as_uint(m.y),
                                              __float_as_uint(m.z), __float_as_uint(m.w)));
}
__device__ __forceinline__ void glr_put_state(const GlrChain& c, int tile, int lane, float2 h) {
  st_slot(glr_slot(c, tile, lane), make_uint4(kSlotState, __float_as_uint(h.x), 0u, __float_as_uint(h.y)));
}
__device__ __forceinline__ float2 glr_slot_state(const uint4& v) {
  return make_float2(__uint_as_float(v.y), __uint_as_float(v.w));
}
__device__ __forceinline__ float2 glr_slot_map(const uint4& v, float2 h) {
  if (v.x == kSlotState) return glr_slot_state(v);
  return make_float2(glr_map(__uint_as_float(v.x), __uint_as_float(v.y), h.x),
                     glr_map(__uint_as_float(v.z), __uint_as_float(v.w), h.y));
}

// The state before the tile of this level (> 0) and column, two channels a
// lane: from the nearest state among the kWindow tiles before it, through the
// pairs that follow it.  One warp.  False when the wait ran out.
// Older slots are never behind: where one holds a state, those before it do.
constexpr int kWindow = 8;
__device__ __forceinline__ bool glr_look_back(const GlrChain& c, const GlrTiles& g, int level, int col, int lane,
                                              float2& h) {
  const long long start = clock64();
  const uint4* slot = glr_slot(c, (level - 1) * g.ncols + col, lane);
  const int64_t step = static_cast<int64_t>(g.ncols) * 32;
  for (;;) {
    uint4 v[kWindow];
    int n = -1, k = 0;  // n: where the whole warp found states; k: slots that are not empty
    v[0] = ld_slot(slot);
    if (__all_sync(kFullMask, v[0].x == kSlotState)) {
      h = glr_slot_state(v[0]);
      return true;
    }
    if (__all_sync(kFullMask, v[0].x != kSlotEmpty)) {
      k = 1;
#pragma unroll
      for (int i = 1; i < kWindow; i += 4) {
        if (k != i || n >= 0) break;
#pragma unroll
        for (int j = i; j < i + 4 && j < kWindow; ++j)
          v[j] = j < level ? ld_slot(slot - j * step) : make_uint4(kSlotEmpty, 0u, 0u, 0u);
#pragma unroll
        for (int j = i; j < i + 4 && j < kWindow; ++j)
          if (k == j && n < 0) {
            if (__all_sync(kFullMask, v[j].x == kSlotState)) n = j;
            if (__all_sync(kFullMask, v[j].x != kSlotEmpty)) k = j + 1;
          }
      }
      if (n > 0) {
#pragma unroll
        for (int i = kWindow - 1; i >= 0; --i) {
          if (i == n) h = glr_slot_state(v[i]);
          if (i < n) h = glr_slot_map(v[i], h);
        }
        return true;
      }
    }
    if (clock64() - start > kWaitBudgetCycles) return false;
    __nanosleep(40);
  }
}

// Host side (glr_fwd.cu): sizes, outputs in pairs.
GlrTiles glr_tiles(int64_t B, int64_t L, int64_t C);
bool glr_pair_out(const void* p, const int64_t* s, Dtype dt);

// A chained kernel follows the memset of its flags: a plain launch.
template <typename... P, typename... A>
cudaError_t glr_launch(void (*kernel)(P...), const GlrTiles& g, unsigned grid, unsigned threads, size_t smem,
                       cudaStream_t stream, A&&... args) {
  if (g.levels <= kGlrSerial) return launch_pdl(kernel, grid, threads, smem, stream, std::forward<A>(args)...);
  kernel<<<grid, threads, smem, stream>>>(std::forward<A>(args)...);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- pairs of channels

// Two adjacent channels of a staged row (rows of 64 elements).
template <int DT>
__device__ __forceinline__ uint64_t glr_lds(const uint8_t* base, int row, int lane) {
  if constexpr (DT == kF32) {
    const float2 v = *reinterpret_cast<const float2*>(base + row * (kGlrC * 4) + lane * 8);
    return pk(v.x, v.y);
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(base + row * (kGlrC * 2) + lane * 4);
    return pk(Fmt<DT>::word_elem(w, 0), Fmt<DT>::word_elem(w, 1));
  }
}

template <int DT>
__device__ __forceinline__ void glr_sts(uint8_t* base, int row, int lane, uint64_t v) {
  float a, b;
  upk(v, a, b);
  if constexpr (DT == kF32) {
    *reinterpret_cast<float2*>(base + row * (kGlrC * 4) + lane * 8) = make_float2(a, b);
  } else {
    *reinterpret_cast<uint32_t*>(base + row * (kGlrC * 2) + lane * 4) = Fmt<DT>::pack2(a, b);
  }
}

// Two channels of an any-stride tensor at p (`in0`, `in1`: they exist).
template <int DT>
__device__ __forceinline__ uint64_t glr_ldg(const void* p, int64_t off, int64_t cs, bool in0, bool in1) {
  const typename Fmt<DT>::E* e = static_cast<const typename Fmt<DT>::E*>(p) + off;
  return pk(in0 ? Fmt<DT>::to_f(e[0]) : 0.f, in1 ? Fmt<DT>::to_f(e[cs]) : 0.f);
}

template <int DT>
__device__ __forceinline__ void glr_stg(typename Fmt<DT>::E* e, int64_t cs, bool pair, bool in0, bool in1, uint64_t v) {
  float a, b;
  upk(v, a, b);
  if (pair) {
    if constexpr (DT == kF32) {
      __stcs(reinterpret_cast<float2*>(e), make_float2(a, b));
    } else {
      __stcs(reinterpret_cast<unsigned*>(e), Fmt<DT>::pack2(a, b));
    }
  } else {
    if (in0) e[0] = Fmt<DT>::from_f(a);
    if (in1) e[cs] = Fmt<DT>::from_f(b);
  }
}

// Sigmoids of a pair: s, and e = 2^(-z log2 e) as it was taken.
__device__ __forceinline__ void glr_sigmoid2(uint64_t z, uint64_t& s, uint64_t& e) {
  float a, b;
  upk(fmul2(z, twice(-kLog2e)), a, b);
  e = pk(ex2_approx(a), ex2_approx(b));
  upk(fadd2(e, twice(1.f)), a, b);
  s = pk(rcp_approx(a), rcp_approx(b));
}

// a and 1 - a^2 of a pair of logarithms, as glr_decay (NEAR: neither is below
// kGlrSeries).
template <bool NEAR>
__device__ __forceinline__ void glr_decay2(uint64_t l, uint64_t& a, uint64_t& m2) {
  uint64_t E = twice(glr_poly(0));
#pragma unroll
  for (int i = 1; i < 7; ++i) E = ffma2(E, l, twice(glr_poly(i)));
  E = fmul2(E, l);
  a = fadd2(E, twice(1.f));
  if constexpr (!NEAR) {
    float f0, f1, n0, n1, l0, l1, e0, e1;
    upk(l, l0, l1);
    f0 = glr_positive(ex2_approx(__fmul_rn(l0, kLog2e))), f1 = glr_positive(ex2_approx(__fmul_rn(l1, kLog2e)));
    upk(a, n0, n1);
    upk(E, e0, e1);
    const bool c0 = l0 >= kGlrSeries, c1 = l1 >= kGlrSeries;
    a = pk(c0 ? n0 : f0, c1 ? n1 : f1);
    E = pk(c0 ? e0 : __fadd_rn(f0, -1.f), c1 ? e1 : __fadd_rn(f1, -1.f));
  }
  m2 = fmul2(E, ffma2(E, twice(-1.f), twice(-2.f)));
}

}  // namespace ccv

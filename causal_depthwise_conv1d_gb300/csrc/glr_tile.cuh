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
// unfinished tile never waits.  Each tile first publishes its (A, H); the state
// after it is then DEFINED as A h + H for the state h before it, and whoever
// needs a state folds the published pairs from the last published state on.
// The chain of operations is the same wherever that fold starts, so results
// do not depend on timing.
#pragma once

#include <cuda.h>

#include "ccv_tma.cuh"
#include "glr.cuh"

namespace ccv {

constexpr int kGlrT = kGlrChunk;  // tokens of a tile
constexpr int kGlrC = 64;         // channels of a tile
static_assert(kGlrT == 64 && kGlrC == 64, "reset masks are two words, a lane has two channels");

// Workspace of the chain: ticket, flags, pairs and states, [tile][lane].
struct GlrChain {
  unsigned* ticket;
  unsigned* flags;
  float4* pairs;
  float2* states;
};

__host__ __device__ inline uint64_t glr_flag_bytes(uint64_t tiles) { return (256 + tiles * 4 + 255) / 256 * 256; }
inline uint64_t glr_chain_bytes(uint64_t tiles) { return glr_flag_bytes(tiles) + tiles * (512 + 256); }
inline GlrChain glr_chain(void* ws, uint64_t tiles) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  const uint64_t f = glr_flag_bytes(tiles);
  return {reinterpret_cast<unsigned*>(p), reinterpret_cast<unsigned*>(p + 256), reinterpret_cast<float4*>(p + f),
          reinterpret_cast<float2*>(p + f + tiles * 512)};
}

// What the tile kernels get beside their arguments: sizes in 32 bits.
struct GlrTiles {
  int ncols;   // columns: batch rows x channel tiles
  int nct;     // channel tiles of a row
  int levels;  // tiles along the time
  int total;   // ncols * levels
  bool tma;    // tensor copies of the inputs (else loads of single elements)
  bool pair;   // outputs may be stored in pairs
  bool one;    // a block for every tile: a block takes one
};

constexpr float kMinusZero = -0.0f;
__device__ __forceinline__ bool glr_cut(float A) { return __float_as_uint(A) == 0x80000000u; }
__device__ __forceinline__ float glr_map(float A, float H, float h) { return glr_cut(A) ? H : fmaf(A, h, H); }
// (A, H) after (A0, H0)
__device__ __forceinline__ void glr_join(float A, float H, float& A0, float& H0) {
  H0 = glr_map(A, H, H0);
  A0 = glr_cut(A) || glr_cut(A0) ? kMinusZero : __fmul_rn(A, A0);
}

__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(unsigned* p, unsigned v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Publish a lane's part and then the tile's flag.
__device__ __forceinline__ void glr_publish_pair(const GlrChain& c, int tile, int lane, float2 A, float2 H) {
  __stcg(c.pairs + static_cast<int64_t>(tile) * 32 + lane, make_float4(A.x, H.x, A.y, H.y));
  __syncwarp();
  if (lane == 0) {
    __threadfence();
    st_release(c.flags + tile, 1u);
  }
}
__device__ __forceinline__ void glr_publish_state(const GlrChain& c, int tile, int lane, float2 h) {
  __stcg(c.states + static_cast<int64_t>(tile) * 32 + lane, h);
  __syncwarp();
  if (lane == 0) {
    __threadfence();
    st_release(c.flags + tile, 2u);
  }
}

// The state before the tile of this level (> 0) and column: from the nearest
// published state among the 32 tiles before it.  One warp, two channels a
// lane.  False when the wait ran out.
__device__ __forceinline__ bool glr_look_back(const GlrChain& c, const GlrTiles& g, int level, int col, int lane,
                                              float2& h) {
  const int mine = level - 1 - lane;
  const unsigned* flag = c.flags + static_cast<int64_t>(mine < 0 ? 0 : mine) * g.ncols + col;
  const long long start = clock64();
  int n;
  for (;;) {
    const unsigned f = mine >= 0 ? ld_acquire(flag) : 0u;
    const unsigned whole = __ballot_sync(kFullMask, f == 2u), some = __ballot_sync(kFullMask, f != 0u);
    n = __ffs(whole) - 1;
    if (n >= 0 && ((~some) & ((1u << n) - 1u)) == 0u) break;
    if (clock64() - start > kWaitBudgetCycles) return false;
    __nanosleep(20);
  }
  __syncwarp();
  __threadfence();
  int tile = (level - 1 - n) * g.ncols + col;
  h = __ldcg(c.states + static_cast<int64_t>(tile) * 32 + lane);
  for (int k = 0; k < n; k += 4) {
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k + i < n) v[i] = __ldcg(c.pairs + static_cast<int64_t>(tile + (k + i + 1) * g.ncols) * 32 + lane);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k + i < n) h = make_float2(glr_map(v[i].x, v[i].y, h.x), glr_map(v[i].z, v[i].w, h.y));
  }
  return true;
}

// Host side (glr_fwd.cu): sizes, maps of the tensor copies, outputs in pairs.
GlrTiles glr_tiles(int64_t B, int64_t L, int64_t C);
bool glr_map_eligible(const void* p, const int64_t* s, int64_t B, int64_t L, int64_t C, Dtype dt);
bool glr_map3(CUtensorMap* m, const void* p, const int64_t* s, int64_t B, int64_t L, int64_t C, const int64_t* box2,
              Dtype dt);
bool glr_pair_out(const void* p, const int64_t* s, Dtype dt);

// A chained kernel follows the memset of its flags: a plain launch.
template <typename... P, typename... A>
cudaError_t glr_launch(void (*kernel)(P...), const GlrTiles& g, unsigned grid, unsigned threads, size_t smem,
                       cudaStream_t stream, A&&... args) {
  if (g.levels <= 1) return launch_pdl(kernel, grid, threads, smem, stream, std::forward<A>(args)...);
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

// Two channels of an any-stride tensor at p (`in0`, `in1`: they exist).
template <int DT>
__device__ __forceinline__ uint64_t glr_ldg(const void* p, int64_t off, int64_t cs, bool in0, bool in1) {
  const typename Fmt<DT>::E* e = static_cast<const typename Fmt<DT>::E*>(p) + off;
  return pk(in0 ? Fmt<DT>::to_f(e[0]) : 0.f, in1 ? Fmt<DT>::to_f(e[cs]) : 0.f);
}

template <int DT>
__device__ __forceinline__ void glr_stg(void* p, int64_t off, int64_t cs, bool pair, bool in0, bool in1, uint64_t v) {
  using E = typename Fmt<DT>::E;
  E* e = static_cast<E*>(p) + off;
  float a, b;
  upk(v, a, b);
  if (pair && in1) {
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
  upk(fmul2(z, pk(-kLog2e, -kLog2e)), a, b);
  e = pk(ex2_approx(a), ex2_approx(b));
  upk(fadd2(e, pk(1.f, 1.f)), a, b);
  s = pk(rcp_approx(a), rcp_approx(b));
}

// a and 1 - a^2 of a pair of logarithms, as glr_decay.
__device__ __forceinline__ void glr_decay2(uint64_t l, uint64_t& a, uint64_t& m2) {
  auto two = [](float x) { return pk(x, x); };
  uint64_t E = ffma2(l, two(1.f / 5040.f), two(1.f / 720.f));
  E = ffma2(E, l, two(1.f / 120.f));
  E = ffma2(E, l, two(1.f / 24.f));
  E = ffma2(E, l, two(1.f / 6.f));
  E = ffma2(E, l, two(0.5f));
  E = ffma2(E, l, two(1.f));
  E = fmul2(E, l);
  const uint64_t near = fadd2(E, two(1.f));
  float t0, t1, n0, n1, l0, l1, e0, e1;
  upk(fmul2(l, two(kLog2e)), t0, t1);
  const float f0 = ex2_approx(t0), f1 = ex2_approx(t1);
  float g0, g1;
  upk(fadd2(pk(f0, f1), two(-1.f)), g0, g1);
  upk(near, n0, n1);
  upk(l, l0, l1);
  upk(E, e0, e1);
  const bool c0 = l0 >= kGlrSeries, c1 = l1 >= kGlrSeries;
  a = pk(c0 ? n0 : f0, c1 ? n1 : f1);
  E = pk(c0 ? e0 : g0, c1 ? e1 : g1);
  m2 = fmul2(E, ffma2(E, two(-1.f), two(-2.f)));
}

}  // namespace ccv

// Group normalisation where every row is normalised on its own (S = 1): the
// norm of each token's heads.
//
// A group's vectors lie in LPG adjacent lanes, NV vectors a lane, and its sums
// are exchanges between these lanes: no barrier, no shared memory.  A lane keeps
// its channels' parameters (and, backwards, their gradients' sums) in registers
// and walks over rows; the loads of the next rows are in flight while the
// present ones are worked on.
//
// bf16, 16384 rows x 5120 channels in 40 groups with SiLU 78.9 us (4.3 TB/s), the
// backward pass of 8192 x 4096 in 32 groups 44.5 us (4.5 TB/s).  What bounds it:
// 14 (24) instructions an element at 55 % of the issue slots beside the loads'
// latency.  Two vectors a lane instead of one halve the exchanges (backward 68 ->
// 45); a row more in flight (76, backward 50) and rings of bulk copies a warp did
// not pay.
#include <type_traits>

#include "ccv_common.cuh"
#include "rec_internal.h"
#include "rec_pairs.cuh"

namespace ccv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sums over the LPG lanes of a group.
template <int LPG, int NS>
__device__ __forceinline__ void lanes_sum(float (&v)[NS]) {
#pragma unroll
  for (int m = LPG / 2; m > 0; m >>= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] += __shfl_xor_sync(kFullMask, v[i], m);
}

// A lane's place: its group, vectors and rows.  Warp tasks are (rows, column
// block of 32 / LPG groups); a block's warps have the same column block.
template <int LPG>
struct Lane {
  int64_t g, row, step;
  int sub;
  bool on;
  __device__ Lane(const GnArgs& a, int colblocks) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t cb = blockIdx.x % colblocks, slot = blockIdx.x / colblocks;
    g = cb * (32 / LPG) + lane / LPG;
    sub = lane % LPG;
    on = g < a.G;
    row = slot * kWarps + warp;
    step = static_cast<int64_t>(gridDim.x / colblocks) * kWarps;
  }
};

template <int DT, int LPG, int NV, bool FULL, bool SILU>
__global__ void __launch_bounds__(kThreads, NV == 1 ? 4 : NV == 2 ? 3 : 1) gn_rows_fwd(const GnArgs a, int colblocks) {
  constexpr int V = Fmt<DT>::VEC, H = V / 2;
  using E = typename Fmt<DT>::E;
  pdl_enter();
  const Lane<LPG> l(a, colblocks);
  const int cg = static_cast<int>(a.C / a.G);
  const float inv = 1.f / static_cast<float>(cg);
  uint64_t w[NV][H], b[NV][H];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (l.sub + i * LPG) * V, ch = l.g * cg + col;
    in[i] = FULL || (l.on && col < cg);
#pragma unroll
    for (int j = 0; j < H; ++j) {
      float x[2], y[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        x[k] = a.w == nullptr ? 1.f : in[i] ? ld_param(a.w, (ch + 2 * j + k) * a.ws, a.wdt) : 0.f;
        y[k] = a.b == nullptr || !in[i] ? 0.f : ld_param(a.b, (ch + 2 * j + k) * a.bs, a.wdt);
      }
      w[i][j] = pk(x[0], x[1]), b[i][j] = pk(y[0], y[1]);
    }
  }
  const E* x = static_cast<const E*>(a.x) + l.row * a.xs[0] + l.g * cg + l.sub * V;
  E* out = static_cast<E*>(a.out) + l.row * a.os[0] + l.g * cg + l.sub * V;
  const int64_t x_hop = l.step * a.xs[0], out_hop = l.step * a.os[0];
  uint4 raw[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      raw[i] = (FULL || in[i]) && row < a.N ? ld_stream16(x + i * LPG * V) : make_uint4(0, 0, 0, 0);
    x += x_hop;
  };
  fetch(l.row);
  for (int64_t row = l.row; row < a.N; row += l.step) {
    uint64_t f[NV][H], acc = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack_pairs<DT>(raw[i], f[i]);
#pragma unroll
      for (int j = 0; j < H; ++j) acc = fadd2(acc, f[i][j]);
    }
    fetch(row + l.step);
    float s[1] = {pair_sum(acc)};
    lanes_sum<LPG>(s);
    const float mean = s[0] * inv;
    const uint64_t minus = pk(-mean, -mean);
    acc = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < H; ++j) {
        f[i][j] = FULL || in[i] ? fadd2(f[i][j], minus) : 0;
        acc = ffma2(f[i][j], f[i][j], acc);
      }
    s[0] = pair_sum(acc);
    lanes_sum<LPG>(s);
    const float r = rsqrtf(fmaf(s[0], inv, a.eps));
    const uint64_t r2 = pk(r, r);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[V];
#pragma unroll
      for (int j = 0; j < H; ++j) {
        uint64_t z = ffma2(fmul2(f[i][j], r2), w[i][j], b[i][j]);
        if constexpr (SILU) z = silu_pair(z);
        upk(z, o[2 * j], o[2 * j + 1]);
      }
      if (FULL || in[i]) st16_stream(out + i * LPG * V, pack16<DT>(o));
    }
    out += out_hop;
  }
}

template <int DT, int LPG, int NV, bool FULL, bool SILU>
__global__ void __launch_bounds__(kThreads, NV == 1 ? 3 : NV == 2 ? 2 : 1) gn_rows_bwd(const GnArgs a, int colblocks) {
  constexpr int V = Fmt<DT>::VEC, H = V / 2;
  using E = typename Fmt<DT>::E;
  __shared__ float sums[kWarps][32][NV * V];
  pdl_enter();
  const Lane<LPG> l(a, colblocks);
  const int cg = static_cast<int>(a.C / a.G);
  const float inv = 1.f / static_cast<float>(cg);
  uint64_t w[NV][H], b[NV][H], dw[NV][H], db[NV][H];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (l.sub + i * LPG) * V, ch = l.g * cg + col;
    in[i] = FULL || (l.on && col < cg);
#pragma unroll
    for (int j = 0; j < H; ++j) {
      float x[2], y[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        x[k] = a.w == nullptr ? 1.f : in[i] ? ld_param(a.w, (ch + 2 * j + k) * a.ws, a.wdt) : 0.f;
        y[k] = a.b == nullptr || !in[i] ? 0.f : ld_param(a.b, (ch + 2 * j + k) * a.bs, a.wdt);
      }
      w[i][j] = pk(x[0], x[1]), b[i][j] = pk(y[0], y[1]);
      dw[i][j] = db[i][j] = 0;
    }
  }
  const int64_t c0 = l.g * cg + l.sub * V;
  const E* x = static_cast<const E*>(a.x) + l.row * a.xs[0] + c0;
  const E* dy = static_cast<const E*>(a.dout) + l.row * a.gs[0] + c0;
  E* dx = static_cast<E*>(a.dx) + l.row * a.dxs[0] + c0;
  const int64_t x_hop = l.step * a.xs[0], dy_hop = l.step * a.gs[0], dx_hop = l.step * a.dxs[0];
  uint4 rx[NV], rg[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool on = (FULL || in[i]) && row < a.N;
      rx[i] = on ? ld_stream16(x + i * LPG * V) : make_uint4(0, 0, 0, 0);
      rg[i] = on ? ld_stream16(dy + i * LPG * V) : make_uint4(0, 0, 0, 0);
    }
    x += x_hop, dy += dy_hop;
  };
  fetch(l.row);
  for (int64_t row = l.row; row < a.N; row += l.step) {
    uint64_t f[NV][H], d[NV][H], acc = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack_pairs<DT>(rx[i], f[i]);
      unpack_pairs<DT>(rg[i], d[i]);
#pragma unroll
      for (int j = 0; j < H; ++j) acc = fadd2(acc, f[i][j]);
    }
    fetch(row + l.step);
    float s[1] = {pair_sum(acc)};
    lanes_sum<LPG>(s);
    const float mean = s[0] * inv;
    const uint64_t minus = pk(-mean, -mean);
    acc = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < H; ++j) {
        f[i][j] = FULL || in[i] ? fadd2(f[i][j], minus) : 0;
        acc = ffma2(f[i][j], f[i][j], acc);
      }
    s[0] = pair_sum(acc);
    lanes_sum<LPG>(s);
    const float r = rsqrtf(fmaf(s[0], inv, a.eps));
    const uint64_t r2 = pk(r, r);
    uint64_t a1 = 0, a2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < H; ++j) {
        f[i][j] = fmul2(f[i][j], r2);  // xh
        if constexpr (SILU) d[i][j] = silu_grad_pair(ffma2(f[i][j], w[i][j], b[i][j]), d[i][j]);
        dw[i][j] = ffma2(d[i][j], f[i][j], dw[i][j]);
        db[i][j] = fadd2(db[i][j], d[i][j]);
        d[i][j] = fmul2(d[i][j], w[i][j]);
        a1 = fadd2(a1, d[i][j]);
        a2 = ffma2(d[i][j], f[i][j], a2);
      }
    float q[2] = {pair_sum(a1), pair_sum(a2)};
    lanes_sum<LPG>(q);
    const float c1 = -r * (q[0] * inv), c2 = -r * (q[1] * inv);
    const uint64_t k1 = pk(c1, c1), k2 = pk(c2, c2);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[V];
#pragma unroll
      for (int j = 0; j < H; ++j) upk(ffma2(d[i][j], r2, ffma2(f[i][j], k2, k1)), o[2 * j], o[2 * j + 1]);
      if (FULL || in[i]) st16_stream(dx + i * LPG * V, pack16<DT>(o));
    }
    dx += dx_hop;
  }
  if (a.part == nullptr) return;
  // the block's warps in order, one partial sum a block
  float* part = a.part + static_cast<int64_t>(blockIdx.x / colblocks) * 2 * a.C;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < H; ++j) {
        float u, v;
        upk(which == 0 ? dw[i][j] : db[i][j], u, v);
        sums[warp][lane][i * V + 2 * j] = u;
        sums[warp][lane][i * V + 2 * j + 1] = v;
      }
    __syncthreads();
    for (int k = threadIdx.x; k < 32 * NV * V; k += kThreads) {
      const int ln = k / (NV * V), e = k % (NV * V);
      const int64_t g = (blockIdx.x % colblocks) * (32 / LPG) + ln / LPG;
      const int64_t col = (ln % LPG + e / V * LPG) * V + e % V;
      if (g < a.G && col < cg) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) v += sums[i][ln][e];
        part[which * a.C + g * cg + col] = v;
      }
    }
  }
}

// Lanes of a group and vectors a lane.  Two vectors a lane halve the exchanges
// for each element.
struct Shape {
  int lpg, nv;
};
Shape shape_of(int64_t vecs) {
  if (vecs <= 4) return {4, 1};
  if (vecs <= 8) return {4, 2};
  if (vecs <= 16) return {8, 2};
  if (vecs <= 32) return {16, 2};
  if (vecs <= 64) return {32, 2};
  return {32, 4};
}

template <int DT, int LPG, int NV>
cudaError_t launch(const GnArgs& a, bool bwd, int64_t slots, cudaStream_t s) {
  const int colblocks = static_cast<int>((a.G + 32 / LPG - 1) / (32 / LPG));
  const unsigned grid = static_cast<unsigned>(colblocks * slots);
  const bool full = a.C / a.G == LPG * NV * Fmt<DT>::VEC && a.G % (32 / LPG) == 0;
  auto go = [&](auto f, auto y) {
    constexpr bool F = decltype(f)::value, Y = decltype(y)::value;
    if (bwd) return launch_pdl(gn_rows_bwd<DT, LPG, NV, F, Y>, grid, kThreads, 0, s, a, colblocks);
    return launch_pdl(gn_rows_fwd<DT, LPG, NV, F, Y>, grid, kThreads, 0, s, a, colblocks);
  };
  if (full) return a.silu ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
  return a.silu ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
}

template <int DT>
cudaError_t launch_dt(const GnArgs& a, bool bwd, int64_t slots, cudaStream_t s) {
  const Shape h = shape_of(a.C / a.G / Fmt<DT>::VEC);
  switch (h.lpg * 10 + h.nv) {
    case 41: return launch<DT, 4, 1>(a, bwd, slots, s);
    case 42: return launch<DT, 4, 2>(a, bwd, slots, s);
    case 82: return launch<DT, 8, 2>(a, bwd, slots, s);
    case 162: return launch<DT, 16, 2>(a, bwd, slots, s);
    case 322: return launch<DT, 32, 2>(a, bwd, slots, s);
    default: return launch<DT, 32, 4>(a, bwd, slots, s);
  }
}

bool aligned(const void* p, const int64_t* s, int64_t N, int64_t v) {
  return s[2] == 1 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && (N == 1 || s[0] % v == 0);
}

}  // namespace

// Rows of their own, in groups of whole vectors, at most 128 of them.
bool gn_rows_eligible(const GnArgs& a, Dtype dt, bool bwd) {
  const int64_t v = dt == kF32 ? 4 : 8, cg = a.C / a.G;
  if (a.S != 1 || cg % v != 0 || cg / v > 128 || !aligned(a.x, a.xs, a.N, v)) return false;
  return bwd ? aligned(a.dout, a.gs, a.N, v) && aligned(a.dx, a.dxs, a.N, v) : aligned(a.out, a.os, a.N, v);
}

// Blocks side by side over the rows: one wave (152 SMs) of the column blocks,
// a function of the sizes alone.
int64_t gn_rows_slots(int64_t N, int64_t C, int64_t G, int64_t esize, bool bwd) {
  const Shape h = shape_of(C / G / (16 / esize));
  const int64_t colblocks = (G + 32 / h.lpg - 1) / (32 / h.lpg);
  const int64_t most = 152 * (bwd ? (h.nv == 1 ? 3 : h.nv == 2 ? 2 : 1) : (h.nv == 1 ? 4 : h.nv == 2 ? 3 : 1));
  int64_t slots = (most + colblocks - 1) / colblocks;
  const int64_t rows = (N + kWarps - 1) / kWarps;
  if (slots > rows) slots = rows;
  return slots < 1 ? 1 : slots;
}

cudaError_t launch_gn_rows(const GnArgs& a, Dtype dt, bool bwd, cudaStream_t stream) {
  const int64_t slots = gn_rows_slots(a.N, a.C, a.G, dt == kF32 ? 4 : 2, bwd);
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, bwd, slots, stream);
    case kF16: return launch_dt<kF16>(a, bwd, slots, stream);
    case kBF16: return launch_dt<kBF16>(a, bwd, slots, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ccv

// Layer normalisation over the last dimension, forward and backward.
//
//   xh = (x - m) r,  m = mean(x),  r = 1 / sqrt(mean((x - m)^2) + eps);   y = xh w + b
//   d = dy w;   dx = r (d - mean(d) - xh mean(d xh));   dw = sum_rows dy xh;   db = sum_rows dy
//
// Mean and variance are two reductions over the row held in registers (the
// variance of x - m, so a large mean costs no precision), all sums in FP32.
// The backward pass needs nothing saved by the forward: it reads x and dy
// once, takes the row's statistics again, and keeps each column's dw and db
// in registers over all rows of a block; a block writes one partial sum per
// column, and a second kernel adds the partials in a fixed order (bitwise
// reproducible, no atomics).
//
// What bounds it: HBM (2 N D elements forward, 3 N D backward).  Rows of more
// than 32 vectors come through a ring of row-sized stages in shared memory,
// filled by bulk copies: the bytes in flight do not depend on how many
// registers the arithmetic takes, blocks are persistent (weights stay in
// registers), and a stage is refilled right after the row's first reduction,
// whose barrier is also the proof that every thread has read it.  Shorter
// rows take a warp each.  16384 rows of 5120 in bf16 forward: 61.9 us (336 MB,
// 5.4 TB/s, 0.80 of the copy rate); 8192 rows of 4096 backward: 42.6 us (201 MB,
// 4.7 TB/s, 0.70).  Without the ring (plain loads into registers) they took 141
// and 93 us; other vectors a thread and blocks an SM (2 of either, 4 blocks) 69
// to 83 us forward, and backward with three blocks an SM 61 us.
#include "ccv_common.cuh"
#include "ccv_tma.cuh"
#include "mix_internal.h"

namespace ccv {
namespace {

__device__ unsigned g_fault;

constexpr int kRingBytes = 200 * 1024;  // stages of all blocks of an SM
constexpr int kMaxStages = 8;

// Sum of NS values over the threads that share a row: one warp, or the block.
template <bool WARP, int NS>
__device__ __forceinline__ void row_sum(float (&v)[NS], float* red, int nwarps) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] += __shfl_xor_sync(kFullMask, v[i], m);
  if constexpr (!WARP) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < NS; ++i) red[warp * NS + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      float x = lane < nwarps ? red[lane * NS + i] : 0.f;
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(kFullMask, x, m);
      v[i] = x;
    }
    __syncthreads();
  }
}

// Elements of one vector access: 16 bytes, or one element where the row is
// not aligned (V = 1).
template <int DT, int V>
__device__ __forceinline__ void load_v(const void* base, int64_t off, int64_t stride, float* f) {
  using E = typename Fmt<DT>::E;
  const E* p = static_cast<const E*>(base);
  if constexpr (V == 1) {
    f[0] = Fmt<DT>::to_f(p[off * stride]);
  } else {
    unpack16<DT>(*reinterpret_cast<const uint4*>(p + off), f);
  }
}

template <int DT, int V>
__device__ __forceinline__ void store_v(void* base, int64_t off, int64_t stride, const float* f) {
  using E = typename Fmt<DT>::E;
  E* p = static_cast<E*>(base);
  if constexpr (V == 1) {
    p[off * stride] = Fmt<DT>::from_f(f[0]);
  } else {
    *reinterpret_cast<uint4*>(p + off) = pack16<DT>(f);
  }
}

// Sum over the block with one barrier: `red` (NS x 32 floats, zero beyond the
// block's warps) is not written again before another barrier has passed.
template <int NS>
__device__ __forceinline__ void block_sum(float (&v)[NS], float* red, int nwarps) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] += __shfl_xor_sync(kFullMask, v[i], m);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < NS; ++i) red[i * 32 + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const float4 x = *reinterpret_cast<const float4*>(red + i * 32);
    v[i] = (x.x + x.y) + (x.z + x.w);
  }
  for (int k = 4; k < nwarps; k += 4)
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(red + i * 32 + k);
      v[i] += (x.x + x.y) + (x.z + x.w);
    }
}

// The vector at p as pairs; zeros where it lies outside the row.
template <int DT>
__device__ __forceinline__ void load_pairs(const uint8_t* p, bool in, uint64_t* f) {
  constexpr int V = Fmt<DT>::VEC;
  float x[V];
  unpack16<DT>(in ? lds128(p) : make_uint4(0, 0, 0, 0), x);
#pragma unroll
  for (int j = 0; j < V / 2; ++j) f[j] = pk(x[2 * j], x[2 * j + 1]);
}

__device__ __forceinline__ float pair_sum(uint64_t v) {
  float a, b;
  upk(v, a, b);
  return a + b;
}

// V parameters from column col: one or two vector loads where the vector is
// dense and aligned (`vec`).
template <int V>
__device__ __forceinline__ void load_par_vec(const void* w, int64_t col, int64_t ws, int wdt, bool vec, float fill,
                                             float* f) {
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = fill;
  } else if (vec && V >= 4) {
    if (wdt == kF32) {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + col + j));
        f[j] = x.x, f[j + 1] = x.y, f[j + 2] = x.z, f[j + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + col + j));
        const uint32_t y[2] = {x.x, x.y};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f[j + i] = wdt == kF16 ? Fmt<kF16>::word_elem(y[i >> 1], i & 1) : Fmt<kBF16>::word_elem(y[i >> 1], i & 1);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = ld_param(w, (col + j) * ws, wdt);
  }
}

// NV vectors of V elements a thread; WARP: a warp owns a row, else the block.
template <int DT, int V, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) ln_fwd_kernel(const LnArgs a) {
  pdl_enter();
  __shared__ float red[32];
  const int G = WARP ? 32 : blockDim.x;  // threads of one row
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int nwarps = blockDim.x >> 5;
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * nwarps + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.N) return;
  using E = typename Fmt<DT>::E;
  const E* x = static_cast<const E*>(a.x) + row * a.xs0;
  E* y = static_cast<E*>(a.out) + row * a.os0;
  float f[NV][V];
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (static_cast<int64_t>(i) * G + t) * V;
    if (col < a.D) {
      load_v<DT, V>(x, col, a.xs1, f[i]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) f[i][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s[0] += f[i][j];
  }
  row_sum<WARP>(s, red, nwarps);
  const float inv_d = 1.f / static_cast<float>(a.D);
  const float mean = s[0] * inv_d;
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (static_cast<int64_t>(i) * G + t) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      f[i][j] -= mean;
      if (col < a.D) q[0] = fmaf(f[i][j], f[i][j], q[0]);
    }
  }
  row_sum<WARP>(q, red, nwarps);
  const float r = rsqrtf(q[0] * inv_d + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (static_cast<int64_t>(i) * G + t) * V;
    if (col < a.D) {
      float w[V], b[V];
      load_par_vec<V>(a.w, col, a.ws, a.wdt, a.wvec, 1.f, w);
      load_par_vec<V>(a.b, col, a.bs, a.wdt, a.wvec, 0.f, b);
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = fmaf(f[i][j] * r, w[j], b[j]);
      store_v<DT, V>(y, col, a.os1, w);
    }
  }
}

// Persistent block, rows blockIdx, blockIdx + grid, ... through the ring.
template <int DT, int NV>
__global__ void __launch_bounds__(512) ln_fwd_ring(const LnArgs a, int stages) {
  constexpr int V = Fmt<DT>::VEC;
  using E = typename Fmt<DT>::E;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ __align__(16) float red[2][32];
  const uint32_t row_bytes = static_cast<uint32_t>(a.D) * sizeof(E);
  const int t = threadIdx.x, T = blockDim.x, nwarps = T >> 5;
  const int64_t step = gridDim.x;
  if (t < 32) red[0][t] = red[1][t] = 0.f;
  auto fill = [&](int64_t row, int s) {
    mbar_arrive_expect_tx(&full[s], row_bytes);
    bulk_load(ring + s * row_bytes, static_cast<const E*>(a.x) + row * a.xs0, row_bytes, &full[s]);
  };
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  pdl_enter();
  if (t == 0)
    for (int s = 0; s < stages && blockIdx.x + s * step < a.N; ++s) fill(blockIdx.x + s * step, s);
  // elements in pairs: packed arithmetic
  constexpr int H = V / 2;
  uint64_t w[NV][H], b[NV][H];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (static_cast<int64_t>(i) * T + t) * V;
    float pw[V], pb[V];
#pragma unroll
    for (int j = 0; j < V; ++j) pw[j] = pb[j] = 0.f;
    if (col < a.D) {
      load_par_vec<V>(a.w, col, a.ws, a.wdt, a.wvec, 1.f, pw);
      load_par_vec<V>(a.b, col, a.bs, a.wdt, a.wvec, 0.f, pb);
    }
#pragma unroll
    for (int j = 0; j < H; ++j) w[i][j] = pk(pw[2 * j], pw[2 * j + 1]), b[i][j] = pk(pb[2 * j], pb[2 * j + 1]);
  }
  __syncthreads();
  const float inv_d = 1.f / static_cast<float>(a.D);
  int s = 0;
  uint32_t parity = 0;
  for (int64_t row = blockIdx.x; row < a.N; row += step) {
    if (!mbar_wait(&full[s], parity)) {
      if (t == 0) {
        atomicOr(&g_fault, kFaultConsumerWait);
        for (int k = 1; k < stages && row + k * step < a.N; ++k)  // the copies still in flight
          mbar_wait(&full[(s + k) % stages], (s + k >= stages) ? parity ^ 1 : parity);
      }
      return;
    }
    uint64_t f[NV][H];
    uint64_t acc = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * T + t) * V;
      load_pairs<DT>(ring + s * row_bytes + col * sizeof(E), col < a.D, f[i]);
#pragma unroll
      for (int j = 0; j < H; ++j) acc = fadd2(acc, f[i][j]);
    }
    float sum[1] = {pair_sum(acc)};
    block_sum(sum, red[0], nwarps);
    if (t == 0 && row + stages * step < a.N) fill(row + stages * step, s);
    if (++s == stages) s = 0, parity ^= 1;
    const float mean = sum[0] * inv_d;
    const uint64_t minus = pk(-mean, -mean);
    acc = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = (i * T + t) * V < a.D;
#pragma unroll
      for (int j = 0; j < H; ++j) {
        f[i][j] = fadd2(f[i][j], minus);
        if (in) acc = ffma2(f[i][j], f[i][j], acc);
      }
    }
    float q[1] = {pair_sum(acc)};
    block_sum(q, red[1], nwarps);
    const float r = rsqrtf(q[0] * inv_d + a.eps);
    const uint64_t r2 = pk(r, r);
    E* y = static_cast<E*>(a.out) + row * a.os0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * T + t) * V;
      if (col < a.D) {
        float o[V];
#pragma unroll
        for (int j = 0; j < H; ++j) upk(ffma2(fmul2(f[i][j], r2), w[i][j], b[i][j]), o[2 * j], o[2 * j + 1]);
        *reinterpret_cast<uint4*>(y + col) = pack16<DT>(o);
      }
    }
  }
}

// Rows of any size and strides: three sweeps over the row by one block.
template <int DT>
__global__ void ln_fwd_any(const LnArgs a) {
  pdl_enter();
  __shared__ float red[32];
  using F = Fmt<DT>;
  using E = typename F::E;
  const int nwarps = blockDim.x >> 5;
  const E* x = static_cast<const E*>(a.x) + blockIdx.x * a.xs0;
  E* y = static_cast<E*>(a.out) + blockIdx.x * a.os0;
  float s[1] = {0.f};
  for (int64_t c = threadIdx.x; c < a.D; c += blockDim.x) s[0] += F::to_f(x[c * a.xs1]);
  row_sum<false>(s, red, nwarps);
  const float inv_d = 1.f / static_cast<float>(a.D), mean = s[0] * inv_d;
  float q[1] = {0.f};
  for (int64_t c = threadIdx.x; c < a.D; c += blockDim.x) {
    const float d = F::to_f(x[c * a.xs1]) - mean;
    q[0] = fmaf(d, d, q[0]);
  }
  row_sum<false>(q, red, nwarps);
  const float r = rsqrtf(q[0] * inv_d + a.eps);
  for (int64_t c = threadIdx.x; c < a.D; c += blockDim.x) {
    const float w = a.w != nullptr ? ld_param(a.w, c * a.ws, a.wdt) : 1.f;
    const float b = a.b != nullptr ? ld_param(a.b, c * a.bs, a.wdt) : 0.f;
    y[c * a.os1] = F::from_f(fmaf((F::to_f(x[c * a.xs1]) - mean) * r, w, b));
  }
}

// Backward: block (or warp) rows blockIdx, blockIdx + grid, ...; partial sums
// of dw and db in registers.
template <int DT, int V, int NV, bool WARP, int MAXT>
__global__ void __launch_bounds__(MAXT) ln_bwd_kernel(const LnBwdArgs a) {
  pdl_enter();
  extern __shared__ float sh[];  // WARP: [warps][2][D]; else the row sums
  const int G = WARP ? 32 : blockDim.x;
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int nwarps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  using E = typename Fmt<DT>::E;
  float dw[NV][V], db[NV][V], w[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (static_cast<int64_t>(i) * G + t) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) dw[i][j] = db[i][j] = w[i][j] = 0.f;
    if (col < a.D) load_par_vec<V>(a.w, col, a.ws, a.wdt, a.wvec, 1.f, w[i]);
  }
  const float inv_d = 1.f / static_cast<float>(a.D);
  const int64_t step = WARP ? static_cast<int64_t>(gridDim.x) * nwarps : gridDim.x;
  for (int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * nwarps + warp : blockIdx.x; row < a.N; row += step) {
    const E* x = static_cast<const E*>(a.x) + row * a.xs0;
    const E* gr = static_cast<const E*>(a.dout) + row * a.gs0;
    E* dx = static_cast<E*>(a.dx) + row * a.dxs0;
    float f[NV][V], d[NV][V];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (static_cast<int64_t>(i) * G + t) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) f[i][j] = d[i][j] = 0.f;
      if (col < a.D) {
        load_v<DT, V>(x, col, a.xs1, f[i]);
        load_v<DT, V>(gr, col, a.gs1, d[i]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) s[0] += f[i][j];
    }
    row_sum<WARP>(s, sh, nwarps);
    const float mean = s[0] * inv_d;
    float q[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (static_cast<int64_t>(i) * G + t) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        f[i][j] -= mean;
        if (col >= a.D) f[i][j] = 0.f;
        q[0] = fmaf(f[i][j], f[i][j], q[0]);
        const float dd = d[i][j] * w[i][j];
        q[1] += dd;
        q[2] = fmaf(dd, f[i][j], q[2]);
      }
    }
    row_sum<WARP>(q, sh, nwarps);
    const float r = rsqrtf(q[0] * inv_d + a.eps);
    const float c1 = q[1] * inv_d, c2 = q[2] * inv_d * r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (static_cast<int64_t>(i) * G + t) * V;
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xh = f[i][j] * r;
        dw[i][j] = fmaf(d[i][j], xh, dw[i][j]);
        db[i][j] += d[i][j];
        o[j] = r * (d[i][j] * w[i][j] - c1 - xh * c2);
      }
      if (col < a.D) store_v<DT, V>(dx, col, a.dxs1, o);
    }
  }
  if (a.part == nullptr) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.D;
  if constexpr (WARP) {
    // the block's warps in order
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (static_cast<int64_t>(i) * 32 + t) * V;
      if (col < a.D)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          sh[(warp * 2 + 0) * a.D + col + j] = dw[i][j];
          sh[(warp * 2 + 1) * a.D + col + j] = db[i][j];
        }
    }
    __syncthreads();
    for (int64_t c = threadIdx.x; c < 2 * a.D; c += blockDim.x) {
      float x = 0.f;
      for (int k = 0; k < nwarps; ++k) x += sh[k * 2 * a.D + c];
      part[c] = x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (static_cast<int64_t>(i) * G + t) * V;
      if (col < a.D)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          part[col + j] = dw[i][j];
          part[a.D + col + j] = db[i][j];
        }
    }
  }
}

// The same through the ring: a stage holds a row of x and of dout.
template <int DT, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) ln_bwd_ring(const LnBwdArgs a, int stages) {
  constexpr int V = Fmt<DT>::VEC;
  using E = typename Fmt<DT>::E;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ __align__(16) float red0[32], red1[96];
  const uint32_t row_bytes = static_cast<uint32_t>(a.D) * sizeof(E);
  const int t = threadIdx.x, T = blockDim.x, nwarps = T >> 5;
  const int64_t step = gridDim.x;
  if (t < 32) red0[t] = red1[t] = red1[32 + t] = red1[64 + t] = 0.f;
  auto fill = [&](int64_t row, int s) {
    mbar_arrive_expect_tx(&full[s], 2 * row_bytes);
    bulk_load(ring + 2 * s * row_bytes, static_cast<const E*>(a.x) + row * a.xs0, row_bytes, &full[s]);
    bulk_load(ring + (2 * s + 1) * row_bytes, static_cast<const E*>(a.dout) + row * a.gs0, row_bytes, &full[s]);
  };
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  pdl_enter();
  if (t == 0)
    for (int s = 0; s < stages && blockIdx.x + s * step < a.N; ++s) fill(blockIdx.x + s * step, s);
  // elements in pairs: packed arithmetic
  constexpr int H = V / 2;
  uint64_t w[NV][H], dw[NV][H], db[NV][H];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (static_cast<int64_t>(i) * T + t) * V;
    float pw[V];
#pragma unroll
    for (int j = 0; j < V; ++j) pw[j] = 0.f;
    if (col < a.D) load_par_vec<V>(a.w, col, a.ws, a.wdt, a.wvec, 1.f, pw);
#pragma unroll
    for (int j = 0; j < H; ++j) {
      w[i][j] = pk(pw[2 * j], pw[2 * j + 1]);
      dw[i][j] = db[i][j] = 0;
    }
  }
  __syncthreads();
  const float inv_d = 1.f / static_cast<float>(a.D);
  int s = 0;
  uint32_t parity = 0;
  for (int64_t row = blockIdx.x; row < a.N; row += step) {
    if (!mbar_wait(&full[s], parity)) {
      if (t == 0) {
        atomicOr(&g_fault, kFaultConsumerWait);
        for (int k = 1; k < stages && row + k * step < a.N; ++k)  // the copies still in flight
          mbar_wait(&full[(s + k) % stages], (s + k >= stages) ? parity ^ 1 : parity);
      }
      return;
    }
    uint64_t f[NV][H], d[NV][H];
    uint64_t acc = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * T + t) * V;
      load_pairs<DT>(ring + 2 * s * row_bytes + col * sizeof(E), col < a.D, f[i]);
      load_pairs<DT>(ring + (2 * s + 1) * row_bytes + col * sizeof(E), col < a.D, d[i]);
#pragma unroll
      for (int j = 0; j < H; ++j) acc = fadd2(acc, f[i][j]);
    }
    float sum[1] = {pair_sum(acc)};
    block_sum(sum, red0, nwarps);
    if (t == 0 && row + stages * step < a.N) fill(row + stages * step, s);
    if (++s == stages) s = 0, parity ^= 1;
    const float mean = sum[0] * inv_d;
    const uint64_t minus = pk(-mean, -mean);
    uint64_t a0 = 0, a1 = 0, a2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = (i * T + t) * V < a.D;
#pragma unroll
      for (int j = 0; j < H; ++j) {
        f[i][j] = in ? fadd2(f[i][j], minus) : 0;
        a0 = ffma2(f[i][j], f[i][j], a0);
        const uint64_t dd = fmul2(d[i][j], w[i][j]);
        a1 = fadd2(a1, dd);
        a2 = ffma2(dd, f[i][j], a2);
      }
    }
    float q[3] = {pair_sum(a0), pair_sum(a1), pair_sum(a2)};
    block_sum(q, red1, nwarps);
    const float r = rsqrtf(q[0] * inv_d + a.eps);
    const float c1 = q[1] * inv_d, c2 = q[2] * inv_d * r;
    // dx = r (d w - c1 - xh c2) = (r w) d + (-r c1) + (-r c2) xh
    const uint64_t r2 = pk(r, r), rc1 = pk(-r * c1, -r * c1), rc2 = pk(-r * c2, -r * c2);
    E* dx = static_cast<E*>(a.dx) + row * a.dxs0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * T + t) * V;
      float o[V];
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const uint64_t xh = fmul2(f[i][j], r2);
        dw[i][j] = ffma2(d[i][j], xh, dw[i][j]);
        db[i][j] = fadd2(db[i][j], d[i][j]);
        upk(ffma2(fmul2(d[i][j], w[i][j]), r2, ffma2(xh, rc2, rc1)), o[2 * j], o[2 * j + 1]);
      }
      if (col < a.D) *reinterpret_cast<uint4*>(dx + col) = pack16<DT>(o);
    }
  }
  if (a.part == nullptr) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (static_cast<int64_t>(i) * T + t) * V;
    if (col < a.D)
#pragma unroll
      for (int j = 0; j < H; j += 2) {
        float x[4];
        upk(dw[i][j], x[0], x[1]);
        upk(dw[i][j + 1], x[2], x[3]);
        *reinterpret_cast<float4*>(part + col + 2 * j) = make_float4(x[0], x[1], x[2], x[3]);
        upk(db[i][j], x[0], x[1]);
        upk(db[i][j + 1], x[2], x[3]);
        *reinterpret_cast<float4*>(part + a.D + col + 2 * j) = make_float4(x[0], x[1], x[2], x[3]);
      }
  }
}

// Rows too long for registers: sweeps over the row, the partial sums of dw
// and db in the block's own slice of the workspace.
template <int DT>
__global__ void ln_bwd_any(const LnBwdArgs a) {
  pdl_enter();
  __shared__ float red[96];
  using F = Fmt<DT>;
  using E = typename F::E;
  const int nwarps = blockDim.x >> 5;
  float* part = a.part != nullptr ? a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.D : nullptr;
  const float inv_d = 1.f / static_cast<float>(a.D);
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    const E* x = static_cast<const E*>(a.x) + row * a.xs0;
    const E* gr = static_cast<const E*>(a.dout) + row * a.gs0;
    E* dx = static_cast<E*>(a.dx) + row * a.dxs0;
    float s[1] = {0.f};
    for (int64_t c = threadIdx.x; c < a.D; c += blockDim.x) s[0] += F::to_f(x[c * a.xs1]);
    row_sum<false>(s, red, nwarps);
    const float mean = s[0] * inv_d;
    float q[3] = {0.f, 0.f, 0.f};
    for (int64_t c = threadIdx.x; c < a.D; c += blockDim.x) {
      const float f = F::to_f(x[c * a.xs1]) - mean;
      const float d = F::to_f(gr[c * a.gs1]) * (a.w != nullptr ? ld_param(a.w, c * a.ws, a.wdt) : 1.f);
      q[0] = fmaf(f, f, q[0]);
      q[1] += d;
      q[2] = fmaf(d, f, q[2]);
    }
    row_sum<false>(q, red, nwarps);
    const float r = rsqrtf(q[0] * inv_d + a.eps);
    const float c1 = q[1] * inv_d, c2 = q[2] * inv_d * r;
    for (int64_t c = threadIdx.x; c < a.D; c += blockDim.x) {
      const float g = F::to_f(gr[c * a.gs1]);
      const float w = a.w != nullptr ? ld_param(a.w, c * a.ws, a.wdt) : 1.f;
      const float xh = (F::to_f(x[c * a.xs1]) - mean) * r;
      dx[c * a.dxs1] = F::from_f(r * (g * w - c1 - xh * c2));
      if (part != nullptr) {
        const bool first = row == blockIdx.x;
        part[c] = fmaf(g, xh, first ? 0.f : part[c]);
        part[a.D + c] = g + (first ? 0.f : part[a.D + c]);
      }
    }
  }
}

// dw and db: partials added in order, 32 strided subsequences and then these.
__global__ void __launch_bounds__(1024) ln_bwd_reduce(const LnBwdArgs a, int P) {
  pdl_enter();
  __shared__ float sh[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float x = 0.f;
  if (col < 2 * a.D) {
    const float* p = a.part + col;
#pragma unroll 8
    for (int i = r; i < P; i += 32) x += p[static_cast<int64_t>(i) * 2 * a.D];
  }
  sh[r][c] = x;
  __syncthreads();
  if (r == 0 && col < 2 * a.D) {
    x = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) x += sh[i][c];
    if (col < a.D) {
      if (a.dw != nullptr) st_param(a.dw, col * a.dws, a.wdt, x);
    } else if (a.db != nullptr) {
      st_param(a.db, (col - a.D) * a.dbs, a.wdt, x);
    }
  }
}

bool al16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

unsigned threads(int64_t n, int nv) { return static_cast<unsigned>(((n + nv - 1) / nv + 31) / 32 * 32); }

// Blocks of an SM (by the registers of NV vectors a thread) and stages of a
// block for rows of `bytes` a stage.  [16384,5120] bf16: 62.3 us with four
// vectors a thread and three blocks, 69.3 with two and three, 79 with four and two.
int ring_blocks(unsigned T, int NV) {
  const int n = (NV >= 4 ? 512 : 1024) / static_cast<int>(T);
  return n < 1 ? 1 : n < 8 ? n : 8;
}
int ring_stages(int blocks, int64_t bytes) {
  const int64_t n = kRingBytes / (blocks * bytes);
  return static_cast<int>(n < kMaxStages ? n : kMaxStages);
}

template <int DT, int NV>
cudaError_t fwd_ring(const LnArgs& a, const Device& dev, cudaStream_t s) {
  const unsigned T = threads(a.D / Fmt<DT>::VEC, NV);
  const int64_t bytes = a.D * static_cast<int64_t>(sizeof(typename Fmt<DT>::E));
  const int blocks = ring_blocks(T, NV), stages = ring_stages(blocks, bytes);
  const int64_t grid = static_cast<int64_t>(dev.sm_count) * blocks;
  const cudaError_t e =
      cudaFuncSetAttribute(ln_fwd_ring<DT, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(ln_fwd_ring<DT, NV>, static_cast<unsigned>(a.N < grid ? a.N : grid), T, stages * bytes, s, a,
                    stages);
}

template <int DT>
cudaError_t fwd_dt(const LnArgs& a, const Device& dev, cudaStream_t s) {
  constexpr int V = Fmt<DT>::VEC;
  const bool vec = a.xs1 == 1 && a.os1 == 1 && a.D % V == 0 && al16(a.x) && al16(a.out) &&
                   (a.N == 1 || (a.xs0 % V == 0 && a.os0 % V == 0));
  const unsigned warps_grid = static_cast<unsigned>((a.N + 7) / 8);
  const unsigned rows = static_cast<unsigned>(a.N);
  if (vec) {
    const int64_t n = a.D / V;
    if (n <= 32) return launch_pdl(ln_fwd_kernel<DT, V, 1, true>, warps_grid, 256, 0, s, a);
    if (n <= 64) return launch_pdl(ln_fwd_kernel<DT, V, 2, true>, warps_grid, 256, 0, s, a);
    if (n <= 256) return fwd_ring<DT, 1>(a, dev, s);
    if (n <= 512) return fwd_ring<DT, 2>(a, dev, s);
    if (n <= 2048) return fwd_ring<DT, 4>(a, dev, s);
  } else {
    if (a.D <= 256) return launch_pdl(ln_fwd_kernel<DT, 1, 8, true>, warps_grid, 256, 0, s, a);
    if (a.D <= 8192) return launch_pdl(ln_fwd_kernel<DT, 1, 8, false>, rows, threads(a.D, 8), 0, s, a);
  }
  return launch_pdl(ln_fwd_any<DT>, rows, 512, 0, s, a);
}

template <int DT, int NV, int MAXT>
cudaError_t bwd_ring(const LnBwdArgs& a, unsigned grid, cudaStream_t s) {
  const unsigned T = threads(a.D / Fmt<DT>::VEC, NV);
  const int64_t bytes = 2 * a.D * static_cast<int64_t>(sizeof(typename Fmt<DT>::E));
  // as many blocks as the grid puts on an SM of 152
  const int blocks = static_cast<int>((grid + 151) / 152), stages = ring_stages(blocks, bytes);
  const cudaError_t e =
      cudaFuncSetAttribute(ln_bwd_ring<DT, NV, MAXT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(ln_bwd_ring<DT, NV, MAXT>, grid, T, stages * bytes, s, a, stages);
}

template <int DT>
cudaError_t bwd_dt(const LnBwdArgs& a, cudaStream_t s) {
  if (a.N == 0) {  // no rows: the parameters' gradients are zero
    if (a.dw == nullptr && a.db == nullptr) return cudaSuccess;
    return launch_pdl(ln_bwd_reduce, static_cast<unsigned>((2 * a.D + 31) / 32), 1024, 0, s, a, 0);
  }
  constexpr int V = Fmt<DT>::VEC;
  const bool vec = a.xs1 == 1 && a.gs1 == 1 && a.dxs1 == 1 && a.D % V == 0 && al16(a.x) && al16(a.dout) &&
                   al16(a.dx) && (a.N == 1 || (a.xs0 % V == 0 && a.gs0 % V == 0 && a.dxs0 % V == 0));
  const unsigned grid = static_cast<unsigned>(ln_bwd_blocks(a.N, a.D));
  const size_t warp_sh = static_cast<size_t>(a.D) * 2 * 8 * sizeof(float);
  const size_t row_sh = 96 * sizeof(float);
  const int64_t n = a.D / V;
  cudaError_t e;
  if (vec && n <= 32)
    e = launch_pdl(ln_bwd_kernel<DT, V, 1, true, 256>, grid, 256, warp_sh, s, a);
  else if (!vec && a.D <= 128)
    e = launch_pdl(ln_bwd_kernel<DT, 1, 4, true, 256>, grid, 256, warp_sh, s, a);
  else if (vec && n <= 128)
    e = bwd_ring<DT, 1, 128>(a, grid, s);
  else if (vec && n <= 512)
    e = bwd_ring<DT, 2, 256>(a, grid, s);
  else if (vec && n <= 1024)
    e = bwd_ring<DT, 2, 512>(a, grid, s);
  else if (vec && n <= 2048)
    e = bwd_ring<DT, 4, 512>(a, grid, s);
  else if (!vec && a.D <= 4096)
    e = launch_pdl(ln_bwd_kernel<DT, 1, 4, false, 1024>, grid, threads(a.D, 4), row_sh, s, a);
  else
    e = launch_pdl(ln_bwd_any<DT>, grid, 512, 0, s, a);
  if (e != cudaSuccess || a.part == nullptr) return e;
  return launch_pdl(ln_bwd_reduce, static_cast<unsigned>((2 * a.D + 31) / 32), 1024, 0, s, a, static_cast<int>(grid));
}

}  // namespace

cudaError_t launch_ln_fwd(const LnArgs& a, Dtype dt, const Device& dev, cudaStream_t stream) {
  switch (dt) {
    case kF32: return fwd_dt<kF32>(a, dev, stream);
    case kF16: return fwd_dt<kF16>(a, dev, stream);
    case kBF16: return fwd_dt<kBF16>(a, dev, stream);
  }
  return cudaErrorInvalidValue;
}

// Multiples of 152 (the SMs of the device this is written for), so that the
// workspace's size depends on nothing but N and D: one wave of the ring
// kernels, whose blocks have a thread for every vector.
int64_t ln_bwd_blocks(int64_t N, int64_t D) {
  const int64_t rows = D <= 256 ? (N + 7) / 8 : N;
  const int64_t most = 152 * (D <= 1024 ? 6 : D <= 2048 ? 4 : D <= 4096 ? 2 : 1);
  return rows < most ? rows : most;
}

unsigned read_and_clear_fault_ln() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_fault, sizeof(v)) != cudaSuccess) return ~0u;
  if (v != 0 && cudaMemcpyToSymbol(g_fault, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

cudaError_t launch_ln_bwd(const LnBwdArgs& a, Dtype dt, cudaStream_t stream) {
  switch (dt) {
    case kF32: return bwd_dt<kF32>(a, stream);
    case kF16: return bwd_dt<kF16>(a, stream);
    case kBF16: return bwd_dt<kBF16>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ccv

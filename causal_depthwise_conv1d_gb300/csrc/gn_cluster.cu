// Group normalisation whose groups fit into the shared memory of a cluster:
// every input is read once.
//
// The blocks of a cluster share a group's positions; tensor copies bring a
// block's part [positions][C / G] into its shared memory, and all sweeps (mean,
// squares about it, backwards the sums of d and d xh, outputs) run over that.
// A thread keeps its vector of channels, so parameters stay in registers and the
// backward pass adds dw and db there.  Each block takes the mean of its own part
// and the squares about it; the cluster's blocks read one another's pairs and
// merge them in the same order (sums of n_k (mean_k - mean)^2: no difference of
// large sums).  What bounds it: HBM.
#include <cooperative_groups.h>
#include <cuda.h>

#include "ccv_common.cuh"
#include "ccv_tma.cuh"
#include "rec_internal.h"
#include "tensor_map.h"

namespace ccv {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned g_fault;

constexpr int kThreads = 256;
constexpr int kMaxCluster = 16;

// How a group is laid out: K blocks of a cluster with `boxes` x `high`
// positions each, channels in `parts` boxes of `wide`.
struct GnGeom {
  int cluster, boxes, high, parts, wide;
  int slots;  // backward: clusters side by side over the samples
  __host__ __device__ int rows() const { return boxes * high; }
};

struct Maps {
  CUtensorMap x, g;
};

__device__ __forceinline__ float pair_sum(uint64_t v) {
  float a, b;
  upk(v, a, b);
  return a + b;
}

template <int DT>
__device__ __forceinline__ void lds_pairs(const uint8_t* p, uint64_t* f) {
  constexpr int V = Fmt<DT>::VEC;
  float x[V];
  unpack16<DT>(lds128(p), x);
#pragma unroll
  for (int j = 0; j < V / 2; ++j) f[j] = pk(x[2 * j], x[2 * j + 1]);
}

// Sums over the block; every thread gets them.  `red` is not written again
// before another barrier has passed.
template <int NS>
__device__ __forceinline__ void block_sum(float (&v)[NS], float* red) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] += __shfl_xor_sync(kFullMask, v[i], m);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < NS; ++i) red[(threadIdx.x >> 5) * NS + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    v[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v[i] += red[w * NS + i];
  }
}

template <int DT, bool BWD>
__global__ void __launch_bounds__(kThreads, 3) gn_cluster_kernel(const GnArgs a, const GnGeom q,
                                                              const __grid_constant__ Maps maps) {
  constexpr int V = Fmt<DT>::VEC, H = V / 2;
  using E = typename Fmt<DT>::E;
  extern __shared__ __align__(128) uint8_t stage[];
  __shared__ uint64_t full;
  __shared__ float red0[8], red1[8], red2[16];
  __shared__ float2 part_stats, part_sums;
  __shared__ float fold[BWD ? kThreads * V : 1];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = static_cast<int>(cluster.block_rank());
  const int cgr = static_cast<int>(a.C / a.G), vecs = cgr / V, lanes = kThreads / vecs;
  const int vec = tid % vecs, lane = tid / vecs;  // a thread's vector of channels and its first position
  const bool on = lane < lanes;
  const int rows = q.rows();
  const int64_t s0 = static_cast<int64_t>(rank) * rows;
  const int n_rows = static_cast<int>(a.S - s0 < 0 ? 0 : a.S - s0 < rows ? a.S - s0 : rows);
  const int64_t task = blockIdx.x / q.cluster, g = task % a.G;
  const int per = q.wide / V;                       // vectors of a box's row
  const int plane = rows * cgr * static_cast<int>(sizeof(E));
  const uint8_t* mine = stage + (static_cast<size_t>(vec / per) * rows * q.wide + vec % per * V) * sizeof(E);
  const int pitch = q.wide * static_cast<int>(sizeof(E));

  if (tid == 0) {
    mbar_init(&full, 1);
    fence_barrier_init();
  }
  pdl_enter();
  __syncthreads();
  auto fill = [&](int64_t n) {
    mbar_arrive_expect_tx(&full, static_cast<uint32_t>((BWD ? 2 : 1) * plane));
    for (int p = 0; p < q.parts; ++p)
      for (int i = 0; i < q.boxes; ++i) {
        uint8_t* to = stage + (static_cast<size_t>(p) * rows + i * q.high) * pitch;
        const int c = static_cast<int>(g) * cgr + p * q.wide, t = static_cast<int>(s0) + i * q.high;
        tma_load_3d(to, &maps.x, c, t, static_cast<int>(n), &full);
        if (BWD) tma_load_3d(to + plane, &maps.g, c, t, static_cast<int>(n), &full);
      }
  };
  int64_t n = task / a.G;
  if (tid == 0 && n < a.N) fill(n);

  uint64_t w[H], b[H], dw[H], db[H];
  const int64_t ch = g * cgr + vec * V;
#pragma unroll
  for (int j = 0; j < H; ++j) {
    float x[2], y[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x[k] = a.w == nullptr ? 1.f : ld_param(a.w, (ch + 2 * j + k) * a.ws, a.wdt);
      y[k] = a.b == nullptr ? 0.f : ld_param(a.b, (ch + 2 * j + k) * a.bs, a.wdt);
    }
    w[j] = pk(x[0], x[1]), b[j] = pk(y[0], y[1]);
    dw[j] = db[j] = 0;
  }
  const float total = static_cast<float>(a.S) * static_cast<float>(cgr), inv = 1.f / total;
  const float mine_n = static_cast<float>(n_rows) * static_cast<float>(cgr);
  bool late = false;
  uint32_t parity = 0;
  for (; n < a.N; n += q.slots, parity ^= 1) {
    // A wait that runs out is recorded and the block goes on with what is there: the others of its cluster read
    // its shared memory.
    if (!mbar_wait(&full, parity)) {
      if (tid == 0) atomicOr(&g_fault, kFaultConsumerWait);
      late = true;
    }
    uint64_t acc = 0, f[H];
    if (on)
      for (int t = lane; t < n_rows; t += lanes) {
        lds_pairs<DT>(mine + t * pitch, f);
#pragma unroll
        for (int j = 0; j < H; ++j) acc = fadd2(acc, f[j]);
      }
    float s[1] = {pair_sum(acc)};
    block_sum(s, red0);
    float mean = n_rows > 0 ? s[0] / mine_n : 0.f;
    uint64_t minus = pk(-mean, -mean);
    acc = 0;
    if (on)
      for (int t = lane; t < n_rows; t += lanes) {
        lds_pairs<DT>(mine + t * pitch, f);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          f[j] = fadd2(f[j], minus);
          acc = ffma2(f[j], f[j], acc);
        }
      }
    s[0] = pair_sum(acc);
    block_sum(s, red1);
    float var = s[0];
    if (q.cluster > 1) {
      if (tid == 0) part_stats = make_float2(mean, var);
      cluster.sync();
      auto weight = [&](int k) {
        const int64_t left = a.S - static_cast<int64_t>(k) * rows;
        return static_cast<float>(left < 0 ? 0 : left < rows ? left : rows) * static_cast<float>(cgr);
      };
      float m = 0.f;
      for (int k = 0; k < q.cluster; ++k) m = fmaf(cluster.map_shared_rank(&part_stats, k)->x, weight(k) * inv, m);
      var = 0.f;
      for (int k = 0; k < q.cluster; ++k) {
        const float2 p = *cluster.map_shared_rank(&part_stats, k);
        var += fmaf((p.x - m) * (p.x - m), weight(k), p.y);
      }
      mean = m;
      minus = pk(-mean, -mean);
    }
    const float r = rsqrtf(fmaf(var, inv, a.eps));
    const uint64_t r2 = pk(r, r);
    if constexpr (!BWD) {
      E* out = static_cast<E*>(a.out) + n * a.os[0] + s0 * a.os[1] + ch;
      if (on)
        for (int t = lane; t < n_rows; t += lanes) {
          lds_pairs<DT>(mine + t * pitch, f);
          float o[V];
#pragma unroll
          for (int j = 0; j < H; ++j) {
            uint64_t z = ffma2(fmul2(fadd2(f[j], minus), r2), w[j], b[j]);
            if (a.silu) z = activate2_for<true, DT>(z);
            upk(z, o[2 * j], o[2 * j + 1]);
          }
          st16_stream(out + t * a.os[1], pack16<DT>(o));
        }
    } else {
      uint64_t a1 = 0, a2 = 0, d[H];
      if (on)
        for (int t = lane; t < n_rows; t += lanes) {
          lds_pairs<DT>(mine + t * pitch, f);
          lds_pairs<DT>(mine + plane + t * pitch, d);
#pragma unroll
          for (int j = 0; j < H; ++j) {
            f[j] = fmul2(fadd2(f[j], minus), r2);
            if (a.silu) d[j] = dz_pair<true>(ffma2(f[j], w[j], b[j]), d[j]);
            dw[j] = ffma2(d[j], f[j], dw[j]);
            db[j] = fadd2(db[j], d[j]);
            d[j] = fmul2(d[j], w[j]);
            a1 = fadd2(a1, d[j]);
            a2 = ffma2(d[j], f[j], a2);
          }
        }
      float c[2] = {pair_sum(a1), pair_sum(a2)};
      block_sum(c, red2);
      if (q.cluster > 1) {
        if (tid == 0) part_sums = make_float2(c[0], c[1]);
        cluster.sync();
        c[0] = c[1] = 0.f;
        for (int k = 0; k < q.cluster; ++k) {
          const float2 p = *cluster.map_shared_rank(&part_sums, k);
          c[0] += p.x, c[1] += p.y;
        }
      }
      const float c1 = -r * (c[0] * inv), c2 = -r * (c[1] * inv);
      const uint64_t k1 = pk(c1, c1), k2 = pk(c2, c2);
      E* dx = static_cast<E*>(a.dx) + n * a.dxs[0] + s0 * a.dxs[1] + ch;
      if (on)
        for (int t = lane; t < n_rows; t += lanes) {
          lds_pairs<DT>(mine + t * pitch, f);
          lds_pairs<DT>(mine + plane + t * pitch, d);
          float o[V];
#pragma unroll
          for (int j = 0; j < H; ++j) {
            f[j] = fmul2(fadd2(f[j], minus), r2);
            if (a.silu) d[j] = dz_pair<true>(ffma2(f[j], w[j], b[j]), d[j]);
            d[j] = fmul2(d[j], w[j]);
            upk(ffma2(d[j], r2, ffma2(f[j], k2, k1)), o[2 * j], o[2 * j + 1]);
          }
          st16_stream(dx + t * a.dxs[1], pack16<DT>(o));
        }
      __syncthreads();  // the stage has been read
      if (tid == 0 && n + q.slots < a.N) {
        fence_proxy_async_smem();
        fill(n + q.slots);
      }
    }
  }
  if constexpr (BWD) {
    if (a.part != nullptr) {
      // a block's positions in order, one partial sum a block
      float* part = a.part + (task / a.G * q.cluster + rank) * 2 * a.C;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
        if (on)
#pragma unroll
          for (int j = 0; j < H; ++j) {
            float u, v;
            upk(which == 0 ? dw[j] : db[j], u, v);
            fold[tid * V + 2 * j] = u;
            fold[tid * V + 2 * j + 1] = v;
          }
        __syncthreads();
        for (int c = tid; c < cgr; c += kThreads) {
          float v = 0.f;
          for (int k = 0; k < lanes; ++k) v += fold[k * cgr + c];
          part[which * a.C + g * cgr + c] = v;
        }
      }
    }
  }
  if (late) mbar_wait(&full, parity ^ 1);  // the copies in flight
  if (q.cluster > 1) cluster.sync();  // nobody reads this block's shared memory any more
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Bytes of shared memory that leave room for three, two or one blocks an SM.
constexpr int64_t kSmem[3] = {64 * 1024, 104 * 1024, 212 * 1024};

// False where a group does not fit.
bool geometry(int64_t N, int64_t S, int64_t C, int64_t G, int64_t esize, bool bwd, GnGeom* q) {
  const int64_t v = 16 / esize, cgr = C / G;
  if (cgr % v != 0 || cgr / v > kThreads || S > (1 << 24)) return false;
  q->parts = 1;
  while (cgr % q->parts != 0 || cgr / q->parts > 256 || cgr / q->parts % v != 0) ++q->parts;
  q->wide = static_cast<int>(cgr / q->parts);
  for (const int64_t room : kSmem)
    for (int k = 1; k <= kMaxCluster; k *= 2) {
      const int64_t rows = up((S + k - 1) / k, 8), boxes = (rows + 255) / 256, high = up((rows + boxes - 1) / boxes, 8);
      if (boxes * high * cgr * esize * (bwd ? 2 : 1) > room) continue;
      q->cluster = k, q->boxes = static_cast<int>(boxes), q->high = static_cast<int>(high);
      // backward: a wave of clusters, and no more partial sums than samples
      int64_t slots = bwd ? (152 * 3 + G * k - 1) / (G * k) : N;
      if (slots > N) slots = N;
      q->slots = static_cast<int>(slots < 1 ? 1 : slots);
      return true;
    }
  return false;
}

template <int DT, bool BWD>
cudaError_t launch(const GnArgs& a, const GnGeom& q, cudaStream_t s) {
  constexpr Dtype dt = static_cast<Dtype>(DT);
  Maps maps = {};
  const int64_t box[2] = {q.wide, q.high};
  if (!tensor_map3(&maps.x, a.x, a.xs, a.N, a.S, a.C, box, dt) ||
      (BWD && !tensor_map3(&maps.g, a.dout, a.gs, a.N, a.S, a.C, box, dt)))
    return cudaErrorInvalidValue;
  const int64_t bytes = static_cast<int64_t>(q.rows()) * (a.C / a.G) * (DT == kF32 ? 4 : 2) * (BWD ? 2 : 1);
  cudaError_t e = cudaFuncSetAttribute(gn_cluster_kernel<DT, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmem[2]));
  if (e == cudaSuccess && q.cluster > 8)
    e = cudaFuncSetAttribute(gn_cluster_kernel<DT, BWD>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.G * q.slots * q.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(q.cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, gn_cluster_kernel<DT, BWD>, a, q, maps);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

bool stores(const void* p, const int64_t* s, int64_t N, int64_t S, int64_t v) {
  return s[2] == 1 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && (N == 1 || s[0] % v == 0) && (S == 1 || s[1] % v == 0);
}

}  // namespace

bool gn_cluster_eligible(const GnArgs& a, Dtype dt, bool bwd) {
  const int64_t e = dt == kF32 ? 4 : 2, v = 16 / e;
  GnGeom q = {};
  if (!tensor_map_eligible(a.x, a.xs, a.N, a.S, a.C, dt) || !geometry(a.N, a.S, a.C, a.G, e, bwd, &q)) return false;
  if (static_cast<__int128>(a.G) * q.slots * q.cluster > 0x7fffffff) return false;
  return bwd ? tensor_map_eligible(a.dout, a.gs, a.N, a.S, a.C, dt) && stores(a.dx, a.dxs, a.N, a.S, v)
             : stores(a.out, a.os, a.N, a.S, v);
}

int64_t gn_cluster_parts(int64_t N, int64_t S, int64_t C, int64_t G, int64_t esize) {
  GnGeom q = {};
  return geometry(N, S, C, G, esize, true, &q) ? static_cast<int64_t>(q.slots) * q.cluster : 0;
}

cudaError_t launch_gn_cluster(const GnArgs& a, Dtype dt, bool bwd, cudaStream_t s) {
  GnGeom q = {};
  if (!geometry(a.N, a.S, a.C, a.G, dt == kF32 ? 4 : 2, bwd, &q)) return cudaErrorInvalidValue;
  switch (dt) {
    case kF32: return bwd ? launch<kF32, true>(a, q, s) : launch<kF32, false>(a, q, s);
    case kF16: return bwd ? launch<kF16, true>(a, q, s) : launch<kF16, false>(a, q, s);
    case kBF16: return bwd ? launch<kBF16, true>(a, q, s) : launch<kBF16, false>(a, q, s);
  }
  return cudaErrorInvalidValue;
}

unsigned read_and_clear_fault_gn() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_fault, sizeof(v)) != cudaSuccess) return ~0u;
  if (v != 0 && cudaMemcpyToSymbol(g_fault, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace ccv

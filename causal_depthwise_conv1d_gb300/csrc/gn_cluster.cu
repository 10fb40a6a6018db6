// Group normalisation whose groups fit into the shared memory of a cluster: x
// is read once.
//
// The blocks of a cluster share a group's positions; tensor copies bring a
// block's part [positions][C / G] of x into its shared memory in two boxes, and
// all sweeps (statistics, backwards the sums of d and d xh, outputs) run over
// that: the first takes the boxes as they arrive, the last hands each box back
// for the next group's copy as soon as it has been used.  A thread keeps its
// vector of channels, so parameters stay in registers and the backward pass adds
// dw and db there over all samples.  A thread takes its squares about its mean from
// one sweep, as a difference whose loss is bounded (see the loop); threads' and
// blocks' means and squares, which the cluster's blocks send one another, are merged
// in the same order as sums of n_k (mean_k - mean)^2, without differences of large sums.
//
// The backward pass reads dout in both of its sweeps, the second time from the
// L2 cache: with dout in the stage as well, a group of 2048 x 128 bf16 took
// sixteen blocks instead of eight (8 x 2048 x 4096 194 us, now 142).  What costs
// time beside the bytes is that a block's phases follow one another: sums and
// exchange about 5000 cycles, the output sweep 7000, of which SiLU's reciprocals
// and exponentials are 2600 (silu_pair; with a reciprocal for each element the
// forward pass took 89 instead of 77 us for 8 x 2048 x 5120).
#include <cooperative_groups.h>
#include <cuda.h>

#include <type_traits>

#include "ccv_common.cuh"
#include "ccv_tma.cuh"
#include "rec_internal.h"
#include "rec_pairs.cuh"
#include "tensor_map.h"

namespace ccv {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned g_fault;

constexpr int kThreads = 256;
constexpr int kMaxCluster = 16;
constexpr int kBoxes = 2;  // boxes of a block's part, at most

// How a group is laid out: K blocks of a cluster with `boxes` x `high`
// positions each, channels in `parts` boxes of `wide`.
struct GnGeom {
  int cluster, boxes, high, parts, wide;
  int slots;  // clusters side by side over the samples of a group
  __host__ __device__ int rows() const { return boxes * high; }
};

template <int DT>
__device__ __forceinline__ void lds_pairs(const uint8_t* p, uint64_t* f) {
  unpack_pairs<DT>(lds128(p), f);
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
    for (int i = 0; i < NS; ++i) red[i * (kThreads / 32) + (threadIdx.x >> 5)] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    v[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w += 4) {
      const float4 x = *reinterpret_cast<const float4*>(red + i * (kThreads / 32) + w);
      v[i] += (x.x + x.y) + (x.z + x.w);
    }
  }
}

// A pair of this block for slot `slot` and barrier `bar` of another block of the
// cluster (their addresses here name the same places there): it arrives with
// the barrier's transaction count, no fence and no cluster-wide barrier.
__device__ __forceinline__ void send_pair(float2* slot, uint64_t* bar, int rank, float2 v) {
  uint32_t to, at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(slot)), "r"(rank));
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(to),
               "l"(pk(v.x, v.y)), "r"(at)
               : "memory");
}

// Sum over the first 16 lanes (the upper ones hold the same), in every lane.
__device__ __forceinline__ float ranks_sum(float v) {
#pragma unroll
  for (int m = 8; m > 0; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
  return v;
}

template <int DT, bool BWD>
__global__ void __launch_bounds__(kThreads, 2)
    gn_cluster_kernel(const GnArgs a, const GnGeom q, const __grid_constant__ CUtensorMap map) {
  constexpr int V = Fmt<DT>::VEC, H = V / 2;
  using E = typename Fmt<DT>::E;
  extern __shared__ __align__(128) uint8_t stage[];
  __shared__ uint64_t full[kBoxes];
  __shared__ __align__(16) float red0[kThreads / 32], red1[kThreads / 32], red2[kThreads / 16];
  // what the cluster's blocks send one another: two exchanges in turn, so that one is read while the next arrives
  __shared__ float2 pairs[2][kMaxCluster];
  __shared__ uint64_t sent[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = static_cast<int>(cluster.block_rank());
  const int cgr = static_cast<int>(a.C / a.G), vecs = cgr / V, lanes = kThreads / vecs;
  const int vec = tid % vecs, lane = tid / vecs;  // a thread's vector of channels and its first position
  const int rows = q.rows();
  const int64_t s0 = static_cast<int64_t>(rank) * rows;
  const int n_rows = static_cast<int>(a.S - s0 < 0 ? 0 : a.S - s0 < rows ? a.S - s0 : rows);
  const int last = lane < lanes ? n_rows : 0;  // this thread's positions end here
  const int64_t task = blockIdx.x / q.cluster, g = task % a.G;
  const int per = q.wide / V;  // vectors of a box's row
  const int pitch = q.wide * static_cast<int>(sizeof(E)), hop = lanes * pitch;
  const uint8_t* mine = stage + static_cast<size_t>(vec / per) * rows * pitch + vec % per * 16;

  if (tid == 0) {
    for (int i = 0; i < q.boxes; ++i) mbar_init(&full[i], 1);
    mbar_init(&sent[0], 1);
    mbar_init(&sent[1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_barrier_init();
  }
  pdl_enter();
  if (q.cluster > 1)
    cluster.sync();  // the others' barriers are there
  else
    __syncthreads();
  auto fill = [&](int64_t n, int i) {
    mbar_arrive_expect_tx(&full[i], static_cast<uint32_t>(q.high * cgr * static_cast<int>(sizeof(E))));
    for (int p = 0; p < q.parts; ++p) {
      uint8_t* to = stage + (static_cast<size_t>(p) * rows + i * q.high) * pitch;
      const int c = static_cast<int>(g) * cgr + p * q.wide, t = static_cast<int>(s0) + i * q.high;
      tma_load_3d(to, &map, c, t, static_cast<int>(n), &full[i]);
    }
  };
  int64_t n = task / a.G;
  if (tid == 0)
    for (int i = 0; i < q.boxes; ++i) fill(n, i);

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
  const float inv = 1.f / (static_cast<float>(a.S) * static_cast<float>(cgr));
  const float mine_inv = n_rows > 0 ? 1.f / (static_cast<float>(n_rows) * static_cast<float>(cgr)) : 0.f;
  const float cnt = last > lane ? static_cast<float>((last - lane + lanes - 1) / lanes * V) : 0.f;  // this thread's
  const float cnt_inv = cnt > 0.f ? 1.f / cnt : 0.f;
  // the block of the cluster that this lane reads, and its number of elements
  const int peer = tid & 15;
  float peer_n = 0.f;
  if (peer < q.cluster) {
    const int64_t left = a.S - static_cast<int64_t>(peer) * rows;
    peer_n = static_cast<float>(left < 0 ? 0 : left < rows ? left : rows) * static_cast<float>(cgr);
  }
  bool late = false;
  uint32_t parity = 0, rounds = 0;
  // Sends v to every block of the cluster; this lane's peer's pair.  A block sends for the second time after this
  // one's when all others have sent once more, and so have read these.
  auto exchange = [&](float2 v) -> float2 {
    const uint32_t k = rounds & 1, ph = rounds >> 1 & 1;
    ++rounds;
    if (tid == 0) mbar_arrive_expect_tx(&sent[k], static_cast<uint32_t>(q.cluster) * 8u);
    if (tid < q.cluster) send_pair(&pairs[k][rank], &sent[k], tid, v);
    if (!late && !mbar_wait(&sent[k], ph)) {
      if (tid == 0) atomicOr(&g_fault, kFaultConsumerWait);
      late = true;
    }
    return peer < q.cluster ? pairs[k][peer] : make_float2(0.f, 0.f);
  };
  for (; n < a.N; n += q.slots, parity ^= 1) {
    // One sweep: sums of x - shift and of its square, the shift being the mean of the thread's first vector.  As that
    // is part of the data, the squares about the thread's mean are at least V / n of those about the shift for n
    // elements, so the difference below loses no more than log2(n / V) bits, whatever the values.
    uint64_t f[H], minus = 0, acc = 0, sq = 0;
    float shift = 0.f;
    for (int i = 0, t = lane; i < q.boxes; ++i) {
      // A wait that runs out is recorded and the block goes on with what is there: the others of its cluster write
      // into its shared memory.  One warp polls and the others wait at the barrier.
      if (tid < 32 && !late && !mbar_wait(&full[i], parity)) {
        if (tid == 0) atomicOr(&g_fault, kFaultConsumerWait);
        late = true;
      }
      __syncthreads();
      const int end = last < (i + 1) * q.high ? last : (i + 1) * q.high;
      const uint8_t* at = mine + t * pitch;
      if (t == lane && t < end) {
        lds_pairs<DT>(at, f);
        acc = f[0];
#pragma unroll
        for (int j = 1; j < H; ++j) acc = fadd2(acc, f[j]);
        shift = pair_sum(acc) * (1.f / V);
        minus = pk(-shift, -shift);
        acc = 0;
      }
#pragma unroll 4
      for (; t < end; t += lanes, at += hop) {
        lds_pairs<DT>(at, f);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          f[j] = fadd2(f[j], minus);
          acc = fadd2(acc, f[j]);
          sq = ffma2(f[j], f[j], sq);
        }
      }
    }
    const float off = pair_sum(acc) * cnt_inv;  // of this thread's mean from the shift
    float mean = shift + off;
    float s[1] = {mean * cnt};
    block_sum(s, red0);
    const float own = s[0] * mine_inv;
    s[0] = cnt > 0.f ? fmaf((mean - own) * (mean - own), cnt, fmaf(-off * off, cnt, pair_sum(sq))) : 0.f;
    block_sum(s, red1);
    mean = own;
    float var = s[0];
    if (q.cluster > 1) {
      const float2 p = exchange(make_float2(mean, var));
      mean = ranks_sum(p.x * (peer_n * inv));
      var = ranks_sum(fmaf((p.x - mean) * (p.x - mean), peer_n, p.y));
    }
    minus = pk(-mean, -mean);
    const float r = rsqrtf(fmaf(var, inv, a.eps));
    const uint64_t r2 = pk(r, r);
    float c[2] = {0.f, 0.f};
    if constexpr (BWD) {
      uint64_t a1 = 0, a2 = 0, d[H];
      auto sums = [&](auto silu) {
        const uint8_t* at = mine + lane * pitch;
        const E* gy = static_cast<const E*>(a.dout) + n * a.gs[0] + (s0 + lane) * a.gs[1] + ch;
#pragma unroll 4
        for (int t = lane; t < last; t += lanes, at += hop, gy += lanes * a.gs[1]) {
          lds_pairs<DT>(at, f);
          unpack_pairs<DT>(__ldg(reinterpret_cast<const uint4*>(gy)), d);
#pragma unroll
          for (int j = 0; j < H; ++j) {
            f[j] = fmul2(fadd2(f[j], minus), r2);
            if constexpr (decltype(silu)::value) d[j] = silu_grad_pair2(ffma2(f[j], w[j], b[j]), d[j]);
            dw[j] = ffma2(d[j], f[j], dw[j]);
            db[j] = fadd2(db[j], d[j]);
            d[j] = fmul2(d[j], w[j]);
            a1 = fadd2(a1, d[j]);
            a2 = ffma2(d[j], f[j], a2);
          }
        }
      };
      if (a.silu)
        sums(std::true_type{});
      else
        sums(std::false_type{});
      c[0] = pair_sum(a1), c[1] = pair_sum(a2);
      block_sum(c, red2);
      if (q.cluster > 1) {
        const float2 p = exchange(make_float2(c[0], c[1]));
        c[0] = ranks_sum(p.x), c[1] = ranks_sum(p.y);
      }
    }
    const float c1 = -r * (c[0] * inv), c2 = -r * (c[1] * inv);
    const uint64_t k1 = pk(c1, c1), k2 = pk(c2, c2);
    uint64_t wr[H];
    if (!BWD)
#pragma unroll
      for (int j = 0; j < H; ++j) wr[j] = fmul2(w[j], r2);
    const int64_t step = BWD ? a.dxs[1] : a.os[1];
    E* out = (BWD ? static_cast<E*>(a.dx) + n * a.dxs[0] : static_cast<E*>(a.out) + n * a.os[0]) + (s0 + lane) * step + ch;
    auto write = [&](auto silu) {
      for (int i = 0, t = lane; i < q.boxes; ++i) {
        const int end = last < (i + 1) * q.high ? last : (i + 1) * q.high;
        const uint8_t* at = mine + t * pitch;
        const E* gy = BWD ? static_cast<const E*>(a.dout) + n * a.gs[0] + (s0 + t) * a.gs[1] + ch : nullptr;
#pragma unroll 4
        for (; t < end; t += lanes, at += hop, out += lanes * step, gy += lanes * a.gs[1]) {
          float o[V];
          lds_pairs<DT>(at, f);
          if constexpr (BWD) {
            uint64_t d[H];
            unpack_pairs<DT>(__ldg(reinterpret_cast<const uint4*>(gy)), d);
#pragma unroll
            for (int j = 0; j < H; ++j) {
              f[j] = fmul2(fadd2(f[j], minus), r2);
              if constexpr (decltype(silu)::value) d[j] = silu_grad_pair2(ffma2(f[j], w[j], b[j]), d[j]);
              d[j] = fmul2(d[j], w[j]);
              upk(ffma2(d[j], r2, ffma2(f[j], k2, k1)), o[2 * j], o[2 * j + 1]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < H; ++j) {
              uint64_t z = ffma2(fadd2(f[j], minus), wr[j], b[j]);
              if constexpr (decltype(silu)::value) z = silu_pair(z);
              upk(z, o[2 * j], o[2 * j + 1]);
            }
          }
          st16_stream(out, pack16<DT>(o));
        }
        if (n + q.slots < a.N) {
          __syncthreads();  // the box has been read
          if (tid == 0) {
            fence_proxy_async_smem();
            fill(n + q.slots, i);
          }
        }
      }
    };
    if (a.silu)
      write(std::true_type{});
    else
      write(std::false_type{});
  }
  if (late)
    for (int i = 0; i < q.boxes; ++i) mbar_wait(&full[i], parity ^ 1);  // the copies in flight
  if constexpr (BWD) {
    if (a.part != nullptr) {
      // a block's positions in order, one partial sum a block; the stage is free now
      float* part = a.part + (task / a.G * q.cluster + rank) * 2 * a.C;
      float* fold = reinterpret_cast<float*>(stage);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
        if (lane < lanes)
#pragma unroll
          for (int j = 0; j < H; ++j) {
            float u, v;
            upk(which == 0 ? dw[j] : db[j], u, v);
            fold[tid * V + 2 * j] = u;
            fold[tid * V + 2 * j + 1] = v;
          }
        __syncthreads();
        for (int k = tid; k < cgr; k += kThreads) {
          float v = 0.f;
          for (int i = 0; i < lanes; ++i) v += fold[i * cgr + k];
          part[which * a.C + g * cgr + k] = v;
        }
      }
    }
  }
  if (q.cluster > 1) cluster.sync();  // nobody writes into this block's shared memory any more
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Bytes of a block's stage (the backward pass folds its sums there too).
int64_t stage_bytes(const GnGeom& q, int64_t cgr, int64_t esize, bool bwd) {
  const int64_t data = q.rows() * cgr * esize, fold = bwd ? kThreads * 16 / esize * 4 : 0;
  return data > fold ? data : fold;
}

constexpr int64_t kSmem = 216 * 1024;  // of a stage, at most

// False where a group does not fit.
bool geometry(int64_t N, int64_t S, int64_t C, int64_t G, int64_t esize, bool bwd, GnGeom* q) {
  const int64_t v = 16 / esize, cgr = C / G, vecs = cgr / v;
  if (cgr % v != 0 || vecs > 256 || S > (1 << 24) || N > 0x7fffffff) return false;
  q->parts = 1;
  while (cgr % q->parts != 0 || cgr / q->parts > 256 || cgr / q->parts % v != 0) ++q->parts;
  q->wide = static_cast<int>(cgr / q->parts);
  auto fits = [&](int k, int64_t room) {
    // boxes of at least 8 and at most 256 positions
    const int64_t share = (S + k - 1) / k, high = up((share + kBoxes - 1) / kBoxes, 8);
    if (high > 256) return false;
    q->cluster = k, q->high = static_cast<int>(high), q->boxes = static_cast<int>((share + high - 1) / high);
    return stage_bytes(*q, cgr, esize, bwd) <= room;
  };
  // Clusters of at most eight blocks with two blocks an SM, else of sixteen, else one block an SM.
  constexpr struct {
    int least, most;
    int64_t room;
    int per_sm;
  } kTry[] = {{1, 8, 108 * 1024, 2}, {16, 16, 108 * 1024, 2}, {1, 8, kSmem, 1}, {16, 16, kSmem, 1}};
  for (const auto& c : kTry)
    for (int k = c.least; k <= c.most; k *= 2) {
      if (!fits(k, c.room)) continue;
      // as many clusters of a group side by side as make few rounds on 152 SMs
      const int64_t most = 152 * c.per_sm / k;
      int64_t best = 0;
      q->slots = 1;
      auto rate = [&](int64_t n) {
        const int64_t rounds = (n * G + most - 1) / most * ((N + n - 1) / n);
        if (best == 0 || rounds < best) best = rounds, q->slots = static_cast<int>(n);
      };
      rate(1);
      if (G < most) rate(most / G < N ? most / G : N);
      return true;
    }
  return false;
}

template <int DT, bool BWD>
cudaError_t launch(const GnArgs& a, const GnGeom& q, cudaStream_t s) {
  CUtensorMap map = {};
  const int64_t box[2] = {q.wide, q.high};
  if (!tensor_map3(&map, a.x, a.xs, a.N, a.S, a.C, box, static_cast<Dtype>(DT))) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(gn_cluster_kernel<DT, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmem));
  if (e == cudaSuccess && q.cluster > 8)
    e = cudaFuncSetAttribute(gn_cluster_kernel<DT, BWD>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.G * q.slots * q.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(stage_bytes(q, a.C / a.G, DT == kF32 ? 4 : 2, BWD));
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(q.cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, gn_cluster_kernel<DT, BWD>, a, q, map);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

bool vectors(const void* p, const int64_t* s, int64_t N, int64_t S, int64_t v) {
  return s[2] == 1 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && (N == 1 || s[0] % v == 0) && (S == 1 || s[1] % v == 0);
}

}  // namespace

bool gn_cluster_eligible(const GnArgs& a, Dtype dt, bool bwd) {
  const int64_t e = dt == kF32 ? 4 : 2, v = 16 / e;
  GnGeom q = {};
  if (!tensor_map_eligible(a.x, a.xs, a.N, a.S, a.C, dt) || !geometry(a.N, a.S, a.C, a.G, e, bwd, &q)) return false;
  if (static_cast<__int128>(a.G) * q.slots * q.cluster > 0x7fffffff) return false;
  return bwd ? vectors(a.dout, a.gs, a.N, a.S, v) && vectors(a.dx, a.dxs, a.N, a.S, v) : vectors(a.out, a.os, a.N, a.S, v);
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

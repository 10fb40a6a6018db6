// Gated linear recurrence over whole sequences: one pass, every input read and
// every output written once.
//
// A block of four warps takes tiles of 64 tokens x 64 channels; a warp has 16
// tokens, a lane two channels.  Tensor copies bring the next tile's x and gates
// into shared memory while the present one is worked on.  A warp computes its
// tokens' decays and inputs into registers and their (A, H); after the tile's
// one barrier every warp gets the state before the tile (see glr_tile.cuh), the
// first one publishes the state after it, and each runs its tokens, writes them
// over x in the stage and stores them as a box.  So a state costs no second
// pass over the inputs, however few channels there are to split the device by.
//
// bf16, 8192 x 5120 83 us (4.1 TB/s of 336 MB), 8 x 2048 x 5120 in five packed
// sequences 128 us (5.3 TB/s); 30 instructions an element at 57 % of the issue slots
// of 16 warps an SM.  Warps with a rate above 0.85 take the exponential of the decay
// too: 35 instructions at 63 %, 87 and 135 us.  Runs of 16 tokens: with eight 115 and
// 164 us; three blocks an SM instead of four 98 and 149.
#include <type_traits>

#include "glr_tile.cuh"

namespace ccv {
namespace {

__device__ unsigned g_fault;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = kGlrT / kWarps;  // tokens of a warp
constexpr int kStages = 2;
constexpr int kPublisher = 1;  // the warp that publishes (the first one starts the copies)

struct Maps {
  CUtensorMap x, p, q, out;
};

template <int DT>
constexpr int plane_bytes() {
  return kGlrT * kGlrC * (DT == kF32 ? 4 : 2);
}

struct __align__(16) Shared {
  float4 pair[2][kWarps][32];
  uint64_t full[kStages];
  GlrPlace place[kStages];
  float2 carried[kStages][32];  // serial: the state after the tile before
};

// The runs' maps, first run first, as one.
__device__ __forceinline__ float4 joined(const float4 (*runs)[32], int lane) {
  float4 m = runs[0][lane];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    const float4 v = runs[w][lane];
    glr_join(v.x, v.y, m.x, m.y);
    glr_join(v.z, v.w, m.z, m.w);
  }
  m.x = glr_positive(m.x), m.z = glr_positive(m.z);
  return m;
}

template <int DT, bool SEQ, bool TMA>
__global__ void __launch_bounds__(kThreads, DT == kF32 ? 2 : 4)
    glr_fwd_kernel(const GlrArgs a, const GlrTiles g, const GlrChain chain, const __grid_constant__ Maps maps) {
  constexpr int PLANE = plane_bytes<DT>();
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool chained = g.levels > 1 && !g.serial;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sh.full[s], 1);
    fence_barrier_init();
  }
  pdl_enter();
  __syncthreads();

  // Thread 0 draws tiles and starts their copies.
  int drawn = 0;
  auto draw = [&]() -> int {
    if (chained) return static_cast<int>(atomicAdd(chain.ticket, 1u) + 1u);
    return glr_serial_tile(g, drawn++);
  };
  auto fill = [&](int s, int t) {
    GlrPlace p;
    p.tile = t;
    p.level = glr_div(t, g.ncols_inv), p.col = t - p.level * g.ncols;
    p.b = glr_div(p.col, g.nct_inv), p.c0 = (p.col - p.b * g.nct) * kGlrC;
    sh.place[s] = p;
    if (!TMA || t >= g.total) {
      mbar_arrive(&sh.full[s]);
      return;
    }
    uint8_t* st = stages + s * 3 * PLANE;
    mbar_arrive_expect_tx(&sh.full[s], 3 * PLANE);
    tma_load_3d(st, &maps.x, p.c0, p.level * kGlrT, p.b, &sh.full[s]);
    tma_load_3d(st + PLANE, &maps.p, p.c0, p.level * kGlrT, p.b, &sh.full[s]);
    tma_load_3d(st + 2 * PLANE, &maps.q, p.c0, p.level * kGlrT, p.b, &sh.full[s]);
  };
  int next = g.total;
  if (tid == 0) {
    fill(0, draw());
    if (!g.one) next = draw();
  }

  for (int it = 0;; ++it) {
    const int s = it & 1;
    if (it == 1 && g.one) break;
    if (!mbar_wait(&sh.full[s], (it >> 1) & 1)) {
      if (lane == 0) atomicOr(&g_fault, kFaultConsumerWait);
      mbar_wait(&sh.full[s], (it >> 1) & 1);  // the one copy in flight, again with a limit
      break;
    }
    const GlrPlace at = sh.place[s];
    if (at.tile >= g.total) break;
    const int level = at.level, b = at.b, c = at.c0 + 2 * lane;
    const int64_t t0 = static_cast<int64_t>(level) * kGlrT + warp * kRun;
    const bool in0 = c < a.C, in1 = c + 1 < a.C;
    const int64_t left = a.L - t0;
    const int n = left >= kRun ? kRun : left > 0 ? static_cast<int>(left) : 0;  // tokens of this warp
    uint4 before = make_uint4(kSlotEmpty, 0u, 0u, 0u);
    if (chained && level > 0) before = ld_slot(glr_slot(chain, at.tile - g.ncols, lane));  // it may be there already
    unsigned reset = 0;  // bit j: a sequence starts at the warp's token j
    if constexpr (SEQ) {
      bool start = false;
      if (lane < n && t0 + lane > 0) {
        const int32_t* id = a.seq + b * a.ss[0] + (t0 + lane) * a.ss[1];
        start = id[0] != id[-a.ss[1]];
      }
      reset = __ballot_sync(kFullMask, start);
    }
    const float rate0 = in0 ? __ldg(a.rate + c * a.rs) : 0.f, rate1 = in1 ? __ldg(a.rate + (c + 1) * a.rs) : 0.f;
    const uint64_t rate = pk(-rate0, -rate1);

    uint64_t dec[kRun], in[kRun];
    uint8_t* st = stages + s * 3 * PLANE + warp * (PLANE / kWarps);  // this warp's rows
    auto gates = [&](auto near) {
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        uint64_t x, p, q;
        if constexpr (TMA) {
          x = glr_lds<DT>(st, j, lane);
          p = glr_lds<DT>(st + PLANE, j, lane);
          q = glr_lds<DT>(st + 2 * PLANE, j, lane);
        } else {
          const bool on = j < n;
          const int64_t t = t0 + j;
          x = glr_ldg<DT>(a.x, b * a.xs[0] + t * a.xs[1] + c * a.xs[2], a.xs[2], on && in0, on && in1);
          p = glr_ldg<DT>(a.p, b * a.ps[0] + t * a.ps[1] + c * a.ps[2], a.ps[2], on && in0, on && in1);
          q = glr_ldg<DT>(a.q, b * a.qs[0] + t * a.qs[1] + c * a.qs[2], a.qs[2], on && in0, on && in1);
        }
        uint64_t r, i, e, m2;
        glr_sigmoid2(p, r, e);
        glr_sigmoid2(q, i, e);
        glr_decay2<decltype(near)::value>(fmul2(rate, r), dec[j], m2);
        float u, v;
        upk(m2, u, v);
        in[j] = fmul2(pk(sqrt_approx(u), sqrt_approx(v)), fmul2(i, x));
      }
    };
    if (__all_sync(kFullMask, rate0 <= -kGlrSeries && rate1 <= -kGlrSeries))
      gates(std::true_type{});
    else
      gates(std::false_type{});
    if (n < kRun)
#pragma unroll
      for (int j = 0; j < kRun; ++j)
        if (j >= n) dec[j] = pk(1.f, 1.f), in[j] = 0;
    uint64_t A = dec[0], H = in[0];
    // Tensor copies: runs without a start as code of their own (128 us instead of 131 for the packed batch above); with
    // plain loads that spills more registers (8 x 2048 x 5001, packed, 372 us instead of 320).
    if (!SEQ || (TMA && reset == 0)) {
#pragma unroll
      for (int j = 1; j < kRun; ++j) {
        A = fmul2(A, dec[j]);
        H = ffma2(dec[j], H, in[j]);
      }
    } else {
#pragma unroll
      for (int j = 1; j < kRun; ++j) {
        A = fmul2(A, dec[j]);
        H = reset >> j & 1 ? in[j] : ffma2(dec[j], H, in[j]);
      }
    }
    float4 (*pairs)[32] = sh.pair[s];
    pairs[warp][lane] = glr_run(A, H, SEQ && reset != 0);
    if (TMA && lane == 0) bulk_wait_read<>();  // the box of the tile before has left its stage
    __syncthreads();  // pairs are there, the other stage is free
    if (tid == 0 && !g.one) {
      fence_proxy_async_smem();
      fill(s ^ 1, next);
      if (next < g.total) next = draw();
    }

    float2 h2 = make_float2(0.f, 0.f);
    if (level == 0) {
      if (a.s0 != nullptr) {
        const float* p = a.s0 + b * a.s0s[0] + c * a.s0s[1];
        h2 = make_float2(in0 ? p[0] : 0.f, in1 ? p[a.s0s[1]] : 0.f);
      }
    } else if (g.serial) {
      h2 = sh.carried[s ^ 1][lane];
    } else if (__all_sync(kFullMask, before.x == kSlotState)) {
      h2 = glr_slot_state(before);
    } else {
      if (warp == kPublisher && level + 1 < g.levels) glr_put_pair(chain, at.tile, lane, joined(pairs, lane));
      if (!glr_look_back(chain, g, level, at.col, lane, h2)) {
        if (lane == 0) atomicOr(&g_fault, kFaultConsumerWait);
        h2 = make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));  // no state: nothing that passes for one
      }
    }
    if (warp == kPublisher) {
      if (level + 1 < g.levels) {
        const float4 m = joined(pairs, lane);
        const float2 after = make_float2(glr_map(m.x, m.y, h2.x), glr_map(m.z, m.w, h2.y));
        if (g.serial)
          sh.carried[s][lane] = after;
        else
          glr_put_state(chain, at.tile, lane, after);
      }
      if (a.cs != nullptr) {
        float* p = a.cs + b * a.css[0] + level * a.css[1] + c * a.css[2];
        if (in0) p[0] = h2.x;
        if (in1) p[a.css[2]] = h2.y;
      }
    }
    for (int w = 0; w < warp; ++w) {
      const float4 v = pairs[w][lane];
      h2 = make_float2(glr_map(v.x, v.y, h2.x), glr_map(v.z, v.w, h2.y));
    }
    uint64_t h = pk(h2.x, h2.y);
    if (TMA) {
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        h = SEQ && (reset >> j & 1) ? in[j] : ffma2(dec[j], h, in[j]);
        glr_sts<DT>(st, j, lane, h);
      }
      if (a.out != nullptr && n > 0) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&maps.out, st, at.c0, static_cast<int>(t0), b);
          bulk_commit();
        }
      }
    } else {
      const bool pair = g.pair && in1;
      typename Fmt<DT>::E* out = static_cast<typename Fmt<DT>::E*>(a.out) + (b * a.os[0] + t0 * a.os[1] + c * a.os[2]);
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        h = SEQ && (reset >> j & 1) ? in[j] : ffma2(dec[j], h, in[j]);
        if (j < n && a.out != nullptr) glr_stg<DT>(out, a.os[2], pair, in0, in1, h);
        out += a.os[1];
      }
    }
    if (a.s1 != nullptr && n > 0 && t0 + n == a.L) {
      float* p = a.s1 + b * a.s1s[0] + c * a.s1s[1];
      upk(h, h2.x, h2.y);
      if (in0) p[0] = h2.x;
      if (in1) p[a.s1s[1]] = h2.y;
    }
  }
  if (TMA && lane == 0) bulk_wait_read<>();
}

template <int DT, bool SEQ, bool TMA>
cudaError_t launch(const GlrArgs& a, const GlrTiles& t, const GlrChain& chain, const Device& dev, cudaStream_t s) {
  Maps maps = {};
  if constexpr (TMA) {
    const int64_t box[2] = {kGlrC, kGlrT};
    if (!tensor_map3(&maps.x, a.x, a.xs, a.B, a.L, a.C, box, static_cast<Dtype>(DT)) ||
        !tensor_map3(&maps.p, a.p, a.ps, a.B, a.L, a.C, box, static_cast<Dtype>(DT)) ||
        !tensor_map3(&maps.q, a.q, a.qs, a.B, a.L, a.C, box, static_cast<Dtype>(DT)))
      return cudaErrorInvalidValue;
    const int64_t run[2] = {kGlrC, kRun};
    if (a.out != nullptr && !tensor_map3(&maps.out, a.out, a.os, a.B, a.L, a.C, run, static_cast<Dtype>(DT)))
      return cudaErrorInvalidValue;
  }
  const int smem = TMA ? kStages * 3 * plane_bytes<DT>() : 0;
  cudaError_t e = cudaFuncSetAttribute(glr_fwd_kernel<DT, SEQ, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t most = static_cast<int64_t>(dev.sm_count) * (DT == kF32 ? 2 : 4);
  GlrTiles g = t;
  g.serial = g.levels > 1 && g.levels <= kGlrSerial;
  g.one = !g.serial && g.total <= most;
  const int64_t grid = g.serial ? g.ncols : g.total;
  return glr_launch(glr_fwd_kernel<DT, SEQ, TMA>, g, static_cast<unsigned>(grid < most ? grid : most), kThreads, smem, s, a, g,
                    chain, maps);
}

template <int DT>
cudaError_t fwd_dt(const GlrArgs& a, const GlrTiles& t, const GlrChain& c, bool tma, const Device& dev,
                   cudaStream_t s) {
  if (a.seq != nullptr) return tma ? launch<DT, true, true>(a, t, c, dev, s) : launch<DT, true, false>(a, t, c, dev, s);
  return tma ? launch<DT, false, true>(a, t, c, dev, s) : launch<DT, false, false>(a, t, c, dev, s);
}

}  // namespace

GlrTiles glr_tiles(int64_t B, int64_t L, int64_t C) {
  GlrTiles t = {};
  t.nct = static_cast<int>((C + kGlrC - 1) / kGlrC);
  t.ncols = static_cast<int>(B * t.nct);
  t.levels = static_cast<int>((L + kGlrT - 1) / kGlrT);
  t.total = static_cast<int>(static_cast<int64_t>(t.ncols) * t.levels);
  t.ncols_inv = (uint64_t(1) << 63) / static_cast<uint64_t>(t.ncols) + 1;
  t.nct_inv = (uint64_t(1) << 63) / static_cast<uint64_t>(t.nct) + 1;
  return t;
}

bool glr_pair_out(const void* p, const int64_t* s, Dtype dt) {
  const int64_t e = dt == kF32 ? 4 : 2;
  return s[2] == 1 && s[0] % 2 == 0 && s[1] % 2 == 0 && reinterpret_cast<uintptr_t>(p) % (2 * e) == 0;
}

uint64_t glr_fwd_workspace(int64_t B, int64_t L, int64_t C) {
  const GlrTiles t = glr_tiles(B, L, C);
  return t.levels > kGlrSerial ? glr_chain_bytes(t.total) : 0;
}

cudaError_t launch_glr_fwd(const GlrArgs& a, void* ws, Dtype dt, const Device& dev, cudaStream_t stream) {
  GlrTiles t = glr_tiles(a.B, a.L, a.C);
  const bool tma = tensor_map_eligible(a.x, a.xs, a.B, a.L, a.C, dt) && tensor_map_eligible(a.p, a.ps, a.B, a.L, a.C, dt) &&
                   tensor_map_eligible(a.q, a.qs, a.B, a.L, a.C, dt) &&
                   (a.out == nullptr || tensor_map_eligible(a.out, a.os, a.B, a.L, a.C, dt));
  t.pair = a.out != nullptr && glr_pair_out(a.out, a.os, dt);
  GlrChain chain = {};
  if (t.levels > kGlrSerial) chain = glr_chain(ws);
  switch (dt) {
    case kF32: return fwd_dt<kF32>(a, t, chain, tma, dev, stream);
    case kF16: return fwd_dt<kF16>(a, t, chain, tma, dev, stream);
    case kBF16: return fwd_dt<kBF16>(a, t, chain, tma, dev, stream);
  }
  return cudaErrorInvalidValue;
}

unsigned read_and_clear_fault_glr() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_fault, sizeof(v)) != cudaSuccess) return ~0u;
  if (v != 0 && cudaMemcpyToSymbol(g_fault, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace ccv

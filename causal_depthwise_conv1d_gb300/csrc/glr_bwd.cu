// Gated linear recurrence, backward pass: one pass over x, the gates and dout
// from the last tokens to the first.
//
//   G_t = dout_t + a_{t+1} G_{t+1};   u = m i, k = a^2 / m^2:  b = u x,  W = a h_{t-1} - k b
//   dx = G u;  dq = G b (1 - i);  dp = G W l (1 - r);  drate = -sum G W r
//
// Tiles as in the forward pass (glr_tile.cuh), eight warps of eight tokens.  The
// states before every 64th token are given, so a tile's states need no other
// tile; what is carried from tile to tile, backwards in time, is a G: a run of
// tokens maps the carry into A c + R, published and folded as the states are.
// A warp keeps five values of each token and channel in registers: a, k, u, the
// smaller one of r and 1 - r (with a sign that tells which), 1 - i; when the state
// before the token is known, G's factors u, b (1 - i), W l (1 - r), W r take
// their places.  So every sigmoid and root is taken once.
//
// bf16, 4 x 2048 x 4096 113 us (4.2 TB/s of 478 MB): 76 instructions an element at
// 63 % of the issue slots (warps with a rate above 0.85: 80 instructions, 119 us).
// Eight tokens a warp are what 128 registers hold.
#include <type_traits>

#include "glr_tile.cuh"

namespace ccv {
namespace {

__device__ unsigned g_fault;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = kGlrT / kWarps;  // tokens of a warp
constexpr int kStages = 2;
constexpr int kPublisher = 1;  // the warp that publishes (the first one starts the copies)

struct Maps {
  CUtensorMap x, p, q, o, dx, dp, dq;
};

template <int DT>
constexpr int plane_bytes() {
  return kGlrT * kGlrC * (DT == kF32 ? 4 : 2);
}

struct __align__(16) Shared {
  float4 fwd[kWarps][32];  // (A, H) of the states
  float4 bwd[kWarps][32];  // (A, R) of the carries
  float2 rate[kWarps][32];
  uint64_t full[kStages];
  GlrPlace place[kStages];
  float2 carried[kStages][32];  // serial: the carry out of the tile before
};

// The runs' maps of the carry, last run first, as one.
__device__ __forceinline__ float4 joined(const float4 (*runs)[32], int lane) {
  float4 m = runs[kWarps - 1][lane];
#pragma unroll
  for (int w = kWarps - 2; w >= 0; --w) {
    const float4 v = runs[w][lane];
    glr_join(v.x, v.y, m.x, m.y);
    glr_join(v.z, v.w, m.z, m.w);
  }
  m.x = glr_positive(m.x), m.z = glr_positive(m.z);
  return m;
}

// 1 - s of a sigmoid s = 1 / (1 + e), relatively precise.
__device__ __forceinline__ float one_minus(float s, float e) { return e < 0x1p100f ? __fmul_rn(e, s) : 1.f; }

template <int DT, bool SEQ, bool TMA>
__global__ void __launch_bounds__(kThreads, DT == kF32 ? 1 : 2)
    glr_bwd_kernel(const GlrArgs a, const GlrGrads gr, const GlrTiles g, const GlrChain chain,
                   const __grid_constant__ Maps maps) {
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

  int drawn = 0;
  auto draw = [&]() -> int {
    if (chained) return static_cast<int>(atomicAdd(chain.ticket, 1u) + 1u);
    return glr_serial_tile(g, drawn++);
  };
  // Tile t in the order of work: the last tokens first.
  auto fill = [&](int s, int t) {
    GlrPlace p;
    const int back = glr_div(t, g.ncols_inv);
    p.tile = t;
    p.level = g.levels - 1 - back, p.col = t - back * g.ncols;
    p.b = glr_div(p.col, g.nct_inv), p.c0 = (p.col - p.b * g.nct) * kGlrC;
    sh.place[s] = p;
    if (!TMA || t >= g.total) {
      mbar_arrive(&sh.full[s]);
      return;
    }
    const int t0 = p.level * kGlrT;
    uint8_t* st = stages + s * 4 * PLANE;
    mbar_arrive_expect_tx(&sh.full[s], 4 * PLANE);
    tma_load_3d(st, &maps.x, p.c0, t0, p.b, &sh.full[s]);
    tma_load_3d(st + PLANE, &maps.p, p.c0, t0, p.b, &sh.full[s]);
    tma_load_3d(st + 2 * PLANE, &maps.q, p.c0, t0, p.b, &sh.full[s]);
    tma_load_3d(st + 3 * PLANE, &maps.o, p.c0, t0, p.b, &sh.full[s]);
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
    const int level = at.level, back = g.levels - 1 - level, b = at.b, c = at.c0 + 2 * lane;
    const int64_t t0 = static_cast<int64_t>(level) * kGlrT + warp * kRun;
    const bool in0 = c < a.C, in1 = c + 1 < a.C;
    const int64_t left = a.L - t0;
    const int n = left >= kRun ? kRun : left > 0 ? static_cast<int>(left) : 0;  // tokens of this warp
    uint4 before = make_uint4(kSlotEmpty, 0u, 0u, 0u);
    if (chained && back > 0) before = ld_slot(glr_slot(chain, at.tile - g.ncols, lane));  // it may be there already
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
    const float* csp = a.cs + b * a.css[0] + level * a.css[1] + c * a.css[2];
    float2 h2 = make_float2(in0 ? csp[0] : 0.f, in1 ? csp[a.css[2]] : 0.f);
    uint8_t* st = stages + s * 4 * PLANE + warp * (PLANE / kWarps);  // this warp's rows
    auto load = [&](int plane, const void* p, const int64_t* str, int j) -> uint64_t {
      if constexpr (TMA) return glr_lds<DT>(st + plane * PLANE, j, lane);
      else return glr_ldg<DT>(p, b * str[0] + (t0 + j) * str[1] + c * str[2], str[2], j < n && in0, j < n && in1);
    };

    // dec: a;  f0: k, then W l (1 - r);  f1: u;  f2: the smaller one of r, 1 - r, then W r;  f3: 1 - i, then b (1 - i)
    uint64_t dec[kRun], f0[kRun], f1[kRun], f2[kRun], f3[kRun];
    auto gates = [&](auto near) {
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        const uint64_t p = load(1, a.p, a.ps, j), q = load(2, a.q, a.qs, j);
        uint64_t r, ep, i, eq, m2;
        glr_sigmoid2(p, r, ep);
        glr_sigmoid2(q, i, eq);
        glr_decay2<decltype(near)::value>(fmul2(rate, r), dec[j], m2);
        float v0, v1, e0, e1, m0, m1, s0, s1;
        upk(m2, m0, m1);
        // 1 / m, zero where m is: u and k are zero there too
        s0 = m0 >= 0x1p-126f ? rsqrt_approx(m0) : 0.f;
        s1 = m1 >= 0x1p-126f ? rsqrt_approx(m1) : 0.f;
        const uint64_t rs = pk(s0, s1);
        f1[j] = fmul2(fmul2(m2, rs), i);
        const uint64_t as = fmul2(dec[j], rs);
        f0[j] = fmul2(as, as);
        upk(r, v0, v1), upk(ep, e0, e1);
        f2[j] = pk(v0 < 0.5f ? v0 : -one_minus(v0, e0), v1 < 0.5f ? v1 : -one_minus(v1, e1));
        upk(i, v0, v1), upk(eq, e0, e1);
        f3[j] = pk(one_minus(v0, e0), one_minus(v1, e1));
      }
    };
    if (__all_sync(kFullMask, rate0 <= -kGlrSeries && rate1 <= -kGlrSeries))
      gates(std::true_type{});
    else
      gates(std::false_type{});
    if (n < kRun)  // nothing happens at tokens past the end
#pragma unroll
      for (int j = 0; j < kRun; ++j)
        if (j >= n) dec[j] = pk(1.f, 1.f), f1[j] = 0;
    {
      uint64_t A = pk(1.f, 1.f), H = 0;
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        const uint64_t in = fmul2(f1[j], load(0, a.x, a.xs, j));
        const bool cut = SEQ && (reset >> j & 1);
        A = fmul2(A, dec[j]);
        H = cut ? in : ffma2(dec[j], H, in);
      }
      sh.fwd[warp][lane] = glr_run(A, H, SEQ && reset != 0);
      // the carry's map, last token first
      uint64_t R = 0;
#pragma unroll
      for (int j = kRun - 1; j >= 0; --j) {
        const uint64_t o = load(3, gr.dout, gr.dos, j);
        R = SEQ && (reset >> j & 1) ? 0 : fmul2(dec[j], fadd2(o, R));
      }
      sh.bwd[warp][lane] = glr_run(A, R, SEQ && reset != 0);
    }
    if (TMA && lane == 0) bulk_wait_read<>();  // the boxes of the tile before have left its stage
    __syncthreads();  // the runs' maps are there, the other stage is free
    if (tid == 0 && !g.one) {
      fence_proxy_async_smem();
      fill(s ^ 1, next);
      if (next < g.total) next = draw();
    }

    float2 d2 = make_float2(0.f, 0.f);  // the carry into the tile's last token
    if (back == 0) {
      if (gr.ds1 != nullptr) {
        const float* p = gr.ds1 + b * gr.ds1s[0] + c * gr.ds1s[1];
        d2 = make_float2(in0 ? p[0] : 0.f, in1 ? p[gr.ds1s[1]] : 0.f);
      }
    } else if (g.serial) {
      d2 = sh.carried[s ^ 1][lane];
    } else if (__all_sync(kFullMask, before.x == kSlotState)) {
      d2 = glr_slot_state(before);
    } else {
      if (warp == kPublisher && level > 0) glr_put_pair(chain, at.tile, lane, joined(sh.bwd, lane));
      if (!glr_look_back(chain, g, back, at.col, lane, d2)) {
        if (lane == 0) atomicOr(&g_fault, kFaultConsumerWait);
        d2 = make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));  // nothing that passes for one
      }
    }
    if (warp == kPublisher && (level > 0 || gr.ds0 != nullptr)) {
      const float4 m = joined(sh.bwd, lane);
      const float2 after = make_float2(glr_map(m.x, m.y, d2.x), glr_map(m.z, m.w, d2.y));
      if (level > 0) {
        if (g.serial)
          sh.carried[s][lane] = after;
        else
          glr_put_state(chain, at.tile, lane, after);
      } else {
        float* p = gr.ds0 + b * gr.ds0s[0] + c * gr.ds0s[1];
        if (in0) p[0] = after.x;
        if (in1) p[gr.ds0s[1]] = after.y;
      }
    }

    // the states, and with them G's factors
    for (int w = 0; w < warp; ++w) {
      const float4 v = sh.fwd[w][lane];
      h2 = make_float2(glr_map(v.x, v.y, h2.x), glr_map(v.z, v.w, h2.y));
    }
    uint64_t h = pk(h2.x, h2.y);
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      if (SEQ && (reset >> j & 1)) h = 0;
      const uint64_t in = fmul2(f1[j], load(0, a.x, a.xs, j));
      const uint64_t ah = fmul2(dec[j], h);
      const uint64_t W = ffma2(fmul2(f0[j], pk(-1.f, -1.f)), in, ah);
      h = fadd2(ah, in);
      float v0, v1;
      upk(f2[j], v0, v1);
      const float w0 = __fadd_rn(1.f, -fabsf(v0)), w1 = __fadd_rn(1.f, -fabsf(v1));
      const bool b0 = __float_as_int(v0) >= 0, b1 = __float_as_int(v1) >= 0;  // the sign, of zeros too
      const uint64_t r = pk(b0 ? v0 : w0, b1 ? v1 : w1), om = pk(b0 ? w0 : -v0, b1 ? w1 : -v1);
      f2[j] = fmul2(W, r);
      f0[j] = fmul2(f2[j], fmul2(rate, om));
      f3[j] = fmul2(in, f3[j]);
    }
    for (int w = kWarps - 1; w > warp; --w) {
      const float4 v = sh.bwd[w][lane];
      d2 = make_float2(glr_map(v.x, v.y, d2.x), glr_map(v.z, v.w, d2.y));
    }
    uint64_t d = pk(d2.x, d2.y), sum = 0;
    if (TMA) {
#pragma unroll
      for (int j = kRun - 1; j >= 0; --j) {
        const uint64_t G = fadd2(d, load(3, gr.dout, gr.dos, j));
        glr_sts<DT>(st, j, lane, fmul2(G, f1[j]));
        glr_sts<DT>(st + PLANE, j, lane, fmul2(G, f0[j]));
        glr_sts<DT>(st + 2 * PLANE, j, lane, fmul2(G, f3[j]));
        if (j < n) sum = ffma2(G, f2[j], sum);
        d = SEQ && (reset >> j & 1) ? 0 : fmul2(dec[j], G);
      }
      if (n > 0) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&maps.dx, st, at.c0, static_cast<int>(t0), b);
          tma_store_3d(&maps.dp, st + PLANE, at.c0, static_cast<int>(t0), b);
          tma_store_3d(&maps.dq, st + 2 * PLANE, at.c0, static_cast<int>(t0), b);
          bulk_commit();
        }
      }
    } else {
      const bool pair = g.pair && in1;
      using E = typename Fmt<DT>::E;
      const int64_t tl = t0 + kRun - 1;  // from the last token back
      E* dx = static_cast<E*>(gr.dx) + (b * gr.dxs[0] + tl * gr.dxs[1] + c * gr.dxs[2]);
      E* dp = static_cast<E*>(gr.dp) + (b * gr.dps[0] + tl * gr.dps[1] + c * gr.dps[2]);
      E* dq = static_cast<E*>(gr.dq) + (b * gr.dqs[0] + tl * gr.dqs[1] + c * gr.dqs[2]);
#pragma unroll
      for (int j = kRun - 1; j >= 0; --j) {
        if (j < n) {
          const uint64_t G = fadd2(d, load(3, gr.dout, gr.dos, j));
          glr_stg<DT>(dx, gr.dxs[2], pair, in0, in1, fmul2(G, f1[j]));
          glr_stg<DT>(dp, gr.dps[2], pair, in0, in1, fmul2(G, f0[j]));
          glr_stg<DT>(dq, gr.dqs[2], pair, in0, in1, fmul2(G, f3[j]));
          sum = ffma2(G, f2[j], sum);
          d = SEQ && (reset >> j & 1) ? 0 : fmul2(dec[j], G);
        }
        dx -= gr.dxs[1], dp -= gr.dps[1], dq -= gr.dqs[1];
      }
    }
    upk(sum, d2.x, d2.y);
    sh.rate[warp][lane] = d2;
    __syncthreads();  // the sums are there
    if (warp == kWarps - 1) {
#pragma unroll
      for (int w = kWarps - 2; w >= 0; --w) {
        const float2 v = sh.rate[w][lane];
        d2.x += v.x, d2.y += v.y;
      }
      float* part = gr.part + (static_cast<int64_t>(b) * g.levels + level) * a.C + c;
      if (in0) part[0] = -d2.x;
      if (in1) part[1] = -d2.y;
    }
  }
  if (TMA && lane == 0) bulk_wait_read<>();
}

// drate: the partial sums [P][C] in 32 interleaved subsequences and then these.
__global__ void __launch_bounds__(1024) glr_rate_kernel(const float* part, int64_t P, int64_t C, float* drate,
                                                        int64_t drs) {
  pdl_enter();
  __shared__ float sh[32][33];
  const int i = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + i;
  float x = 0.f;
  if (c < C)
#pragma unroll 4
    for (int64_t k = r; k < P; k += 32) x += part[k * C + c];
  sh[r][i] = x;
  __syncthreads();
  if (r == 0 && c < C) {
    x = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) x += sh[k][i];
    drate[c * drs] = x;
  }
}

template <int DT, bool SEQ, bool TMA>
cudaError_t launch(const GlrArgs& a, const GlrGrads& gr, const GlrTiles& t, const GlrChain& chain, const Device& dev,
                   cudaStream_t s) {
  Maps maps = {};
  constexpr Dtype dt = static_cast<Dtype>(DT);
  if constexpr (TMA) {
    const int64_t box[2] = {kGlrC, kGlrT};
    if (!tensor_map3(&maps.x, a.x, a.xs, a.B, a.L, a.C, box, dt) || !tensor_map3(&maps.p, a.p, a.ps, a.B, a.L, a.C, box, dt) ||
        !tensor_map3(&maps.q, a.q, a.qs, a.B, a.L, a.C, box, dt) ||
        !tensor_map3(&maps.o, gr.dout, gr.dos, a.B, a.L, a.C, box, dt))
      return cudaErrorInvalidValue;
    const int64_t run[2] = {kGlrC, kRun};
    if (!tensor_map3(&maps.dx, gr.dx, gr.dxs, a.B, a.L, a.C, run, dt) ||
        !tensor_map3(&maps.dp, gr.dp, gr.dps, a.B, a.L, a.C, run, dt) ||
        !tensor_map3(&maps.dq, gr.dq, gr.dqs, a.B, a.L, a.C, run, dt))
      return cudaErrorInvalidValue;
  }
  const int smem = TMA ? kStages * 4 * plane_bytes<DT>() : 0;
  const cudaError_t e =
      cudaFuncSetAttribute(glr_bwd_kernel<DT, SEQ, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t most = static_cast<int64_t>(dev.sm_count) * (DT == kF32 ? 1 : 2);
  GlrTiles g = t;
  g.serial = g.levels > 1 && g.levels <= kGlrSerial;
  g.one = !g.serial && g.total <= most;
  const int64_t grid = g.serial ? g.ncols : g.total;
  return glr_launch(glr_bwd_kernel<DT, SEQ, TMA>, g, static_cast<unsigned>(grid < most ? grid : most), kThreads,
                    smem, s, a, gr, g, chain, maps);
}

template <int DT>
cudaError_t bwd_dt(const GlrArgs& a, const GlrGrads& g, const GlrTiles& t, const GlrChain& c, bool tma,
                   const Device& dev, cudaStream_t s) {
  if (a.seq != nullptr)
    return tma ? launch<DT, true, true>(a, g, t, c, dev, s) : launch<DT, true, false>(a, g, t, c, dev, s);
  return tma ? launch<DT, false, true>(a, g, t, c, dev, s) : launch<DT, false, false>(a, g, t, c, dev, s);
}

}  // namespace

cudaError_t launch_glr_bwd(const GlrArgs& a, const GlrGrads& gr, void* ws, Dtype dt, const Device& dev,
                           cudaStream_t stream) {
  GlrTiles t = glr_tiles(a.B, a.L, a.C);
  const bool tma = tensor_map_eligible(a.x, a.xs, a.B, a.L, a.C, dt) && tensor_map_eligible(a.p, a.ps, a.B, a.L, a.C, dt) &&
          tensor_map_eligible(a.q, a.qs, a.B, a.L, a.C, dt) && tensor_map_eligible(gr.dout, gr.dos, a.B, a.L, a.C, dt) &&
          tensor_map_eligible(gr.dx, gr.dxs, a.B, a.L, a.C, dt) && tensor_map_eligible(gr.dp, gr.dps, a.B, a.L, a.C, dt) &&
          tensor_map_eligible(gr.dq, gr.dqs, a.B, a.L, a.C, dt);
  t.pair = glr_pair_out(gr.dx, gr.dxs, dt) && glr_pair_out(gr.dp, gr.dps, dt) && glr_pair_out(gr.dq, gr.dqs, dt);
  GlrChain chain = {};
  cudaError_t e = cudaSuccess;
  if (t.levels > kGlrSerial) chain = glr_chain(ws);
  switch (dt) {
    case kF32: e = bwd_dt<kF32>(a, gr, t, chain, tma, dev, stream); break;
    case kF16: e = bwd_dt<kF16>(a, gr, t, chain, tma, dev, stream); break;
    case kBF16: e = bwd_dt<kBF16>(a, gr, t, chain, tma, dev, stream); break;
  }
  return e;
}

cudaError_t launch_glr_rate(const float* part, int64_t P, int64_t C, float* drate, int64_t drs, cudaStream_t stream) {
  return launch_pdl(glr_rate_kernel, static_cast<unsigned>((C + 31) / 32), 1024, 0, stream, part, P, C, drate, drs);
}

unsigned read_and_clear_fault_glr_bwd() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_fault, sizeof(v)) != cudaSuccess) return ~0u;
  if (v != 0 && cudaMemcpyToSymbol(g_fault, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace ccv

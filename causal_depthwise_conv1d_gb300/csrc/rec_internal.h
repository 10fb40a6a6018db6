// Internal interface between the ABI front end of the gated linear recurrence
// and of group normalisation (rec_api.cpp) and their launchers (glr_*.cu,
// gn*.cu).
#pragma once

#include "ccv_internal.h"

namespace ccv {

constexpr int kGlrChunk = 64;  // tokens between two kept states

// Validated arguments of the gated linear recurrence.  x, the gates' logits
// (p: decay, q: input) and out: [B,L,C]; rate FP32 [C]; states FP32 [.,C].
// Strides in elements, in the order of the dimensions.
struct GlrArgs {
  const void* x;
  int64_t xs[3];
  const void* p;
  int64_t ps[3];
  const void* q;
  int64_t qs[3];
  const float* rate;
  int64_t rs;
  const int32_t* seq;  // [B,L] or null
  int64_t ss[2];
  const float* s0;  // state before the first token, or null (zero)
  int64_t s0s[2];
  float* s1;  // state after the last token, or null
  int64_t s1s[2];
  float* cs;  // [B,ceil(L/64),C]: state before every 64th token, or null
  int64_t css[3];
  const int32_t* slots;  // row b's state is s0[slots[b]] (null: s0[b])
  int64_t slot_stride, n_slots;
  void* out;  // or null
  int64_t os[3];
  int64_t B, L, C;
};

// Backward pass: the forward arguments (out, s1 unused, cs an input) and these.
struct GlrGrads {
  const void* dout;
  int64_t dos[3];
  const float* ds1;  // gradient of the final state, or null
  int64_t ds1s[2];
  void* dx;
  int64_t dxs[3];
  void* dp;
  int64_t dps[3];
  void* dq;
  int64_t dqs[3];
  float* drate;
  int64_t drs;
  float* ds0;  // or null
  int64_t ds0s[2];
  float* part;  // [partial sums][C] of drate
};

cudaError_t launch_glr_step(const GlrArgs& a, Dtype dt, cudaStream_t stream);
// Whole sequences; ws: glr_fwd_workspace() bytes (a function of the sizes
// alone), all bits set by the caller on the same stream.
uint64_t glr_fwd_workspace(int64_t B, int64_t L, int64_t C);
cudaError_t launch_glr_fwd(const GlrArgs& a, void* ws, Dtype dt, const Device& dev, cudaStream_t stream);
// Backward pass with a workspace as the forward's, of its own; then drate from the partial sums, one
// for each batch row and chunk.
cudaError_t launch_glr_bwd(const GlrArgs& a, const GlrGrads& g, void* ws, Dtype dt, const Device& dev,
                           cudaStream_t stream);
cudaError_t launch_glr_rate(const float* part, int64_t P, int64_t C, float* drate, int64_t drs, cudaStream_t stream);
unsigned read_and_clear_fault_glr();
unsigned read_and_clear_fault_glr_bwd();

// Validated arguments of group normalisation.  x, out: [N,S,C]; weight and
// bias [C] in their own dtype, or null (one, zero).
struct GnArgs {
  const void* x;
  int64_t xs[3];
  const void* w;
  int64_t ws;
  const void* b;
  int64_t bs;
  void* out;  // forward
  int64_t os[3];
  const void* dout;  // backward from here
  int64_t gs[3];
  void* dx;
  int64_t dxs[3];
  void* dw;  // or null
  int64_t dws;
  void* db;  // or null
  int64_t dbs;
  float2* stats;  // [N,G,slabs] mean and sum of squared deviations of each slab
  float2* sums;   // [N,G,slabs] backward: sums of d and d xh
  float* part;    // [partial sums][2][C] of dw and db, or null
  int64_t N, S, C, G;
  float eps;
  int wdt;
  bool silu;
};

// How the any-stride kernels cut the problem (a function of the sizes alone):
// a group's positions in `slabs` slabs of `rows`; the backward pass adds the
// parameters' gradients of `slots` interleaved sets of samples, slots * slabs
// partial sums.
struct GnPlan {
  int64_t slabs, rows, slots;
};
GnPlan gn_plan(int64_t N, int64_t S, int64_t C, int64_t G);
cudaError_t launch_gn_fwd(const GnArgs& a, Dtype dt, cudaStream_t stream);
cudaError_t launch_gn_bwd(const GnArgs& a, Dtype dt, cudaStream_t stream);

// Rows on their own (S = 1; gn_rows.cu) and groups that fit into a cluster's
// shared memory (gn_cluster.cu): aligned layouts.  The partial sums of dw and db
// that the backward pass makes there are functions of the sizes alone.
bool gn_rows_eligible(const GnArgs& a, Dtype dt, bool bwd);
int64_t gn_rows_slots(int64_t N, int64_t C, int64_t G, int64_t esize, bool bwd);
cudaError_t launch_gn_rows(const GnArgs& a, Dtype dt, bool bwd, cudaStream_t stream);
bool gn_cluster_eligible(const GnArgs& a, Dtype dt, bool bwd);
int64_t gn_cluster_parts(int64_t N, int64_t S, int64_t C, int64_t G, int64_t esize);
cudaError_t launch_gn_cluster(const GnArgs& a, Dtype dt, bool bwd, cudaStream_t stream);
// Rows on their own in narrow groups of any width and strides (gn_narrow.cu).
bool gn_narrow_eligible(int64_t S, int64_t C, int64_t G);
int64_t gn_narrow_slots(int64_t N, int64_t C, int64_t G);
cudaError_t launch_gn_narrow(const GnArgs& a, Dtype dt, bool bwd, cudaStream_t stream);
// The most partial sums any of the kernels makes for these sizes.
int64_t gn_parts(int64_t N, int64_t S, int64_t C, int64_t G);
unsigned read_and_clear_fault_gn();

// Sums of P partial sums [P][2][C] in a fixed order into dw and db (ln.cu).
cudaError_t launch_param_sums(const float* part, int64_t P, int64_t C, void* dw, int64_t dws, void* db, int64_t dbs,
                              int wdt, cudaStream_t stream);

}  // namespace ccv

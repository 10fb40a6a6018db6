// C-ABI front end of the gated linear recurrence (ccv_glr_*) and of group
// normalisation (ccv_gn_*): argument validation, kernel selection and launch
// on the caller's stream.  See include/ccv.h for the contract.
#include "api_check.h"
#include "rec_internal.h"

namespace {

int64_t glr_chunks(int64_t L) { return (L + ccv::kGlrChunk - 1) / ccv::kGlrChunk; }
uint64_t up256(uint64_t x) { return (x + 255) / 256 * 256; }

ccv_status check_glr_sizes(int64_t B, int64_t L, int64_t C, ccv_dtype dtype) {
  if (B < 0 || L < 0 || C < 0) CCV_FAIL(CCV_ERR_INVALID_ARG, "B, L and C must be >= 0");
  if (!valid_dtype(dtype)) CCV_FAIL(CCV_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
  // element counts and the index arithmetic on them stay within int64, numbers of blocks within int32
  const __int128 lim = static_cast<__int128>(INT64_MAX) >> 8;
  const __int128 bc = static_cast<__int128>(B) * C;
  if (bc > lim || bc * (L > 0 ? L : 1) > lim || B > 0x7fffffff || L > 0x7fffffc0 || C > 0x7fffffc0 ||
      static_cast<__int128>(B) * ((C + 63) / 64) * glr_chunks(L > 0 ? L : 1) > 0x7fffffff)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "B*L*C is too large");
  return CCV_OK;
}

// The backward pass: the states before every 64th token, partial sums of drate,
// the chains of the states' recomputation and of the gradients.
struct GlrBwdWorkspace {
  uint64_t states, part, chain, total;
};

GlrBwdWorkspace glr_bwd_workspace(int64_t B, int64_t L, int64_t C) {
  GlrBwdWorkspace w = {0, 0, 0, 0};
  if (B == 0 || L == 0 || C == 0) return w;
  w.states = up256(static_cast<uint64_t>(B) * static_cast<uint64_t>(glr_chunks(L)) * static_cast<uint64_t>(C) * 4);
  w.part = w.states;
  w.chain = up256(ccv::glr_fwd_workspace(B, L, C));
  w.total = w.states + w.part + 2 * w.chain;
  return w;
}

}  // namespace

extern "C" {

ccv_status ccv_glr_fwd_workspace_size(int64_t B, int64_t L, int64_t C, ccv_dtype dtype, uint64_t* bytes) {
  ccv::api_begin();
  if (bytes == nullptr) CCV_FAIL(CCV_ERR_INVALID_ARG, "bytes is required");
  CCV_TRY(check_glr_sizes(B, L, C, dtype));
  *bytes = B > 0 && L > 0 && C > 0 ? ccv::glr_fwd_workspace(B, L, C) : 0;
  return CCV_OK;
}

ccv_status ccv_glr_fwd(const void* x, const int64_t x_strides[3], const void* decay_gate,
                       const int64_t decay_gate_strides[3], const void* input_gate,
                       const int64_t input_gate_strides[3], const float* rate, int64_t rate_stride,
                       const int32_t* seq_idx, const int64_t seq_idx_strides[2], const float* initial_state,
                       const int64_t initial_state_strides[2], void* out, const int64_t out_strides[3],
                       float* final_state_out, const int64_t final_state_strides[2], float* chunk_states_out,
                       const int64_t chunk_states_strides[3], void* workspace, uint64_t workspace_bytes, int64_t B,
                       int64_t L, int64_t C, ccv_dtype dtype, void* stream) {
  ccv::api_begin();
  CCV_TRY(check_glr_sizes(B, L, C, dtype));
  if (B == 0 || C == 0) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  const int64_t e = dtype_size(dtype);
  const int64_t blc[3] = {B, L, C}, bl[2] = {B, L}, bc[2] = {B, C}, cc[1] = {C}, cs[3] = {B, glr_chunks(L), C};
  Tensors t;
  CCV_TRY(t.add("x", x, x_strides, 3, blc, e, false, true));
  CCV_TRY(t.add("decay_gate", decay_gate, decay_gate_strides, 3, blc, e, false, true));
  CCV_TRY(t.add("input_gate", input_gate, input_gate_strides, 3, blc, e, false, true));
  CCV_TRY(t.add("rate", rate, &rate_stride, 1, cc, 4, false, true));
  CCV_TRY(t.add("seq_idx", seq_idx, seq_idx_strides, 2, bl, 4, false, false));
  CCV_TRY(t.add("initial_state", initial_state, initial_state_strides, 2, bc, 4, false, false));
  CCV_TRY(t.add("out", out, out_strides, 3, blc, e, true, true));
  CCV_TRY(t.add("final_state_out", final_state_out, final_state_strides, 2, bc, 4, true, false));
  CCV_TRY(t.add("chunk_states_out", chunk_states_out, chunk_states_strides, 3, cs, 4, true, false));
  CCV_TRY(add_workspace(t, workspace, workspace_bytes, L > 0 ? ccv::glr_fwd_workspace(B, L, C) : 0, 128));
  CCV_TRY(t.disjoint());
  if (L == 0 && final_state_out == nullptr) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  ccv::GlrArgs a = {};
  a.x = x, a.p = decay_gate, a.q = input_gate, a.rate = rate, a.rs = rate_stride, a.seq = seq_idx;
  a.s0 = initial_state, a.s1 = final_state_out, a.cs = chunk_states_out, a.out = out, a.n_slots = B;
  copy(a.xs, x_strides, 3), copy(a.ps, decay_gate_strides, 3), copy(a.qs, input_gate_strides, 3);
  copy(a.ss, seq_idx_strides, 2), copy(a.s0s, initial_state_strides, 2), copy(a.s1s, final_state_strides, 2);
  copy(a.css, chunk_states_strides, 3), copy(a.os, out_strides, 3);
  a.B = B, a.L = L, a.C = C;
  const ccv::Dtype dt = static_cast<ccv::Dtype>(dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (L == 0) return launched(ccv::launch_glr_step(a, dt, s), "glr_fwd");  // copies the state
  ccv::Device dev;
  CCV_TRY(static_cast<ccv_status>(ccv::api_device(&dev)));
  const uint64_t chain = ccv::glr_fwd_workspace(B, L, C);
  cudaError_t err = chain > 0 ? cudaMemsetAsync(workspace, 0xff, chain, s) : cudaSuccess;
  if (err == cudaSuccess) err = ccv::launch_glr_fwd(a, workspace, dt, dev, s);
  return launched(err, "glr_fwd");
}

ccv_status ccv_glr_step(const void* x, const int64_t x_strides[3], const void* decay_gate,
                        const int64_t decay_gate_strides[3], const void* input_gate,
                        const int64_t input_gate_strides[3], const float* rate, int64_t rate_stride, float* state,
                        const int64_t state_strides[2], int64_t n_slots, const int32_t* state_indices,
                        int64_t state_indices_stride, void* out, const int64_t out_strides[3], int64_t B, int64_t S,
                        int64_t C, ccv_dtype dtype, void* stream) {
  ccv::api_begin();
  CCV_TRY(check_glr_sizes(B, S, C, dtype));
  if (n_slots < 0) CCV_FAIL(CCV_ERR_INVALID_ARG, "n_slots must be >= 0");
  if (state_indices == nullptr && n_slots < B)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "n_slots must be at least B without state_indices");
  if (B == 0 || C == 0 || S == 0) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  const int64_t e = dtype_size(dtype);
  const int64_t bsc[3] = {B, S, C}, st[2] = {n_slots, C}, cc[1] = {C}, idx[1] = {B};
  Tensors t;
  CCV_TRY(t.add("x", x, x_strides, 3, bsc, e, false, true));
  CCV_TRY(t.add("decay_gate", decay_gate, decay_gate_strides, 3, bsc, e, false, true));
  CCV_TRY(t.add("input_gate", input_gate, input_gate_strides, 3, bsc, e, false, true));
  CCV_TRY(t.add("rate", rate, &rate_stride, 1, cc, 4, false, true));
  CCV_TRY(t.add("state_indices", state_indices, &state_indices_stride, 1, idx, 4, false, false));
  CCV_TRY(t.add("state", state, state_strides, 2, st, 4, true, true));
  CCV_TRY(t.add("out", out, out_strides, 3, bsc, e, true, true));
  CCV_TRY(t.disjoint());
  ccv::GlrArgs a = {};
  a.x = x, a.p = decay_gate, a.q = input_gate, a.rate = rate, a.rs = rate_stride, a.s0 = state, a.s1 = state;
  a.out = out, a.slots = state_indices, a.slot_stride = state_indices_stride, a.n_slots = n_slots;
  copy(a.xs, x_strides, 3), copy(a.ps, decay_gate_strides, 3), copy(a.qs, input_gate_strides, 3);
  copy(a.s0s, state_strides, 2), copy(a.s1s, state_strides, 2), copy(a.os, out_strides, 3);
  a.B = B, a.L = S, a.C = C;
  return launched(ccv::launch_glr_step(a, static_cast<ccv::Dtype>(dtype), static_cast<cudaStream_t>(stream)),
                  "glr_step");
}

ccv_status ccv_glr_bwd_workspace_size(int64_t B, int64_t L, int64_t C, ccv_dtype dtype, uint64_t* bytes) {
  ccv::api_begin();
  if (bytes == nullptr) CCV_FAIL(CCV_ERR_INVALID_ARG, "bytes is required");
  CCV_TRY(check_glr_sizes(B, L, C, dtype));
  *bytes = glr_bwd_workspace(B, L, C).total;
  return CCV_OK;
}

ccv_status ccv_glr_bwd(const void* x, const int64_t x_strides[3], const void* decay_gate,
                       const int64_t decay_gate_strides[3], const void* input_gate,
                       const int64_t input_gate_strides[3], const float* rate, int64_t rate_stride,
                       const int32_t* seq_idx, const int64_t seq_idx_strides[2], const float* initial_state,
                       const int64_t initial_state_strides[2], const void* dout, const int64_t dout_strides[3],
                       const float* dfinal_state, const int64_t dfinal_state_strides[2], const float* chunk_states,
                       const int64_t chunk_states_strides[3], void* dx, const int64_t dx_strides[3],
                       void* ddecay_gate, const int64_t ddecay_gate_strides[3], void* dinput_gate,
                       const int64_t dinput_gate_strides[3], float* drate, int64_t drate_stride,
                       float* dinitial_state, const int64_t dinitial_state_strides[2], void* workspace,
                       uint64_t workspace_bytes, int64_t B, int64_t L, int64_t C, ccv_dtype dtype, void* stream) {
  ccv::api_begin();
  CCV_TRY(check_glr_sizes(B, L, C, dtype));
  if (dinitial_state != nullptr && initial_state == nullptr)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "dinitial_state requires initial_state");
  if (C == 0) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  const int64_t e = dtype_size(dtype);
  const int64_t blc[3] = {B, L, C}, bl[2] = {B, L}, bc[2] = {B, C}, cc[1] = {C}, cs[3] = {B, glr_chunks(L), C};
  Tensors t;
  CCV_TRY(t.add("x", x, x_strides, 3, blc, e, false, true));
  CCV_TRY(t.add("decay_gate", decay_gate, decay_gate_strides, 3, blc, e, false, true));
  CCV_TRY(t.add("input_gate", input_gate, input_gate_strides, 3, blc, e, false, true));
  CCV_TRY(t.add("rate", rate, &rate_stride, 1, cc, 4, false, true));
  CCV_TRY(t.add("seq_idx", seq_idx, seq_idx_strides, 2, bl, 4, false, false));
  CCV_TRY(t.add("initial_state", initial_state, initial_state_strides, 2, bc, 4, false, false));
  CCV_TRY(t.add("dout", dout, dout_strides, 3, blc, e, false, true));
  CCV_TRY(t.add("dfinal_state", dfinal_state, dfinal_state_strides, 2, bc, 4, false, false));
  CCV_TRY(t.add("chunk_states", chunk_states, chunk_states_strides, 3, cs, 4, false, false));
  CCV_TRY(t.add("dx", dx, dx_strides, 3, blc, e, true, true));
  CCV_TRY(t.add("ddecay_gate", ddecay_gate, ddecay_gate_strides, 3, blc, e, true, true));
  CCV_TRY(t.add("dinput_gate", dinput_gate, dinput_gate_strides, 3, blc, e, true, true));
  CCV_TRY(t.add("drate", drate, &drate_stride, 1, cc, 4, true, true));
  CCV_TRY(t.add("dinitial_state", dinitial_state, dinitial_state_strides, 2, bc, 4, true, false));
  const GlrBwdWorkspace w = glr_bwd_workspace(B, L, C);
  CCV_TRY(add_workspace(t, workspace, workspace_bytes, w.total, 128));
  CCV_TRY(t.disjoint());
  const ccv::Dtype dt = static_cast<ccv::Dtype>(dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ccv::GlrArgs a = {};
  a.x = x, a.p = decay_gate, a.q = input_gate, a.rate = rate, a.rs = rate_stride, a.seq = seq_idx;
  a.s0 = initial_state, a.n_slots = B;
  copy(a.xs, x_strides, 3), copy(a.ps, decay_gate_strides, 3), copy(a.qs, input_gate_strides, 3);
  copy(a.ss, seq_idx_strides, 2), copy(a.s0s, initial_state_strides, 2);
  a.B = B, a.L = L, a.C = C;
  cudaError_t err = cudaSuccess;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t *chain = ws + w.states + w.part, *chain_states = chain + w.chain;
  ccv::Device dev;
  CCV_TRY(static_cast<ccv_status>(ccv::api_device(&dev)));
  if (chunk_states != nullptr) {
    a.cs = const_cast<float*>(chunk_states);
    copy(a.css, chunk_states_strides, 3);
    if (w.chain > 0) err = cudaMemsetAsync(chain, 0xff, w.chain, s);
  } else if (B > 0 && L > 0) {
    if (w.chain > 0) err = cudaMemsetAsync(chain, 0xff, 2 * w.chain, s);
    a.cs = reinterpret_cast<float*>(ws);
    a.css[0] = glr_chunks(L) * C, a.css[1] = C, a.css[2] = 1;
    if (err == cudaSuccess) err = ccv::launch_glr_fwd(a, chain_states, dt, dev, s);
  }
  ccv::GlrGrads g = {};
  g.dout = dout, g.ds1 = dfinal_state, g.dx = dx, g.dp = ddecay_gate, g.dq = dinput_gate, g.drate = drate;
  g.drs = drate_stride, g.ds0 = dinitial_state;
  copy(g.dos, dout_strides, 3), copy(g.ds1s, dfinal_state_strides, 2), copy(g.dxs, dx_strides, 3);
  copy(g.dps, ddecay_gate_strides, 3), copy(g.dqs, dinput_gate_strides, 3), copy(g.ds0s, dinitial_state_strides, 2);
  g.part = reinterpret_cast<float*>(ws + w.states);
  if (err == cudaSuccess && B > 0 && L > 0) err = ccv::launch_glr_bwd(a, g, chain, dt, dev, s);
  if (err == cudaSuccess && L == 0 && dinitial_state != nullptr && B > 0) {
    // no tokens: the state passes through
    ccv::GlrArgs c = {};
    c.rate = rate, c.rs = rate_stride, c.s0 = dfinal_state, c.s1 = dinitial_state, c.B = B, c.C = C, c.n_slots = B;
    copy(c.s0s, dfinal_state_strides, 2), copy(c.s1s, dinitial_state_strides, 2);
    err = ccv::launch_glr_step(c, dt, s);
  }
  if (err == cudaSuccess)
    err = ccv::launch_glr_rate(g.part, L > 0 ? B * glr_chunks(L) : 0, C, drate, drate_stride, s);
  return launched(err, "glr_bwd");
}

}  // extern "C"

namespace {

ccv_status check_gn(int64_t N, int64_t S, int64_t C, int64_t G, float eps, ccv_activation act, ccv_dtype dtype,
                    ccv_dtype wdtype) {
  if (N < 0 || S < 0 || C < 0) CCV_FAIL(CCV_ERR_INVALID_ARG, "N, S and C must be >= 0");
  if (!valid_dtype(dtype)) CCV_FAIL(CCV_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
  if (!valid_dtype(wdtype)) CCV_FAIL(CCV_ERR_INVALID_ARG, "unknown weight dtype %d", static_cast<int>(wdtype));
  if (act != CCV_ACT_NONE && act != CCV_ACT_SILU)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "unknown activation %d", static_cast<int>(act));
  if (G < 1 || C % G != 0)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "C must be a multiple of groups (got %lld, %lld)", (long long)C, (long long)G);
  // a thread's sums over a slab stay within 2^11 terms (see gn_plan)
  if (C / G > (1 << 18)) CCV_FAIL(CCV_ERR_INVALID_ARG, "groups of at most 262144 channels");
  if (!(eps >= 0.f)) CCV_FAIL(CCV_ERR_INVALID_ARG, "eps must be >= 0");
  const __int128 lim = static_cast<__int128>(INT64_MAX) >> 8;
  const __int128 nc = static_cast<__int128>(N) * C;
  if (nc > lim || nc * (S > 0 ? S : 1) > lim || N > 0x7fffffff || S > 0x7fffffff || C > 0x7fffffff / 4)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "N*S*C is too large");
  const ccv::GnPlan p = ccv::gn_plan(N, S, C, G);
  if (static_cast<__int128>(N) * G * p.slabs > 0x7fffffff) CCV_FAIL(CCV_ERR_INVALID_ARG, "N*S*C is too large");
  return CCV_OK;
}

struct GnWorkspace {
  uint64_t stats, sums, part, total;
};

GnWorkspace gn_workspace(int64_t N, int64_t S, int64_t C, int64_t G, bool backward, bool params) {
  GnWorkspace w = {0, 0, 0, 0};
  if (N == 0 || S == 0 || C == 0) return w;
  const ccv::GnPlan p = ccv::gn_plan(N, S, C, G);
  if (p.slabs > 1) {
    w.stats = up256(static_cast<uint64_t>(N * G * p.slabs) * 8);
    if (backward) w.sums = w.stats;
  }
  if (params) w.part = up256(static_cast<uint64_t>(ccv::gn_parts(N, S, C, G)) * 8 * static_cast<uint64_t>(C));
  w.total = w.stats + w.sums + w.part;
  return w;
}

}  // namespace

extern "C" {

ccv_status ccv_gn_fwd_workspace_size(int64_t N, int64_t S, int64_t C, int64_t groups, uint64_t* bytes) {
  ccv::api_begin();
  if (bytes == nullptr) CCV_FAIL(CCV_ERR_INVALID_ARG, "bytes is required");
  CCV_TRY(check_gn(N, S, C, groups, 0.f, CCV_ACT_NONE, CCV_F32, CCV_F32));
  *bytes = gn_workspace(N, S, C, groups, false, false).total;
  return CCV_OK;
}

ccv_status ccv_gn_fwd(const void* x, const int64_t x_strides[3], const void* weight, int64_t weight_stride,
                      const void* bias, int64_t bias_stride, void* out, const int64_t out_strides[3], void* workspace,
                      uint64_t workspace_bytes, int64_t N, int64_t S, int64_t C, int64_t groups, float eps,
                      ccv_activation activation, ccv_dtype dtype, ccv_dtype weight_dtype, void* stream) {
  ccv::api_begin();
  CCV_TRY(check_gn(N, S, C, groups, eps, activation, dtype, weight_dtype));
  if (N == 0 || S == 0 || C == 0) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  const int64_t nsc[3] = {N, S, C}, c[1] = {C};
  const int64_t e = dtype_size(dtype), we = dtype_size(weight_dtype);
  Tensors t;
  CCV_TRY(t.add("x", x, x_strides, 3, nsc, e, false, true));
  CCV_TRY(t.add("weight", weight, &weight_stride, 1, c, we, false, false));
  CCV_TRY(t.add("bias", bias, &bias_stride, 1, c, we, false, false));
  CCV_TRY(t.add("out", out, out_strides, 3, nsc, e, true, true));
  const GnWorkspace w = gn_workspace(N, S, C, groups, false, false);
  CCV_TRY(add_workspace(t, workspace, workspace_bytes, w.total, 128));
  CCV_TRY(t.disjoint());
  ccv::GnArgs a = {};
  a.x = x, a.w = weight, a.ws = weight_stride, a.b = bias, a.bs = bias_stride, a.out = out;
  copy(a.xs, x_strides, 3), copy(a.os, out_strides, 3);
  a.stats = static_cast<float2*>(workspace);
  a.N = N, a.S = S, a.C = C, a.G = groups, a.eps = eps, a.wdt = static_cast<int>(weight_dtype);
  a.silu = activation == CCV_ACT_SILU;
  return launched(ccv::launch_gn_fwd(a, static_cast<ccv::Dtype>(dtype), static_cast<cudaStream_t>(stream)), "gn_fwd");
}

ccv_status ccv_gn_bwd_workspace_size(int64_t N, int64_t S, int64_t C, int64_t groups, uint64_t* bytes) {
  ccv::api_begin();
  if (bytes == nullptr) CCV_FAIL(CCV_ERR_INVALID_ARG, "bytes is required");
  CCV_TRY(check_gn(N, S, C, groups, 0.f, CCV_ACT_NONE, CCV_F32, CCV_F32));
  *bytes = gn_workspace(N, S, C, groups, true, true).total;
  return CCV_OK;
}

ccv_status ccv_gn_bwd(const void* x, const int64_t x_strides[3], const void* weight, int64_t weight_stride,
                      const void* bias, int64_t bias_stride, const void* dout, const int64_t dout_strides[3], void* dx,
                      const int64_t dx_strides[3], void* dweight, int64_t dweight_stride, void* dbias,
                      int64_t dbias_stride, void* workspace, uint64_t workspace_bytes, int64_t N, int64_t S, int64_t C,
                      int64_t groups, float eps, ccv_activation activation, ccv_dtype dtype, ccv_dtype weight_dtype,
                      void* stream) {
  ccv::api_begin();
  CCV_TRY(check_gn(N, S, C, groups, eps, activation, dtype, weight_dtype));
  if (C == 0) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  const int64_t nsc[3] = {N, S, C}, c[1] = {C};
  const int64_t e = dtype_size(dtype), we = dtype_size(weight_dtype);
  const bool params = dweight != nullptr || dbias != nullptr;
  Tensors t;
  CCV_TRY(t.add("x", x, x_strides, 3, nsc, e, false, true));
  CCV_TRY(t.add("weight", weight, &weight_stride, 1, c, we, false, false));
  CCV_TRY(t.add("bias", bias, &bias_stride, 1, c, we, false, false));
  CCV_TRY(t.add("dout", dout, dout_strides, 3, nsc, e, false, true));
  CCV_TRY(t.add("dx", dx, dx_strides, 3, nsc, e, true, true));
  CCV_TRY(t.add("dweight", dweight, &dweight_stride, 1, c, we, true, false));
  CCV_TRY(t.add("dbias", dbias, &dbias_stride, 1, c, we, true, false));
  const GnWorkspace w = gn_workspace(N, S, C, groups, true, params);
  CCV_TRY(add_workspace(t, workspace, workspace_bytes, w.total, 128));
  CCV_TRY(t.disjoint());
  if ((N == 0 || S == 0) && !params) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  ccv::GnArgs a = {};
  a.x = x, a.w = weight, a.ws = weight_stride, a.b = bias, a.bs = bias_stride, a.dout = dout, a.dx = dx;
  a.dw = dweight, a.dws = dweight_stride, a.db = dbias, a.dbs = dbias_stride;
  copy(a.xs, x_strides, 3), copy(a.gs, dout_strides, 3), copy(a.dxs, dx_strides, 3);
  a.stats = reinterpret_cast<float2*>(ws), a.sums = reinterpret_cast<float2*>(ws + w.stats);
  a.part = w.part > 0 ? reinterpret_cast<float*>(ws + w.stats + w.sums) : nullptr;
  a.N = N, a.S = S, a.C = C, a.G = groups, a.eps = eps, a.wdt = static_cast<int>(weight_dtype);
  a.silu = activation == CCV_ACT_SILU;
  return launched(ccv::launch_gn_bwd(a, static_cast<ccv::Dtype>(dtype), static_cast<cudaStream_t>(stream)), "gn_bwd");
}

}  // extern "C"

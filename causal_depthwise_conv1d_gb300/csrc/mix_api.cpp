// C-ABI front end of the gated delta rule (ccv_gdr_*) and of layer
// normalisation (ccv_ln_*): argument validation, kernel selection and launch
// on the caller's stream.  See include/ccv.h for the contract.
#include "api_check.h"
#include "mix_internal.h"

namespace {

// The chunked kernels take Dk up to kGdrChunkDk.  They cost about 20 us before
// their first chunk (FP32, with two terms of k and q, 30), the token-by-token
// kernel 0.37 us a token while its blocks, three an SM of 152, run at once:
// 64 tokens of 32 heads of 128 take 22.6 against 28.7 us in bf16, 48 of them 22.3
// against 22.6, of 256 heads 53 against 84 (FP32 74 against 88), and 77 tokens of
// 24 heads in FP32 39.2 against 31.3.  (152: the workspace's size, which follows
// from this, is a function of the sizes alone.)
bool gdr_chunked(int64_t B, int64_t L, int64_t Hv, int64_t Dk, int64_t Dv, ccv_dtype dtype) {
  if (Dk > ccv::kGdrChunkDk) return false;
  const bool at_once = B * Hv * ((Dv + 31) / 32) <= 3 * 152;
  return L >= (dtype == CCV_F32 && at_once ? 96 : 48);
}
int gdr_chunks(int64_t L) { return static_cast<int>((L + ccv::kGdrChunk - 1) / ccv::kGdrChunk); }

struct GdrWorkspace {
  uint64_t qk, pack, total;
};

GdrWorkspace gdr_workspace(int64_t B, int64_t L, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, ccv_dtype dtype) {
  GdrWorkspace w = {0, 0, 0};
  if (B == 0 || Hv == 0 || Dv == 0 || !gdr_chunked(B, L, Hv, Dk, Dv, dtype)) return w;
  ccv::GdrArgs a = {};
  a.B = B, a.L = L, a.Hk = Hk, a.Hv = Hv, a.Dk = Dk, a.Dv = Dv;
  w.qk = ccv::gdr_qk_bytes(a, static_cast<ccv::Dtype>(dtype), gdr_chunks(L));
  w.pack = ccv::gdr_pack_bytes(a, gdr_chunks(L));
  w.total = w.qk + w.pack;
  return w;
}

// The backward pass: every part on a 256-byte boundary.
struct GdrBwdWorkspace {
  uint64_t qk, pack, img_f, img_b, total;
};

GdrBwdWorkspace gdr_bwd_workspace(int64_t B, int64_t L, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv,
                                  ccv_dtype dtype) {
  GdrBwdWorkspace w = {0, 0, 0, 0, 0};
  if (B == 0 || Hv == 0 || Dv == 0 || L == 0) return w;
  ccv::GdrArgs a = {};
  a.B = B, a.L = L, a.Hk = Hk, a.Hv = Hv, a.Dk = Dk, a.Dv = Dv;
  const ccv::Dtype dt = static_cast<ccv::Dtype>(dtype);
  const int nc = gdr_chunks(L);
  const uint64_t slices = static_cast<uint64_t>(B * Hv) * nc * static_cast<uint64_t>((Dv + 15) / 16);
  auto up = [](uint64_t x) { return (x + 255) / 256 * 256; };
  w.qk = up(ccv::gdr_qk_bytes(a, dt, nc));
  w.pack = up(ccv::gdr_pack_bytes(a, nc));
  w.img_f = up(slices * ccv::gdr_img_f_bytes(Dk));
  w.img_b = up(slices * ccv::gdr_img_b_bytes(Dk, dt));
  w.total = w.qk + w.pack + w.img_f + w.img_b;
  return w;
}

ccv_status check_gdr_sizes(int64_t B, int64_t L, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, int64_t max_dk,
                           ccv_dtype dtype) {
  if (B < 0 || L < 0 || Hk < 0 || Hv < 0 || Dk < 0 || Dv < 0)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "B, L, Hk, Hv, Dk and Dv must be >= 0");
  if (!valid_dtype(dtype)) CCV_FAIL(CCV_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
  if (Hv > 0 && (Hk == 0 || Hv % Hk != 0))
    CCV_FAIL(CCV_ERR_INVALID_ARG, "Hv must be a multiple of Hk (got %lld, %lld)", (long long)Hv, (long long)Hk);
  if (Dk > max_dk)
    CCV_FAIL(CCV_ERR_UNSUPPORTED, "Dk must be at most %lld (got %lld)", (long long)max_dk, (long long)Dk);
  if (Dk == 0 && Hv > 0 && Dv > 0) CCV_FAIL(CCV_ERR_INVALID_ARG, "Dk must be >= 1");
  // counts and the index arithmetic on them stay within int64, grids within int32
  const __int128 lim = static_cast<__int128>(INT64_MAX) >> 8;
  const __int128 n = static_cast<__int128>(B) * (L > 0 ? L : 1) * (Hv > 0 ? Hv : 1);
  if (n > lim || n * (Dv > 0 ? Dv : 1) > lim || n * (Dk > 0 ? Dk : 1) > lim || L > 0x7fffffc0)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "B*L*Hv*Dv is too large");
  if (static_cast<__int128>(B) * Hv * ((Dv + 15) / 16) > 0x7fffffff ||
      static_cast<__int128>(B) * Hk * ((L + ccv::kGdrChunk - 1) / ccv::kGdrChunk) > 0x7fffffff)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "B*Hv*Dv is too large");
  return CCV_OK;
}

ccv_status check_bwd_dv(int64_t Dv) {
  if (Dv > ccv::kGdrBwdDv)
    CCV_FAIL(CCV_ERR_UNSUPPORTED, "Dv must be at most %d (got %lld)", ccv::kGdrBwdDv, (long long)Dv);
  return CCV_OK;
}

}  // namespace

extern "C" {

ccv_status ccv_gdr_fwd(const void* q, const int64_t q_strides[4], const void* k, const int64_t k_strides[4],
                       const void* v, const int64_t v_strides[4], const float* g, const int64_t g_strides[3],
                       const void* beta, const int64_t beta_strides[3], const int32_t* seq_idx,
                       const int64_t seq_idx_strides[2], const float* initial_state,
                       const int64_t initial_state_strides[4], void* out, const int64_t out_strides[4],
                       float* final_state_out, const int64_t final_state_strides[4], void* workspace,
                       uint64_t workspace_bytes, int64_t B, int64_t L, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv,
                       float scale, ccv_dtype dtype, void* stream) {
  ccv::api_begin();
  CCV_TRY(check_gdr_sizes(B, L, Hk, Hv, Dk, Dv, ccv::kGdrMaxDk, dtype));
  if (B == 0 || Hv == 0 || Dv == 0) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  const int64_t e = dtype_size(dtype);
  const int64_t qk[4] = {B, L, Hk, Dk}, vo[4] = {B, L, Hv, Dv}, gate[3] = {B, L, Hv}, st[4] = {B, Hv, Dk, Dv},
                ids[2] = {B, L};
  Tensors t;
  CCV_TRY(t.add("q", q, q_strides, 4, qk, e, false, true));
  CCV_TRY(t.add("k", k, k_strides, 4, qk, e, false, true));
  CCV_TRY(t.add("v", v, v_strides, 4, vo, e, false, true));
  CCV_TRY(t.add("g", g, g_strides, 3, gate, 4, false, true));
  CCV_TRY(t.add("beta", beta, beta_strides, 3, gate, e, false, true));
  CCV_TRY(t.add("seq_idx", seq_idx, seq_idx_strides, 2, ids, 4, false, false));
  CCV_TRY(t.add("initial_state", initial_state, initial_state_strides, 4, st, 4, false, false));
  CCV_TRY(t.add("out", out, out_strides, 4, vo, e, true, true));
  CCV_TRY(t.add("final_state_out", final_state_out, final_state_strides, 4, st, 4, true, false));
  const GdrWorkspace w = gdr_workspace(B, L, Hk, Hv, Dk, Dv, dtype);
  CCV_TRY(add_workspace(t, workspace, workspace_bytes, w.total, 128));
  CCV_TRY(t.disjoint());
  if (L == 0 && final_state_out == nullptr) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  ccv::Device dev;
  CCV_TRY(static_cast<ccv_status>(ccv::api_device(&dev)));
  ccv::GdrArgs a = {};
  a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.seq = seq_idx, a.s0 = initial_state, a.s1 = final_state_out;
  a.out = out;
  copy(a.qs, q_strides, 4), copy(a.ks, k_strides, 4), copy(a.vs, v_strides, 4), copy(a.gs, g_strides, 3);
  copy(a.bs, beta_strides, 3), copy(a.ss, seq_idx_strides, 2), copy(a.s0s, initial_state_strides, 4);
  copy(a.s1s, final_state_strides, 4), copy(a.os, out_strides, 4);
  a.B = B, a.L = L, a.Hk = Hk, a.Hv = Hv, a.Dk = Dk, a.Dv = Dv, a.scale = scale;
  const ccv::Dtype dt = static_cast<ccv::Dtype>(dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (w.total == 0) return launched(ccv::launch_gdr_token(a, dt, s), "gdr_token");
  uint8_t* qk_ws = static_cast<uint8_t*>(workspace);
  uint8_t* pack_ws = qk_ws + w.qk;
  cudaError_t err = ccv::launch_gdr_prep(a, dt, qk_ws, pack_ws, gdr_chunks(L), s);
  if (err == cudaSuccess) err = ccv::launch_gdr_scan(a, dt, qk_ws, pack_ws, nullptr, gdr_chunks(L), dev, s);
  return launched(err, "gdr_chunk");
}

ccv_status ccv_gdr_fwd_workspace_size(int64_t B, int64_t L, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv,
                                      ccv_dtype dtype, uint64_t* bytes) {
  ccv::api_begin();
  if (bytes == nullptr) CCV_FAIL(CCV_ERR_INVALID_ARG, "bytes is required");
  CCV_TRY(check_gdr_sizes(B, L, Hk, Hv, Dk, Dv, ccv::kGdrMaxDk, dtype));
  *bytes = gdr_workspace(B, L, Hk, Hv, Dk, Dv, dtype).total;
  return CCV_OK;
}

ccv_status ccv_gdr_step(const void* q, const int64_t q_strides[4], const void* k, const int64_t k_strides[4],
                        const void* v, const int64_t v_strides[4], const float* g, const int64_t g_strides[3],
                        const void* beta, const int64_t beta_strides[3], float* state, const int64_t state_strides[4],
                        int64_t n_slots, const int32_t* state_indices, int64_t state_indices_stride, void* out,
                        const int64_t out_strides[4], int64_t B, int64_t S, int64_t Hk, int64_t Hv, int64_t Dk,
                        int64_t Dv, float scale, ccv_dtype dtype, void* stream) {
  ccv::api_begin();
  CCV_TRY(check_gdr_sizes(B, S, Hk, Hv, Dk, Dv, ccv::kGdrMaxDk, dtype));
  if (n_slots < 0) CCV_FAIL(CCV_ERR_INVALID_ARG, "n_slots must be >= 0");
  if (state_indices == nullptr && n_slots < B)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "n_slots must be at least B without state_indices");
  if (B == 0 || Hv == 0 || Dv == 0 || S == 0) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  const int64_t e = dtype_size(dtype);
  const int64_t qk[4] = {B, S, Hk, Dk}, vo[4] = {B, S, Hv, Dv}, gate[3] = {B, S, Hv},
                st[4] = {n_slots, Hv, Dk, Dv}, idx[1] = {B};
  Tensors t;
  CCV_TRY(t.add("q", q, q_strides, 4, qk, e, false, true));
  CCV_TRY(t.add("k", k, k_strides, 4, qk, e, false, true));
  CCV_TRY(t.add("v", v, v_strides, 4, vo, e, false, true));
  CCV_TRY(t.add("g", g, g_strides, 3, gate, 4, false, true));
  CCV_TRY(t.add("beta", beta, beta_strides, 3, gate, e, false, true));
  CCV_TRY(t.add("state_indices", state_indices, &state_indices_stride, 1, idx, 4, false, false));
  CCV_TRY(t.add("state", state, state_strides, 4, st, 4, true, true));
  CCV_TRY(t.add("out", out, out_strides, 4, vo, e, true, true));
  CCV_TRY(t.disjoint());
  ccv::Device dev;
  CCV_TRY(static_cast<ccv_status>(ccv::api_device(&dev)));
  ccv::GdrArgs a = {};
  a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.s0 = state, a.s1 = state, a.out = out;
  a.slots = state_indices, a.slot_stride = state_indices_stride, a.n_slots = n_slots;
  copy(a.qs, q_strides, 4), copy(a.ks, k_strides, 4), copy(a.vs, v_strides, 4), copy(a.gs, g_strides, 3);
  copy(a.bs, beta_strides, 3), copy(a.s0s, state_strides, 4), copy(a.s1s, state_strides, 4);
  copy(a.os, out_strides, 4);
  a.B = B, a.L = S, a.Hk = Hk, a.Hv = Hv, a.Dk = Dk, a.Dv = Dv, a.scale = scale;
  const ccv::Dtype dt = static_cast<ccv::Dtype>(dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (ccv::gdr_step_eligible(a, dev)) return launched(ccv::launch_gdr_step(a, dt, s), "gdr_step");
  return launched(ccv::launch_gdr_token(a, dt, s), "gdr_step");
}

ccv_status ccv_gdr_bwd_workspace_size(int64_t B, int64_t L, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv,
                                      ccv_dtype dtype, uint64_t* bytes) {
  ccv::api_begin();
  if (bytes == nullptr) CCV_FAIL(CCV_ERR_INVALID_ARG, "bytes is required");
  CCV_TRY(check_gdr_sizes(B, L, Hk, Hv, Dk, Dv, ccv::kGdrChunkDk, dtype));
  CCV_TRY(check_bwd_dv(Dv));
  *bytes = gdr_bwd_workspace(B, L, Hk, Hv, Dk, Dv, dtype).total;
  return CCV_OK;
}

ccv_status ccv_gdr_bwd(const void* q, const int64_t q_strides[4], const void* k, const int64_t k_strides[4],
                       const void* v, const int64_t v_strides[4], const float* g, const int64_t g_strides[3],
                       const void* beta, const int64_t beta_strides[3], const int32_t* seq_idx,
                       const int64_t seq_idx_strides[2], const float* initial_state,
                       const int64_t initial_state_strides[4], const void* dout, const int64_t dout_strides[4],
                       const float* dfinal_state, const int64_t dfinal_state_strides[4], void* dq,
                       const int64_t dq_strides[4], void* dk, const int64_t dk_strides[4], void* dv,
                       const int64_t dv_strides[4], float* dg, const int64_t dg_strides[3], void* dbeta,
                       const int64_t dbeta_strides[3], float* dinitial_state, const int64_t dinitial_state_strides[4],
                       void* workspace, uint64_t workspace_bytes, int64_t B, int64_t L, int64_t Hk, int64_t Hv,
                       int64_t Dk, int64_t Dv, float scale, ccv_dtype dtype, void* stream) {
  ccv::api_begin();
  CCV_TRY(check_gdr_sizes(B, L, Hk, Hv, Dk, Dv, ccv::kGdrChunkDk, dtype));
  if (dinitial_state != nullptr && initial_state == nullptr)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "dinitial_state requires initial_state");
  if (B == 0 || Hv == 0) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  if (Dv == 0) CCV_FAIL(CCV_ERR_INVALID_ARG, "Dv must be >= 1");
  CCV_TRY(check_bwd_dv(Dv));
  const int64_t e = dtype_size(dtype);
  const int64_t qk[4] = {B, L, Hk, Dk}, vo[4] = {B, L, Hv, Dv}, gate[3] = {B, L, Hv}, st[4] = {B, Hv, Dk, Dv},
                ids[2] = {B, L};
  Tensors t;
  CCV_TRY(t.add("q", q, q_strides, 4, qk, e, false, true));
  CCV_TRY(t.add("k", k, k_strides, 4, qk, e, false, true));
  CCV_TRY(t.add("v", v, v_strides, 4, vo, e, false, true));
  CCV_TRY(t.add("g", g, g_strides, 3, gate, 4, false, true));
  CCV_TRY(t.add("beta", beta, beta_strides, 3, gate, e, false, true));
  CCV_TRY(t.add("seq_idx", seq_idx, seq_idx_strides, 2, ids, 4, false, false));
  CCV_TRY(t.add("initial_state", initial_state, initial_state_strides, 4, st, 4, false, false));
  CCV_TRY(t.add("dout", dout, dout_strides, 4, vo, e, false, true));
  CCV_TRY(t.add("dfinal_state", dfinal_state, dfinal_state_strides, 4, st, 4, false, false));
  CCV_TRY(t.add("dq", dq, dq_strides, 4, qk, e, true, true));
  CCV_TRY(t.add("dk", dk, dk_strides, 4, qk, e, true, true));
  CCV_TRY(t.add("dv", dv, dv_strides, 4, vo, e, true, true));
  CCV_TRY(t.add("dg", dg, dg_strides, 3, gate, 4, true, true));
  CCV_TRY(t.add("dbeta", dbeta, dbeta_strides, 3, gate, e, true, true));
  CCV_TRY(t.add("dinitial_state", dinitial_state, dinitial_state_strides, 4, st, 4, true, false));
  const GdrBwdWorkspace ws = gdr_bwd_workspace(B, L, Hk, Hv, Dk, Dv, dtype);
  CCV_TRY(add_workspace(t, workspace, workspace_bytes, ws.total, 128));
  CCV_TRY(t.disjoint());
  if (L == 0 && dinitial_state == nullptr) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  ccv::Device dev;
  CCV_TRY(static_cast<ccv_status>(ccv::api_device(&dev)));
  ccv::GdrArgs a = {};
  a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.seq = seq_idx, a.s0 = initial_state;
  copy(a.qs, q_strides, 4), copy(a.ks, k_strides, 4), copy(a.vs, v_strides, 4), copy(a.gs, g_strides, 3);
  copy(a.bs, beta_strides, 3), copy(a.ss, seq_idx_strides, 2), copy(a.s0s, initial_state_strides, 4);
  a.B = B, a.L = L, a.Hk = Hk, a.Hv = Hv, a.Dk = Dk, a.Dv = Dv, a.scale = scale;
  ccv::GdrGrads gr = {};
  gr.dout = dout, gr.ds1 = dfinal_state, gr.dq = dq, gr.dk = dk, gr.dv = dv, gr.dg = dg, gr.dbeta = dbeta;
  gr.ds0 = dinitial_state;
  copy(gr.dos, dout_strides, 4), copy(gr.ds1s, dfinal_state_strides, 4), copy(gr.dqs, dq_strides, 4);
  copy(gr.dks, dk_strides, 4), copy(gr.dvs, dv_strides, 4), copy(gr.dgs, dg_strides, 3);
  copy(gr.dbs, dbeta_strides, 3), copy(gr.ds0s, dinitial_state_strides, 4);
  const ccv::Dtype dt = static_cast<ccv::Dtype>(dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int nc = gdr_chunks(L);
  uint8_t* p = static_cast<uint8_t*>(workspace);
  uint8_t *qk_ws = p, *pack_ws = qk_ws + ws.qk;
  uint8_t *img_f = pack_ws + ws.pack, *img_b = img_f + ws.img_f;
  const ccv::GdrBwdWs w = {qk_ws, pack_ws, img_f, img_b};
  cudaError_t err = cudaSuccess;
  if (L > 0) {
    err = ccv::launch_gdr_prep(a, dt, qk_ws, pack_ws, nc, s);
    if (err == cudaSuccess) err = ccv::launch_gdr_scan(a, dt, qk_ws, pack_ws, img_f, nc, dev, s);
  }
  if (err == cudaSuccess) err = ccv::launch_gdr_bwd_scan(a, gr, dt, w, nc, dev, s);
  if (err == cudaSuccess && L > 0) err = ccv::launch_gdr_bwd_grad(a, gr, dt, w, nc, s);
  return launched(err, "gdr_bwd");
}

}  // extern "C"

namespace {

// Parameters that vector loads of four elements may read (or none).
bool dense_par(const void* p, int64_t stride, int64_t esz) {
  return p == nullptr || (stride == 1 && reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(4 * esz) == 0);
}

ccv_status check_ln(int64_t N, int64_t D, float eps, ccv_dtype dtype, ccv_dtype wdtype) {
  if (N < 0 || D < 0) CCV_FAIL(CCV_ERR_INVALID_ARG, "N and D must be >= 0");
  if (!valid_dtype(dtype)) CCV_FAIL(CCV_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
  if (!valid_dtype(wdtype)) CCV_FAIL(CCV_ERR_INVALID_ARG, "unknown weight dtype %d", static_cast<int>(wdtype));
  if (!(eps >= 0.f)) CCV_FAIL(CCV_ERR_INVALID_ARG, "eps must be >= 0");
  if (N > 0x7fffffff || D > 0x7fffffff / 2 || static_cast<__int128>(N) * D > (INT64_MAX >> 4))
    CCV_FAIL(CCV_ERR_INVALID_ARG, "N*D is too large");
  return CCV_OK;
}

}  // namespace

extern "C" {

ccv_status ccv_ln_fwd(const void* x, const int64_t x_strides[2], const void* weight, int64_t weight_stride,
                      const void* bias, int64_t bias_stride, void* out, const int64_t out_strides[2], int64_t N,
                      int64_t D, float eps, ccv_dtype dtype, ccv_dtype weight_dtype, void* stream) {
  ccv::api_begin();
  CCV_TRY(check_ln(N, D, eps, dtype, weight_dtype));
  if (N == 0 || D == 0) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  const int64_t nd[2] = {N, D}, d[1] = {D};
  const int64_t e = dtype_size(dtype), we = dtype_size(weight_dtype);
  Tensors t;
  CCV_TRY(t.add("x", x, x_strides, 2, nd, e, false, true));
  CCV_TRY(t.add("weight", weight, &weight_stride, 1, d, we, false, false));
  CCV_TRY(t.add("bias", bias, &bias_stride, 1, d, we, false, false));
  CCV_TRY(t.add("out", out, out_strides, 2, nd, e, true, true));
  CCV_TRY(t.disjoint());
  ccv::LnArgs a = {x, x_strides[0], x_strides[1], weight, weight_stride, bias, bias_stride,
                   out, out_strides[0], out_strides[1], N, D, eps, static_cast<int>(weight_dtype),
                   dense_par(weight, weight_stride, we) && dense_par(bias, bias_stride, we)};
  ccv::Device dev;
  CCV_TRY(static_cast<ccv_status>(ccv::api_device(&dev)));
  return launched(ccv::launch_ln_fwd(a, static_cast<ccv::Dtype>(dtype), dev, static_cast<cudaStream_t>(stream)),
                  "ln_fwd");
}

ccv_status ccv_ln_bwd_workspace_size(int64_t N, int64_t D, uint64_t* bytes) {
  ccv::api_begin();
  if (bytes == nullptr) CCV_FAIL(CCV_ERR_INVALID_ARG, "bytes is required");
  CCV_TRY(check_ln(N, D, 0.f, CCV_F32, CCV_F32));
  *bytes = static_cast<uint64_t>(ccv::ln_bwd_blocks(N, D)) * 2u * static_cast<uint64_t>(D) * sizeof(float);
  return CCV_OK;
}

ccv_status ccv_ln_bwd(const void* x, const int64_t x_strides[2], const void* weight, int64_t weight_stride,
                      const void* dout, const int64_t dout_strides[2], void* dx, const int64_t dx_strides[2],
                      void* dweight, int64_t dweight_stride, void* dbias, int64_t dbias_stride, void* workspace,
                      uint64_t workspace_bytes, int64_t N, int64_t D, float eps, ccv_dtype dtype,
                      ccv_dtype weight_dtype, void* stream) {
  ccv::api_begin();
  CCV_TRY(check_ln(N, D, eps, dtype, weight_dtype));
  if (D == 0) {
    ccv::api_kernel("none");
    return CCV_OK;
  }
  const int64_t nd[2] = {N, D}, d[1] = {D};
  const int64_t e = dtype_size(dtype), we = dtype_size(weight_dtype);
  const bool params = dweight != nullptr || dbias != nullptr;
  const uint64_t need =
      params ? static_cast<uint64_t>(ccv::ln_bwd_blocks(N, D)) * 2u * static_cast<uint64_t>(D) * sizeof(float) : 0;
  Tensors t;
  CCV_TRY(t.add("x", x, x_strides, 2, nd, e, false, true));
  CCV_TRY(t.add("weight", weight, &weight_stride, 1, d, we, false, false));
  CCV_TRY(t.add("dout", dout, dout_strides, 2, nd, e, false, true));
  CCV_TRY(t.add("dx", dx, dx_strides, 2, nd, e, true, true));
  CCV_TRY(t.add("dweight", dweight, &dweight_stride, 1, d, we, true, false));
  CCV_TRY(t.add("dbias", dbias, &dbias_stride, 1, d, we, true, false));
  CCV_TRY(add_workspace(t, workspace, workspace_bytes, need, 16));
  CCV_TRY(t.disjoint());
  ccv::LnBwdArgs a = {};
  a.x = x, a.w = weight, a.ws = weight_stride, a.dout = dout, a.dx = dx;
  a.dw = dweight, a.dws = dweight_stride, a.db = dbias, a.dbs = dbias_stride;
  a.part = need > 0 ? static_cast<float*>(workspace) : nullptr;
  if (N > 0) {
    a.xs0 = x_strides[0], a.xs1 = x_strides[1], a.gs0 = dout_strides[0], a.gs1 = dout_strides[1];
    a.dxs0 = dx_strides[0], a.dxs1 = dx_strides[1];
  }
  a.N = N, a.D = D, a.eps = eps, a.wdt = static_cast<int>(weight_dtype);
  a.wvec = dense_par(weight, weight_stride, we);
  return launched(ccv::launch_ln_bwd(a, static_cast<ccv::Dtype>(dtype), static_cast<cudaStream_t>(stream)), "ln_bwd");
}

}  // extern "C"

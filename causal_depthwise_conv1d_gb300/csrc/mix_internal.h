// Internal interface between the ABI front end of the gated delta rule and of
// layer normalisation (mix_api.cpp) and their launchers (gdr_*.cu, ln.cu).
#pragma once

#include "ccv_internal.h"

namespace ccv {

constexpr int kGdrChunk = 64;     // tokens of one chunk of the chunked kernels
constexpr int kGdrMaxDk = 256;    // largest key size of the token-by-token kernel
constexpr int kGdrChunkDk = 128;  // largest key size of the chunked kernels
constexpr int kGdrBwdDv = 512;    // largest value size of the backward pass

// Validated arguments of the gated delta rule.  q, k: [B,L,Hk,Dk]; v, out:
// [B,L,Hv,Dv]; g (FP32), beta: [B,L,Hv]; states FP32 [.,Hv,Dk,Dv].  Strides in
// elements, in the order of the dimensions.
struct GdrArgs {
  const void* q;
  int64_t qs[4];
  const void* k;
  int64_t ks[4];
  const void* v;
  int64_t vs[4];
  const float* g;
  int64_t gs[3];
  const void* beta;
  int64_t bs[3];
  const int32_t* seq;  // [B,L] or null
  int64_t ss[2];
  const float* s0;     // state before the first token, or null (zero)
  int64_t s0s[4];
  float* s1;           // state after the last token, or null
  int64_t s1s[4];
  const int32_t* slots;  // row b's state is s0[slots[b]] (null: s0[b])
  int64_t slot_stride, n_slots;
  void* out;
  int64_t os[4];
  int64_t B, L, Hk, Hv, Dk, Dv;
  float scale;
};

// Backward pass: the forward arguments (out, s1 unused) and these.
struct GdrGrads {
  const void* dout;
  int64_t dos[4];
  const float* ds1;  // gradient of the final state, or null
  int64_t ds1s[4];
  void* dq;
  int64_t dqs[4];
  void* dk;
  int64_t dks[4];
  void* dv;
  int64_t dvs[4];
  float* dg;
  int64_t dgs[3];
  void* dbeta;
  int64_t dbs[3];
  float* ds0;  // or null
  int64_t ds0s[4];
};

// One token after the other with the state in registers: sequences and decode
// steps of any sizes, and the decode step of a large batch.
bool gdr_vec4_state(const float* p, const int64_t* strides);
cudaError_t launch_gdr_token(const GdrArgs& a, Dtype dt, cudaStream_t stream);
bool gdr_step_eligible(const GdrArgs& a, const Device& dev);
cudaError_t launch_gdr_step(const GdrArgs& a, Dtype dt, cudaStream_t stream);

// Chunked forward pass: the parts that do not depend on the state (qk_ws,
// pack_ws: see gdr_chunk.cuh), then the scan that carries it.  nc = chunks.
cudaError_t launch_gdr_prep(const GdrArgs& a, Dtype dt, uint8_t* qk_ws, uint8_t* pack_ws, int nc,
                            cudaStream_t stream);
// For the backward pass (img given) the scan makes no output but keeps each
// chunk's first state and its U as images [b][h][chunk][16 value channels].
cudaError_t launch_gdr_scan(const GdrArgs& a, Dtype dt, const uint8_t* qk_ws, const uint8_t* pack_ws, uint8_t* img,
                            int nc, const Device& dev, cudaStream_t stream);

// Backward pass after these two: the reverse scan (dv, and its own images) and
// the gradients of one chunk each.
struct GdrBwdWs {
  const uint8_t *qk, *pack, *img_f;
  uint8_t* img_b;
};
cudaError_t launch_gdr_bwd_scan(const GdrArgs& a, const GdrGrads& g, Dtype dt, const GdrBwdWs& w, int nc,
                                const Device& dev, cudaStream_t stream);
cudaError_t launch_gdr_bwd_grad(const GdrArgs& a, const GdrGrads& g, Dtype dt, const GdrBwdWs& w, int nc,
                                cudaStream_t stream);
// Bytes of the images of one chunk, value head and 16 value channels.
uint64_t gdr_img_f_bytes(int64_t Dk);
uint64_t gdr_img_b_bytes(int64_t Dk, Dtype dt);
// Bytes of qk_ws and pack_ws.
uint64_t gdr_qk_bytes(const GdrArgs& a, Dtype dt, int nc);
uint64_t gdr_pack_bytes(const GdrArgs& a, int nc);
unsigned read_and_clear_fault_gdr();
unsigned read_and_clear_fault_gdr_bwd();
unsigned read_and_clear_fault_gdr_grad();

struct LnArgs {
  const void* x;
  int64_t xs0, xs1;
  const void* w;  // or null (one)
  int64_t ws;
  const void* b;  // or null (zero)
  int64_t bs;
  void* out;
  int64_t os0, os1;
  int64_t N, D;
  float eps;
  int wdt;
  bool wvec;  // weight and bias are dense and aligned to four elements
};

struct LnBwdArgs {
  const void* x;
  int64_t xs0, xs1;
  const void* w;
  int64_t ws;
  const void* dout;
  int64_t gs0, gs1;
  void* dx;
  int64_t dxs0, dxs1;
  void* dw;  // or null
  int64_t dws;
  void* db;  // or null
  int64_t dbs;
  float* part;  // [blocks][2][D] partial sums of dw and db, or null
  int64_t N, D;
  float eps;
  int wdt;
  bool wvec;  // weight and bias are dense and aligned to four elements
};

cudaError_t launch_ln_fwd(const LnArgs& a, Dtype dt, const Device& dev, cudaStream_t stream);
unsigned read_and_clear_fault_ln();
// Blocks (= partial sums) of the backward pass: a function of N and D alone.
int64_t ln_bwd_blocks(int64_t N, int64_t D);
cudaError_t launch_ln_bwd(const LnBwdArgs& a, Dtype dt, cudaStream_t stream);

}  // namespace ccv

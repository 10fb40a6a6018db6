// Tensor front end of the gated delta rule and layer normalisation: checks
// that need tensors, allocation of missing outputs and of the workspace, and
// the C-ABI call (include/ccv.h) on the stream.  It does what mixer.py would
// do in Python; a decode step or a small norm takes a few microseconds on the
// device, and marshalling eight tensors in Python several times that.
//
// Every function returns the ABI's status first; mixer.py turns a non-zero
// one into an exception.  Wrong shapes, types and devices raise ValueError.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <cmath>
#include <optional>
#include <sstream>
#include <string>
#include <tuple>

#include "ccv.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using Opt = std::optional<Tensor>;
using Shape = at::IntArrayRef;

ccv_dtype dtype_of(const Tensor& x, const char* what) {
  switch (x.scalar_type()) {
    case at::kFloat: return CCV_F32;
    case at::kHalf: return CCV_F16;
    case at::kBFloat16: return CCV_BF16;
    default: throw py::value_error(std::string("unsupported ") + what + " " + c10::toString(x.scalar_type()));
  }
}

void check(int dev, const char* name, const Tensor& t, Shape shape, at::ScalarType dtype) {
  if (t.is_cuda() && t.get_device() == dev && t.sizes() == shape && t.scalar_type() == dtype) return;
  if (!t.is_cuda() || t.get_device() != dev) throw py::value_error("all tensors must live on one CUDA device");
  std::ostringstream s;
  if (t.sizes() != shape)
    s << name << " must have shape " << shape << ", got " << t.sizes();
  else
    s << name << " must have dtype " << c10::toString(dtype) << ", got " << c10::toString(t.scalar_type());
  throw py::value_error(s.str());
}

void check(int dev, const char* name, const Opt& t, Shape shape, at::ScalarType dtype) {
  if (t) check(dev, name, *t, shape, dtype);
}

// The stream of the call: the one given, or the device's current one.
struct Stream {
  int dev;
  std::optional<c10::cuda::CUDAStream> given;
  Stream(int d, const std::optional<int64_t>& s) : dev(d) {
    if (s) given = c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(*s), static_cast<c10::DeviceIndex>(d));
  }
  void* raw() const {
    return given ? given->stream() : c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  }
  // A new tensor.  For a given stream it comes from that stream's memory: a
  // block freed on the current one may have kernels of the current stream
  // pending, which the given stream does not wait for.  The current stream is
  // where the caller will use it, so it is not reused before that is done either.
  Tensor empty(Shape shape, at::ScalarType dtype) const {
    const auto opt = at::TensorOptions().dtype(dtype).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev));
    if (!given) return at::empty(shape, opt);
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev));
    const c10::cuda::CUDAStreamGuard on(*given);
    Tensor t = at::empty(shape, opt);
    if (t.numel() > 0) t.record_stream(current.unwrap());
    return t;
  }
};

Tensor given(Opt& t, const Stream& s, const char* name, Shape shape, at::ScalarType dtype) {
  if (!t) return s.empty(shape, dtype);
  check(s.dev, name, *t, shape, dtype);
  return *t;
}

// Pointer and strides of a tensor or of a missing one.
const void* ptr(const Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }
void* out_ptr(const Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }
const void* ptr(const Opt& t) { return t ? ptr(*t) : nullptr; }
void* out_ptr(const Opt& t) { return t ? out_ptr(*t) : nullptr; }
const int64_t* str(const Tensor& t) { return t.strides().data(); }
const int64_t* str(const Opt& t) { return t ? t->strides().data() : nullptr; }
int64_t stride0(const Opt& t) { return t ? t->stride(0) : 0; }

int cuda_index(const Tensor& t) {
  if (!t.is_cuda()) throw py::value_error("all tensors must live on one CUDA device");
  return t.get_device();
}

// A workspace of `need` bytes: the caller's (its size is checked by the ABI), or a new one.
struct Workspace {
  Tensor own;
  void* p = nullptr;
  uint64_t bytes = 0;
  Workspace(const Opt& given, uint64_t need, const Stream& s) {
    if (given) {
      if (!given->is_cuda() || given->get_device() != s.dev || !given->is_contiguous())
        throw py::value_error("workspace must be a contiguous tensor on the inputs' CUDA device");
      p = given->data_ptr();
      bytes = static_cast<uint64_t>(given->numel()) * given->element_size();
    } else if (need > 0) {
      own = s.empty({static_cast<int64_t>(need)}, at::kByte);
      p = own.data_ptr();
      bytes = need;
    }
  }
};

struct Sizes {
  int64_t B, L, Hk, Hv, Dk, Dv;
  ccv_dtype dt;
  at::ScalarType type;
  int dev;
  float scale;
};

Sizes sizes(const Tensor& q, const Tensor& k, const Tensor& v, const std::optional<double>& scale) {
  if (q.dim() != 4 || k.dim() != 4 || v.dim() != 4)
    throw py::value_error("q and k must be [B, L, Hk, Dk] and v [B, L, Hv, Dv]");
  Sizes s;
  s.dt = dtype_of(v, "dtype");
  s.B = q.size(0), s.L = q.size(1), s.Hk = q.size(2), s.Dk = q.size(3), s.Hv = v.size(2), s.Dv = v.size(3);
  s.type = v.scalar_type();
  s.dev = cuda_index(v);
  s.scale = static_cast<float>(scale ? *scale : 1.0 / std::sqrt(static_cast<double>(s.Dk > 0 ? s.Dk : 1)));
  return s;
}

void check_inputs(const Sizes& s, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g,
                  const Tensor& beta) {
  check(s.dev, "q", q, {s.B, s.L, s.Hk, s.Dk}, s.type);
  check(s.dev, "k", k, {s.B, s.L, s.Hk, s.Dk}, s.type);
  check(s.dev, "v", v, {s.B, s.L, s.Hv, s.Dv}, s.type);
  check(s.dev, "g", g, {s.B, s.L, s.Hv}, at::kFloat);
  check(s.dev, "beta", beta, {s.B, s.L, s.Hv}, s.type);
}

const float* f32(const void* p) { return static_cast<const float*>(p); }
float* f32(void* p) { return static_cast<float*>(p); }

std::tuple<int, Tensor, Opt> gdr_fwd(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g,
                                     const Tensor& beta, std::optional<double> scale, const Opt& seq_idx,
                                     const Opt& initial_state, bool want_final, Opt final_out, Opt out_given,
                                     const Opt& workspace, std::optional<int64_t> stream) {
  const Sizes s = sizes(q, k, v, scale);
  check_inputs(s, q, k, v, g, beta);
  check(s.dev, "seq_idx", seq_idx, {s.B, s.L}, at::kInt);
  check(s.dev, "initial_state", initial_state, {s.B, s.Hv, s.Dk, s.Dv}, at::kFloat);
  const c10::cuda::OptionalCUDAGuard guard(v.device());
  const Stream on(s.dev, stream);
  const Tensor out = given(out_given, on, "out", {s.B, s.L, s.Hv, s.Dv}, s.type);
  if (want_final || final_out)
    final_out = given(final_out, on, "final_state_out", {s.B, s.Hv, s.Dk, s.Dv}, at::kFloat);
  uint64_t need = 0;
  int rc = ccv_gdr_fwd_workspace_size(s.B, s.L, s.Hk, s.Hv, s.Dk, s.Dv, s.dt, &need);
  if (rc == CCV_OK) {
    const Workspace w(workspace, need, on);
    rc = ccv_gdr_fwd(ptr(q), str(q), ptr(k), str(k), ptr(v), str(v), f32(ptr(g)), str(g), ptr(beta), str(beta),
                     static_cast<const int32_t*>(ptr(seq_idx)), str(seq_idx), f32(ptr(initial_state)),
                     str(initial_state), out_ptr(out), str(out), f32(out_ptr(final_out)), str(final_out), w.p, w.bytes,
                     s.B, s.L, s.Hk, s.Hv, s.Dk, s.Dv, s.scale, s.dt, on.raw());
  }
  return {rc, out, final_out};
}

std::tuple<int, Tensor> gdr_step(const Tensor& q_, const Tensor& k_, const Tensor& v_, const Tensor& g_,
                                 const Tensor& beta_, const Tensor& state, std::optional<double> scale,
                                 const Opt& state_indices, Opt out_given, std::optional<int64_t> stream) {
  const bool one = v_.dim() == 3;
  auto tok = [one](const Tensor& x) { return one ? x.unsqueeze(1) : x; };
  const Tensor q = tok(q_), k = tok(k_), v = tok(v_), g = tok(g_), beta = tok(beta_);
  const Sizes s = sizes(q, k, v, scale);
  if (state.dim() != 4) throw py::value_error("state must be [n_slots, Hv, Dk, Dv]");
  check_inputs(s, q, k, v, g, beta);
  check(s.dev, "state", state, {state.size(0), s.Hv, s.Dk, s.Dv}, at::kFloat);
  check(s.dev, "state_indices", state_indices, {s.B}, at::kInt);
  const c10::cuda::OptionalCUDAGuard guard(v.device());
  const Stream on(s.dev, stream);
  Opt shaped = out_given ? Opt(tok(*out_given)) : Opt();
  const Tensor out = given(shaped, on, "out", {s.B, s.L, s.Hv, s.Dv}, s.type);
  const int rc = ccv_gdr_step(ptr(q), str(q), ptr(k), str(k), ptr(v), str(v), f32(ptr(g)), str(g), ptr(beta), str(beta),
                              f32(out_ptr(state)), str(state), state.size(0),
                              static_cast<const int32_t*>(ptr(state_indices)), stride0(state_indices), out_ptr(out),
                              str(out), s.B, s.L, s.Hk, s.Hv, s.Dk, s.Dv, s.scale, s.dt, on.raw());
  return {rc, out_given ? *out_given : one ? out.squeeze(1) : out};
}

std::tuple<int, Tensor, Tensor, Tensor, Tensor, Tensor, Opt> gdr_bwd(
    const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g, const Tensor& beta, const Tensor& dout,
    std::optional<double> scale, const Opt& seq_idx, const Opt& initial_state, const Opt& dfinal_state, Opt dq_, Opt dk_,
    Opt dv_, Opt dg_, Opt dbeta_, Opt ds0, bool want_ds0, const Opt& workspace, std::optional<int64_t> stream) {
  const Sizes s = sizes(q, k, v, scale);
  check_inputs(s, q, k, v, g, beta);
  const int64_t qk[4] = {s.B, s.L, s.Hk, s.Dk}, vo[4] = {s.B, s.L, s.Hv, s.Dv}, gate[3] = {s.B, s.L, s.Hv},
                st[4] = {s.B, s.Hv, s.Dk, s.Dv};
  check(s.dev, "seq_idx", seq_idx, {s.B, s.L}, at::kInt);
  check(s.dev, "initial_state", initial_state, st, at::kFloat);
  check(s.dev, "dout", dout, vo, s.type);
  check(s.dev, "dfinal_state", dfinal_state, st, at::kFloat);
  const c10::cuda::OptionalCUDAGuard guard(v.device());
  const Stream on(s.dev, stream);
  const Tensor dq = given(dq_, on, "dq", qk, s.type), dk = given(dk_, on, "dk", qk, s.type);
  const Tensor dv = given(dv_, on, "dv", vo, s.type), dg = given(dg_, on, "dg", gate, at::kFloat);
  const Tensor dbeta = given(dbeta_, on, "dbeta", gate, s.type);
  if (ds0 || (want_ds0 && initial_state)) ds0 = given(ds0, on, "dinitial_state", st, at::kFloat);
  uint64_t need = 0;
  int rc = ccv_gdr_bwd_workspace_size(s.B, s.L, s.Hk, s.Hv, s.Dk, s.Dv, s.dt, &need);
  if (rc == CCV_OK) {
    const Workspace w(workspace, need, on);
    rc = ccv_gdr_bwd(ptr(q), str(q), ptr(k), str(k), ptr(v), str(v), f32(ptr(g)), str(g), ptr(beta), str(beta),
                     static_cast<const int32_t*>(ptr(seq_idx)), str(seq_idx), f32(ptr(initial_state)),
                     str(initial_state), ptr(dout), str(dout), f32(ptr(dfinal_state)), str(dfinal_state), out_ptr(dq),
                     str(dq), out_ptr(dk), str(dk), out_ptr(dv), str(dv), f32(out_ptr(dg)), str(dg), out_ptr(dbeta),
                     str(dbeta), f32(out_ptr(ds0)), str(ds0), w.p, w.bytes, s.B, s.L, s.Hk, s.Hv, s.Dk, s.Dv, s.scale,
                     s.dt, on.raw());
  }
  return {rc, dq, dk, dv, dg, dbeta, ds0};
}

// [..., D] as [N, D] without a copy: the strides of both dimensions.
struct Rows {
  int64_t strides[2];
};
Rows rows(const Tensor& x) {
  Rows r = {{0, 1}};
  const int64_t nd = x.dim();
  r.strides[1] = x.stride(nd - 1);
  int64_t step = 0;
  bool first = true;
  for (int64_t d = nd - 2; d >= 0; --d) {
    if (x.size(d) == 1) continue;
    if (first) {
      r.strides[0] = x.stride(d);
      first = false;
    } else if (x.stride(d) != step) {
      throw py::value_error(
          "the leading dimensions of a layer norm's tensor must collapse into one stride (pass a 2-D view)");
    }
    step = x.stride(d) * x.size(d);
  }
  if (first) r.strides[0] = x.size(nd - 1);  // one row
  return r;
}

struct LnSizes {
  int64_t N, D;
  ccv_dtype dt, wdt;
  at::ScalarType wtype;
  int dev;
};

LnSizes ln_sizes(const Tensor& x, const Opt& weight, const Opt& bias) {
  if (x.dim() < 1) throw py::value_error("x must be [..., D]");
  LnSizes s;
  s.dt = dtype_of(x, "dtype");
  const Tensor& par = weight ? *weight : bias ? *bias : x;
  s.wdt = dtype_of(par, "weight dtype");
  s.wtype = par.scalar_type();
  s.D = x.size(x.dim() - 1);
  s.N = s.D > 0 ? x.numel() / s.D : 0;
  s.dev = cuda_index(x);
  check(s.dev, "weight", weight, {s.D}, s.wtype);
  check(s.dev, "bias", bias, {s.D}, s.wtype);
  return s;
}

std::tuple<int, Tensor> ln_fwd(const Tensor& x, const Opt& weight, const Opt& bias, double eps, Opt out_given,
                               std::optional<int64_t> stream) {
  const LnSizes s = ln_sizes(x, weight, bias);
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  const Stream on(s.dev, stream);
  const Tensor out = given(out_given, on, "out", x.sizes(), x.scalar_type());
  if (s.N == 0) return {CCV_OK, out};
  const Rows xr = rows(x), yr = rows(out);
  const int rc = ccv_ln_fwd(ptr(x), xr.strides, ptr(weight), stride0(weight), ptr(bias), stride0(bias), out_ptr(out),
                            yr.strides, s.N, s.D, static_cast<float>(eps), s.dt, s.wdt, on.raw());
  return {rc, out};
}

std::tuple<int, Tensor, Opt, Opt> ln_bwd(const Tensor& x, const Opt& weight, const Tensor& dout, const Opt& bias,
                                         double eps, Opt dx_, Opt dweight, Opt dbias, const Opt& workspace,
                                         std::optional<int64_t> stream) {
  const LnSizes s = ln_sizes(x, weight, bias);
  check(s.dev, "dout", dout, x.sizes(), x.scalar_type());
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  const Stream on(s.dev, stream);
  const Tensor dx = given(dx_, on, "dx", x.sizes(), x.scalar_type());
  if (dweight || weight) dweight = given(dweight, on, "dweight", {s.D}, s.wtype);
  if (dbias || bias) dbias = given(dbias, on, "dbias", {s.D}, s.wtype);
  Rows xr = {{0, 1}}, gr = xr, dr = xr;
  if (s.N > 0) xr = rows(x), gr = rows(dout), dr = rows(dx);
  uint64_t need = 0;
  int rc = CCV_OK;
  if (dweight || dbias) rc = ccv_ln_bwd_workspace_size(s.N, s.D, &need);
  if (rc == CCV_OK) {
    const Workspace w(workspace, need, on);
    rc = ccv_ln_bwd(ptr(x), xr.strides, ptr(weight), stride0(weight), ptr(dout), gr.strides, out_ptr(dx), dr.strides,
                    out_ptr(dweight), stride0(dweight), out_ptr(dbias), stride0(dbias), w.p, w.bytes, s.N, s.D,
                    static_cast<float>(eps), s.dt, s.wdt, on.raw());
  }
  return {rc, dx, dweight, dbias};
}

}  // namespace

PYBIND11_MODULE(_mixer_ext, m) {
  m.def("gdr_fwd", &gdr_fwd);
  m.def("gdr_step", &gdr_step);
  m.def("gdr_bwd", &gdr_bwd);
  m.def("ln_fwd", &ln_fwd);
  m.def("ln_bwd", &ln_bwd);
}

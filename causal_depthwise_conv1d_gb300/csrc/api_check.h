// Argument checks shared by the ABI front ends of the sequence-mixing operators
// (mix_api.cpp, rec_api.cpp): tensors given as pointer and strides, and
// workspaces.  Host only.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ccv.h"
#include "ccv_internal.h"

namespace {

using ccv::api_fail;

ccv_status fail_invalid(const char* name, const char* what) {
  return static_cast<ccv_status>(api_fail(CCV_ERR_INVALID_ARG, "%s %s", name, what));
}

#define CCV_FAIL(st, ...) return static_cast<ccv_status>(api_fail(st, __VA_ARGS__))
#define CCV_TRY(expr)                  \
  do {                                 \
    const ccv_status st_ = (expr);     \
    if (st_ != CCV_OK) return st_;     \
  } while (0)

bool valid_dtype(ccv_dtype d) { return d == CCV_F32 || d == CCV_F16 || d == CCV_BF16; }
int64_t dtype_size(ccv_dtype d) { return d == CCV_F32 ? 4 : 2; }

// The tensors of one call: each is checked when it is added (strides given,
// alignment, extent, an output's elements distinct), and then the outputs are
// checked against all others.
class Tensors {
 public:
  ccv_status add(const char* name, const void* p, const int64_t* strides, int nd, const int64_t* shape, int64_t esz,
                 bool out, bool required) {
    bool empty = false;
    for (int d = 0; d < nd; ++d) empty |= shape[d] == 0;
    if (empty) return CCV_OK;
    if (p == nullptr) {
      if (required) return fail_invalid(name, "is required");
      return CCV_OK;
    }
    if (strides == nullptr) return fail_invalid(name, "needs its strides");
    if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(esz) != 0)
      return fail_invalid(name, "must be aligned to its element size");
    __int128 lo = 0, hi = 0;
    for (int d = 0; d < nd; ++d) {
      const __int128 span = static_cast<__int128>(strides[d]) * (shape[d] - 1);
      if (span < 0) lo += span; else hi += span;
      if (out && shape[d] > 1 && strides[d] == 0) return fail_invalid(name, "has a zero stride on a dimension of size > 1");
    }
    const __int128 lim = static_cast<__int128>(INT64_MAX) / 16;
    if (lo < -lim || hi > lim) return fail_invalid(name, "extent overflows int64");
    T& t = t_[n_++];
    t.name = name;
    t.base = static_cast<const char*>(p);
    t.lo = t.base + static_cast<int64_t>(lo) * esz;
    t.hi = t.base + static_cast<int64_t>(hi) * esz + (esz - 1);
    t.esz = esz;
    t.out = out;
    t.nd = nd;
    for (int d = 0; d < nd; ++d) {
      t.strides[d] = strides[d];
      t.shape[d] = shape[d];
    }
    return CCV_OK;
  }

  // No output shares an element with another tensor.  Views whose dimensions
  // nest (a stride spans what lies within it), as slices and transposes of
  // buffers do, are told apart exactly; others pass unless one of the two fills
  // its whole range.
  ccv_status disjoint() const {
    for (int i = 0; i < n_; ++i) {
      if (!t_[i].out) continue;
      for (int j = 0; j < n_; ++j) {
        if (j == i) continue;
        const T &a = t_[i], &b = t_[j];
        if (a.lo > b.hi || b.lo > a.hi) continue;
        if (a.base == b.base || overlaps(a, b))
          return static_cast<ccv_status>(
              api_fail(CCV_ERR_INVALID_ARG, "%s must not alias or overlap %s", a.name, b.name));
      }
    }
    return CCV_OK;
  }

 private:
  struct T {
    const char* name;
    const char *base, *lo, *hi;
    int64_t esz;
    int nd;
    bool out;
    int64_t strides[4], shape[4];
  };

  static bool dense(const T& t) {  // every element between lo and hi belongs to it
    __int128 n = t.esz;
    for (int d = 0; d < t.nd; ++d) n *= t.shape[d];
    return n == static_cast<__int128>(t.hi - t.lo) + 1;
  }

  // A tensor as nested blocks of bytes: dimensions of size > 1, positive strides, the largest first.
  struct Box {
    const char* lo;
    int nd;
    __int128 stride[4], span[5];  // span[d]: bytes from the first to the last element of dimensions d..
    int64_t n[4];

    explicit Box(const T& t) : lo(t.lo), nd(0) {
      for (int d = 0; d < t.nd; ++d) {
        if (t.shape[d] == 1 || t.strides[d] == 0) continue;
        const __int128 s = static_cast<__int128>(t.strides[d]) * t.esz;
        int i = nd++;
        for (; i > 0 && stride[i - 1] < (s < 0 ? -s : s); --i) stride[i] = stride[i - 1], n[i] = n[i - 1];
        stride[i] = s < 0 ? -s : s;
        n[i] = t.shape[d];
      }
      span[nd] = t.esz;
      for (int d = nd - 1; d >= 0; --d) span[d] = stride[d] * (n[d] - 1) + span[d + 1];
    }
    bool nested(int d) const { return d < nd && span[d + 1] <= stride[d]; }
  };

  enum Answer { kNo, kYes, kUnknown };

  // Does a's block of dimensions i.. at 0 meet b's of dimensions j.. at `at`?
  // The block with the larger stride is cut at it: of a nested one at most two
  // pieces meet a block that is no longer than the stride, and where both have
  // the same stride their pieces meet at no more than two distances.
  static Answer meet(const Box& a, int i, const Box& b, int j, __int128 at, int* left) {
    if (at >= a.span[i] || at + b.span[j] <= 0) return kNo;
    if (i == a.nd && j == b.nd) return kYes;
    if (--*left < 0) return kUnknown;
    const __int128 sa = i < a.nd ? a.stride[i] : 0, sb = j < b.nd ? b.stride[j] : 0;
    if (sa < sb) return meet(b, j, a, i, -at, left);
    if (!a.nested(i)) return kUnknown;
    const bool both = sa == sb;
    if (both && !b.nested(j)) return kUnknown;
    // piece k of a lies at k sa; both: the distances k between pieces of b and of a
    const __int128 wa = a.span[i + 1], wb = both ? b.span[j + 1] : b.span[j];
    const __int128 first = both ? -(static_cast<__int128>(b.n[j]) - 1) : 0, last = a.n[i] - 1;
    // k sa < at + wb and at < k sa + wa
    __int128 k0 = floor_div(at - wa, sa) + 1, k1 = floor_div(at + wb - 1, sa);
    if (k0 < first) k0 = first;
    if (k1 > last) k1 = last;
    Answer r = kNo;
    for (__int128 k = k0; k <= k1; ++k) {
      const Answer x = meet(a, i + 1, b, both ? j + 1 : j, at - k * sa, left);
      if (x == kYes) return kYes;
      if (x == kUnknown) r = kUnknown;
      if (*left < 0) return kUnknown;
    }
    return r;
  }
  static __int128 floor_div(__int128 x, __int128 y) { return x / y - (x % y < 0 ? 1 : 0); }

  static bool overlaps(const T& a, const T& b) {
    int left = 256;
    const Answer r = meet(Box(a), 0, Box(b), 0, b.lo - a.lo, &left);
    return r == kYes || (r == kUnknown && (dense(a) || dense(b)));
  }

  T t_[20];
  int n_ = 0;
};

// A workspace of at least `need` bytes (none needed: whatever is given is left alone).
ccv_status add_workspace(Tensors& t, const void* workspace, uint64_t bytes, uint64_t need, int64_t align) {
  if (need == 0) return CCV_OK;
  if (workspace == nullptr || bytes < need)
    CCV_FAIL(CCV_ERR_INVALID_ARG, "workspace too small: need %llu bytes (got %llu)", (unsigned long long)need,
             (unsigned long long)(workspace ? bytes : 0));
  const int64_t shape[1] = {static_cast<int64_t>((need + align - 1) / align)}, one = 1;
  return t.add("workspace", workspace, &one, 1, shape, align, true, true);
}

void copy(int64_t* dst, const int64_t* src, int n) {
  for (int i = 0; i < n; ++i) dst[i] = src != nullptr ? src[i] : 0;
}

ccv_status launched(cudaError_t err, const char* kernel) {
  if (err != cudaSuccess) {
    ccv::api_kernel("none");
    CCV_FAIL(CCV_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(err));
  }
  ccv::api_kernel(kernel);
  return CCV_OK;
}

}  // namespace

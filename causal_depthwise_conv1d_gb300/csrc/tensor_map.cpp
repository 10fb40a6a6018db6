// Tensor maps of [outer, rows, channels] views for tiled copies.
#include "tensor_map.h"

#include <cuda_runtime.h>

namespace ccv {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

}  // namespace

// A tensor copy takes rows of unit stride on 16-byte boundaries, in strides that the copy's map can hold.  Rows
// that end inside 16 bytes are not taken: a store clips there, so it would write zeros up to the boundary.
bool tensor_map_eligible(const void* p, const int64_t* s, int64_t B, int64_t L, int64_t C, Dtype dt) {
  const int64_t e = dt == kF32 ? 4 : 2, lim = int64_t(1) << 39;
  return s[2] == 1 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && C < lim && C * e % 16 == 0 &&
         (L == 1 || (s[1] * e % 16 == 0 && s[1] >= C && s[1] * e < lim)) &&
         (B == 1 || (s[0] * e % 16 == 0 && s[0] > 0 && s[0] * e < lim)) && encoder() != nullptr;
}

bool tensor_map3(CUtensorMap* m, const void* p, const int64_t* s, int64_t B, int64_t L, int64_t C, const int64_t* box2,
              Dtype dt) {
  const int64_t e = dt == kF32 ? 4 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(C), static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(B)};
  const int64_t s1 = L > 1 ? s[1] * e : C * e;
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1), static_cast<cuuint64_t>(B > 1 ? s[0] * e : s1 * L)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box2[0]), static_cast<cuuint32_t>(box2[1]), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encoder()(m, dt == kF32 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3,
                   const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ccv

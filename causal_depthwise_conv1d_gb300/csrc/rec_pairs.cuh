// Pairs of the recurrence's and the group norm's kernels (packed FP32, see
// ccv_common.cuh).
#pragma once

#include "ccv_common.cuh"

namespace ccv {

__device__ __forceinline__ uint64_t twice(float c) { return pk(c, c); }

__device__ __forceinline__ float pair_sum(uint64_t v) {
  float a, b;
  upk(v, a, b);
  return a + b;
}

// Vectors as pairs.
template <int DT>
__device__ __forceinline__ void unpack_pairs(const uint4& v, uint64_t* f) {
  constexpr int V = Fmt<DT>::VEC;
  float x[V];
  unpack16<DT>(v, x);
#pragma unroll
  for (int j = 0; j < V / 2; ++j) f[j] = pk(x[2 * j], x[2 * j + 1]);
}

}  // namespace ccv

// Tensor maps of [B, L, C] views (strides in elements) for tiled copies of
// boxes of box2[1] rows x box2[0] channels.
#pragma once

#include <cuda.h>

#include "ccv_internal.h"

namespace ccv {

bool tensor_map_eligible(const void* p, const int64_t* s, int64_t B, int64_t L, int64_t C, Dtype dt);
bool tensor_map3(CUtensorMap* m, const void* p, const int64_t* s, int64_t B, int64_t L, int64_t C, const int64_t* box2,
                 Dtype dt);

}  // namespace ccv

// Device-side pieces shared by the streaming and the tile kernels of the
// experts' int8 products.
#pragma once

#include "device_common.h"

namespace fp8moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// One 16x16x64 int8 MFMA on 16 bytes of each lane; both operands take the
// same bytes of a K step, so the order of K within it is immaterial.
__device__ __forceinline__ i32x4 mfma16x16x64_i8(const v4i& a, const v4i& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

}  // namespace fp8moe

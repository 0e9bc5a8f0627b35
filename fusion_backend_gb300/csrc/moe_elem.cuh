// Element access by dtype code (moe_ffn_act_dtype) for the operators around
// the layer: their tensors come in fp32, bf16 and fp16, and the code is the
// same in every thread of a launch.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "moe_common.cuh"

namespace moe {

enum : int { kF32 = 0, kBf16 = 1, kF16 = 2 };

__host__ __device__ constexpr int elem_bytes(int dtype) { return dtype == kF32 ? 4 : 2; }

MOE_DEV float elem_load(const void* p, int dtype, size_t i) {
  if (dtype == kF32) return static_cast<const float*>(p)[i];
  if (dtype == kBf16) return bf16_to_float(static_cast<const uint16_t*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
// Rounded to nearest even where the type is narrower than fp32.
MOE_DEV void elem_store(void* p, int dtype, size_t i, float v) {
  if (dtype == kF32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == kBf16)
    static_cast<uint16_t*>(p)[i] = float_to_bf16_rne(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

}  // namespace moe

// Element access by dtype code (moe_ffn_act_dtype) for the operators around
// the layer: their tensors come in fp32, bf16 and fp16, and the code is the
// same in every thread of a launch.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
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

// Two floats as bf16 (fp16) in one word, each rounded to nearest even.
MOE_DEV uint32_t pack2(int dtype, float lo, float hi) {
  if (dtype == kF16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
MOE_DEV void unpack2(int dtype, uint32_t w, float& lo, float& hi) {
  if (dtype == kF16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  } else {
    lo = bf16_lo(w);
    hi = bf16_hi(w);
  }
}
// Eight consecutive elements, their address 16-byte aligned.
MOE_DEV void elem_load8(const void* p, int dtype, size_t i, float* v) {
  if (dtype == kF32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    unpack2(dtype, a.x, v[0], v[1]);
    unpack2(dtype, a.y, v[2], v[3]);
    unpack2(dtype, a.z, v[4], v[5]);
    unpack2(dtype, a.w, v[6], v[7]);
  }
}
MOE_DEV void elem_store8(void* p, int dtype, size_t i, const float* v) {
  if (dtype == kF32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(
        pack2(dtype, v[0], v[1]), pack2(dtype, v[2], v[3]), pack2(dtype, v[4], v[5]), pack2(dtype, v[6], v[7]));
  }
}

// Launch behind the previous kernel of the stream with programmatic stream
// serialisation.  The kernels launched this way wait (griddepcontrol.wait)
// before they touch what an earlier kernel may write, and let the next one
// start only behind that wait: so a kernel that starts early knows every
// kernel before its predecessor to be complete.
template <typename Kern, typename Params>
inline cudaError_t launch_behind(Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                 const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace moe

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
// One element, and four consecutive ones (their address aligned to the four), as
// they lie in memory: the loads of several tensors go out one behind the other,
// since nothing waits for a value between them, and are converted where they are
// used.  Four, not eight: neighbouring lanes then cover whole sectors in one
// access with fp32 too (16 bytes a lane), and a thread's columns are the same for
// tensors of every type.
MOE_DEV uint32_t raw_load(const void* p, int dtype, size_t i) {
  if (dtype == kF32) return static_cast<const uint32_t*>(p)[i];
  return static_cast<const uint16_t*>(p)[i];
}
MOE_DEV float raw_value(uint32_t w, int dtype) {
  if (dtype == kF32) return __uint_as_float(w);
  return dtype == kBf16 ? __uint_as_float(w << 16) : __half2float(__ushort_as_half((unsigned short)w));
}
MOE_DEV uint4 raw_load4(const void* p, int dtype, size_t i) {
  if (dtype == kF32) return *reinterpret_cast<const uint4*>(static_cast<const uint32_t*>(p) + i);
  const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  return make_uint4(v.x, v.y, 0u, 0u);
}
MOE_DEV void raw_values4(const uint4& w, int dtype, float* v) {
  if (dtype == kF32) {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
  } else {
    unpack2(dtype, w.x, v[0], v[1]);
    unpack2(dtype, w.y, v[2], v[3]);
  }
}
MOE_DEV void elem_store4(void* p, int dtype, size_t i, const float* v) {
  if (dtype == kF32)
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
        make_uint2(pack2(dtype, v[0], v[1]), pack2(dtype, v[2], v[3]));
}

// Launch behind the previous kernel of the stream with programmatic stream
// serialisation.  The kernels launched this way wait (griddepcontrol.wait)
// before they touch what an earlier kernel may write.  The routing, the order and
// the first product of the adapters let the next kernel start right behind that
// wait: so a kernel that starts early knows every kernel before its predecessor to
// be complete.  The norms and the adapters' second product do not: the caller may
// take what they write for weights, which the layer's row kernel reads ahead of
// its own wait.  (That costs a norm and the layer behind it 1.1 us of 25.5 at one
// token; calls of many rows got faster, without the next call's blocks waiting on
// their SMs: 24.5 -> 23.7 us for 4096 x 2048 fp32 rows, 55.5 -> 48.5 for adapters of
// 8192 tokens.)
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

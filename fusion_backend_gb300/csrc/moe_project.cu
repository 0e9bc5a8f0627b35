// Products of few tokens with 4-bit weights (moe_ffn_project):
//   y_tn = sum_g d_ng sum_{k in g} (c_nk - 8) x_tk + bias_n
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kWarps = 8;

// One warp a row of W and eight tokens.
__global__ void __launch_bounds__(32 * kWarps) k_project(const __grid_constant__ ProjectParams P) {
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * kWarps + (threadIdx.x >> 5), t0 = blockIdx.y * 8;
  pdl_wait();
  if (n >= P.N) return;
  const uint8_t* const row = P.w + (long long)n * P.w_stride;
  const __half* const scales = reinterpret_cast<const __half*>(row + P.K / 2);
  const int xd = P.f16 ? kF16 : kBf16;
  float acc[8] = {};
  for (int k = 2 * lane; k < P.K; k += 64) {
    const uint32_t b = row[k >> 1];
    const float d = __half2float(scales[k / P.group]);
    const float w0 = d * (float)((int)(b & 15u) - 8), w1 = d * (float)((int)(b >> 4) - 8);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t0 + t >= P.T) break;
      const size_t at = (size_t)(t0 + t) * P.x_stride + k;
      acc[t] = fmaf(w1, elem_load(P.x, xd, at + 1), fmaf(w0, elem_load(P.x, xd, at), acc[t]));
    }
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    float v = acc[t];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && t0 + t < P.T)
      elem_store(P.y, P.y_dtype, (size_t)(t0 + t) * P.y_stride + n, P.bias ? v + P.bias[n] : v);
  }
}

}  // namespace

cudaError_t launch_project(ProjectParams p, cudaStream_t stream) {
  return launch_behind(k_project, dim3((p.N + kWarps - 1) / kWarps, (p.T + 7) / 8), 32 * kWarps, 0, stream, p);
}

}  // namespace moe

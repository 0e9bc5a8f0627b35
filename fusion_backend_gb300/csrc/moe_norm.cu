// The norms after one block and before the next, with the block's gate and
// the residual scale between them (moe_ffn_norm_residual).
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

MOE_DEV float block_sum(float v, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) s += red[w];
  return s;
}

// r' of column c
MOE_DEV float residual(const NormParams& P, size_t t, int c, float inv_y) {
  const float r = P.alpha * elem_load(P.res, P.r_dtype, t * P.r_stride + c);
  if (!P.y) return r;
  float z = elem_load(P.y, P.y_dtype, t * P.y_stride + c);
  if (P.post_norm) z *= inv_y * (P.w_post ? P.w_offset + elem_load(P.w_post, P.wpost_dtype, c) : 1.f);
  if (P.gate) {
    const size_t gi = P.gate_layout == 0 ? c : P.gate_layout == 1 ? t * P.g_stride : t * P.g_stride + c;
    const float g = elem_load(P.gate, P.g_dtype, gi);
    z *= P.gate_sigmoid ? 1.f / (1.f + expf(-g)) : g;
  }
  return fmaf(P.beta, z, r);
}

__global__ void __launch_bounds__(kThreads) k_norm(const __grid_constant__ NormParams P) {
  __shared__ float red[kThreads / 32];
  extern __shared__ float row[];  // r' of the token
  const size_t t = blockIdx.x;
  float inv_y = 1.f;
  if (P.post_norm) {
    float q = 0.f;
    for (int c = threadIdx.x; c < P.H; c += kThreads) {
      const float v = elem_load(P.y, P.y_dtype, t * P.y_stride + c);
      q = fmaf(v, v, q);
    }
    inv_y = 1.f / sqrtf(block_sum(q, red) / (float)P.H + P.eps);
  }
  float q = 0.f;
  for (int c = threadIdx.x; c < P.H; c += kThreads) {
    const float r = residual(P, t, c, inv_y);
    row[c] = r;
    q = fmaf(r, r, q);
  }
  const float inv = 1.f / sqrtf(block_sum(q, red) / (float)P.H + P.eps);
  for (int c = threadIdx.x; c < P.H; c += kThreads) {
    const float r = row[c];
    if (P.res_out) elem_store(P.res_out, P.r_dtype, t * P.ro_stride + c, r);
    if (P.normed)
      elem_store(P.normed, P.n_dtype, t * P.n_stride + c,
                 r * inv * (P.w_pre ? P.w_offset + elem_load(P.w_pre, P.wpre_dtype, c) : 1.f));
  }
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
  const int smem = p.H * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k_norm, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  k_norm<<<p.T, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe

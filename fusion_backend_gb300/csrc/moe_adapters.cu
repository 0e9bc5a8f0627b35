// Low-rank adapters of many requests beside a shared projection
// (moe_ffn_add_adapters): v_t = A_a x_t, then out_t = y_t + scale_a B_a v_t.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

// Rank of adapter a; 0 where there is none of that index.
MOE_DEV int adapter_rank(const AdapterParams& P, int a) {
  if (a < 0 || a >= P.n) return 0;
  return P.ranks ? max(0, min(P.R, P.ranks[a])) : P.R;
}

// Block per token: warp w the rows w, w + 8, ... of A_a.
__global__ void __launch_bounds__(256) k_shrink(const __grid_constant__ AdapterParams P) {
  const size_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, a = P.ids[t], rank = adapter_rank(P, a);
  const int dt = P.f16 ? kF16 : kBf16;
  for (int r = threadIdx.x >> 5; r < rank; r += 8) {
    const uint16_t* row = P.A + ((size_t)a * P.R + r) * P.K;
    float s = 0.f;
    for (int k = lane; k < P.K; k += 32) s = fmaf(elem_load(row, dt, k), elem_load(P.x, dt, t * P.x_stride + k), s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) P.v[t * P.R + r] = s;
  }
}

// Thread per output column.
__global__ void __launch_bounds__(256) k_expand(const __grid_constant__ AdapterParams P) {
  const size_t t = blockIdx.x;
  const int a = P.ids[t], rank = adapter_rank(P, a);
  for (int n = threadIdx.x; n < P.N; n += 256) {
    float s = 0.f;
    if (rank > 0) {
      const uint16_t* row = P.B + ((size_t)a * P.N + n) * P.R;
      for (int r = 0; r < rank; ++r) s = fmaf(elem_load(row, P.f16 ? kF16 : kBf16, r), P.v[t * P.R + r], s);
      if (P.scales) s *= P.scales[a];
    }
    elem_store(P.out, P.y_dtype, t * P.out_stride + n, elem_load(P.y, P.y_dtype, t * P.y_stride + n) + s);
  }
}

}  // namespace

size_t adapters_workspace(int T, int K, int N, int R) {
  (void)K;
  (void)N;
  return ((size_t)T * R * 4 + 255) & ~size_t(255);
}

cudaError_t launch_adapters(const AdapterParams& p, cudaStream_t stream) {
  k_shrink<<<p.T, 256, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_expand<<<p.T, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe

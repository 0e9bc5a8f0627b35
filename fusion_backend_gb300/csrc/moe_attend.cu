// Attention over a paged cache (moe_ffn_attend):
//   out_t = sum_i exp(s_ti) v_i / sum_i exp(s_ti),  s_ti = cap(scale q_t k_i)
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// One warp a row and query head, its lanes over the elements of a head.
__global__ void __launch_bounds__(128) k_attend(const __grid_constant__ AttendParams P) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  pdl_wait();
  const int t_first = min(max(P.q_start[b], 0), P.T), t_end = min(max(P.q_start[b + 1], 0), P.T);
  const int n = t_end - t_first;
  const int len = (int)min((long long)max(P.lens[b], 0), (long long)P.max_pages * P.page_size);
  const int dt = P.f16 ? kF16 : kBf16;
  const int units = n * P.Hq;
  for (int u = blockIdx.x * 4 + (threadIdx.x >> 5); u < units; u += gridDim.x * 4) {
    const int j = u / P.Hq, h = u % P.Hq, t = t_first + j, hk = h / P.G;
    float q[8], o[8], m = -INFINITY, l = 0.f;
    for (int e = 0; e < 8; ++e) {
      const int d = lane + 32 * e;
      q[e] = d < P.D ? elem_load(P.q, dt, (size_t)t * P.q_stride + h * P.q_head + d) : 0.f;
      o[e] = 0.f;
    }
    for (int i = 0; i < len; ++i) {
      const int own = i - (len - n);
      if (own >= 0 && (P.mask ? own / 32 >= P.mask_words || !(P.mask[t * P.mask_stride + own / 32] >> own % 32 & 1)
                              : own > j))
        continue;
      const int page = P.table[b * P.table_stride + i / P.page_size], at = i % P.page_size;
      if ((uint32_t)page >= (uint32_t)P.pages) continue;
      const size_t ka = page * P.kc_page + at * P.kc_slot + hk * P.kc_head;
      const size_t va = page * P.vc_page + at * P.vc_slot + hk * P.vc_head;
      float s = 0.f;
      for (int e = 0; e < 8; ++e) {
        const int d = lane + 32 * e;
        if (d < P.D) s = fmaf(q[e], elem_load(P.k, dt, ka + d), s);
      }
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(kAll, s, x);
      s *= P.scale;
      if (P.softcap > 0.f) s = P.softcap * tanhf(s / P.softcap);
      const float m1 = fmaxf(m, s);
      if (m1 == -INFINITY && s == s) continue;
      const float old = m == -INFINITY ? 0.f : expf(m - m1), p = expf(s - m1);
      l = l * old + p;
      for (int e = 0; e < 8; ++e) {
        const int d = lane + 32 * e;
        if (d < P.D) o[e] = o[e] * old + p * elem_load(P.v, dt, va + d);
      }
      m = m1;
    }
    for (int e = 0; e < 8; ++e) {
      const int d = lane + 32 * e;
      if (d < P.D)
        elem_store(P.out, P.out_dtype, (size_t)t * P.o_stride + h * P.o_head + d, l == 0.f ? 0.f : o[e] / l);
    }
    if (P.lse && lane == 0) P.lse[(size_t)t * P.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
  }
}

}  // namespace

size_t attend_workspace(const AttendParams& p) { return 256; }

cudaError_t launch_attend(AttendParams p, cudaStream_t stream) {
  const int units = (p.T * p.Hq + 3) / 4;
  return launch_behind(k_attend, dim3(units < 1024 ? units : 1024, p.B), 128, 0, stream, p);
}

}  // namespace moe

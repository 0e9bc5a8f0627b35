// Keys and values of new tokens into a paged cache, keys and queries rotated by
// position on the way (moe_ffn_append_kv).
//
// The angle of pair i is position times inv_freq_i, reduced exactly: f / 2 pi as
// a 64-bit fixed-point fraction of a turn (its error 2^-64 turns), times the
// integer position modulo 2^64, so that whole turns fall away by themselves: at
// position 2^31 the error is 2^-33 turns.  (A product in fp32 has lost the angle
// at position 2^24, and fp64 is slow on this GPU.)
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

// f / 2 pi modulo 1 in units of 2^-64.  |f| < 256.
MOE_DEV uint64_t turn_fraction(float f) {
  // round(2^96 / 2 pi)
  const unsigned __int128 inv = ((unsigned __int128)0x28BE60DBull << 64) | 0x9391054A7F09D5F4ull;
  const uint32_t u = __float_as_uint(f), e = u >> 23 & 0xFFu;
  const uint32_t m = (u & 0x7FFFFFu) | (e ? 0x800000u : 0u);  // f = m 2^(max(e, 1) - 150)
  const int shift = 32 + 150 - (int)(e ? e : 1u);
  if (shift >= 128) return 0ull;
  const uint64_t v = (uint64_t)(m * inv >> shift);
  return u >> 31 ? 0ull - v : v;
}

// cos and sin of the phase (2^-64 turns).
MOE_DEV float2 cos_sin(uint64_t phase) {
  const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));  // within an eighth of a turn
  float s, c;
  sincospif((float)rest * 0x1p-63f, &s, &c);
  if (quarter & 1u) {
    const float t = c;
    c = -s;
    s = t;
  }
  return quarter & 2u ? make_float2(-c, -s) : make_float2(c, s);
}

// One block a token.
__global__ void __launch_bounds__(kThreads) k_append(const __grid_constant__ AppendParams P) {
  __shared__ float2 s_turn[kAppendMaxD / 2];
  const int tid = threadIdx.x, t = blockIdx.x;
  pdl_wait();
  const int slot = P.slot[t];
  if ((uint32_t)slot >= (uint32_t)P.slots) return;
  const int half = P.rot / 2;
  const long long pos = P.positions[t];
  for (int i = tid; i < half; i += kThreads) {
    const float f = P.inv_freq[i];
    float2 cs = cos_sin(turn_fraction(f) * (uint64_t)pos);
    const float scale = fabsf(f) < 256.f ? P.scale : __int_as_float(0x7FFFFFFF);
    s_turn[i] = make_float2(cs.x * scale, cs.y * scale);
  }
  __syncthreads();
  const int page = slot / P.page_size, at = slot % P.page_size;
  auto rotate_head = [&](const void* x, size_t from, void* out, int dtype, size_t to) {
    for (int i = tid; i < half; i += kThreads) {
      const int a = P.interleaved ? 2 * i : i, b = P.interleaved ? 2 * i + 1 : i + half;
      const float va = elem_load(x, P.x_dtype, from + a), vb = elem_load(x, P.x_dtype, from + b);
      const float2 cs = s_turn[i];
      elem_store(out, dtype, to + a, va * cs.x - vb * cs.y);
      elem_store(out, dtype, to + b, va * cs.y + vb * cs.x);
    }
    for (int d = P.rot + tid; d < P.D; d += kThreads) elem_store(out, dtype, to + d, elem_load(x, P.x_dtype, from + d));
  };
  for (int h = 0; h < P.Hq; ++h)
    rotate_head(P.q, t * P.q_stride + h * P.q_head, P.q_out, P.q_dtype, t * P.qo_stride + h * P.qo_head);
  for (int h = 0; h < P.Hkv; ++h) {
    rotate_head(P.k, t * P.k_stride + h * P.k_head, P.k_cache, P.c_dtype,
                page * P.kc_page + at * P.kc_slot + h * P.kc_head);
    for (int d = tid; d < P.D; d += kThreads)
      elem_store(P.v_cache, P.c_dtype, page * P.vc_page + at * P.vc_slot + h * P.vc_head + d,
                 elem_load(P.v, P.x_dtype, t * P.v_stride + h * P.v_head + d));
  }
}

}  // namespace

cudaError_t launch_append(AppendParams p, cudaStream_t stream) {
  return launch_behind(k_append, dim3(p.T), kThreads, 0, stream, p);
}

}  // namespace moe

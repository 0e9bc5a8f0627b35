// Keys and values of new tokens into a paged cache, keys and queries rotated by
// position on the way (moe_ffn_append_kv).
//
// The angle of pair i is position times inv_freq_i, reduced exactly: f / 2 pi as
// a 64-bit fixed-point fraction of a turn (its error 2^-64 turns), times the
// integer position modulo 2^64, so that whole turns fall away by themselves: at
// position 2^31 the error is 2^-33 turns.  (A product in fp32 has lost the angle
// at position 2^24, and fp64 is slow on this GPU.)
//
// A block takes some neighbouring tokens: their angles once, in shared memory, for
// all heads.  What the heads hold is on its way meanwhile: a thread asks for its
// items of all the block's tokens before the angles are formed.  An item is VEC
// elements, or VEC pairs whose halves lie apart; where it lies in a head is found
// once for all tokens.
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kMaxThreads = 512;

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

// VEC elements as they lie in memory, fp32 or 16-bit ones.
template <int VEC, bool F32>
struct Raw {
  uint4 w[VEC == 8 && F32 ? 2 : 1];
};
template <int VEC, bool F32>
MOE_DEV void raw_read(Raw<VEC, F32>& r, const void* p, long long i) {
  constexpr int kAny = F32 ? kF32 : kBf16;
  if constexpr (VEC == 8 && F32) {
    const uint4* const a = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    r.w[0] = a[0];
    r.w[1] = a[1];
  } else if constexpr (VEC == 8) {
    r.w[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  } else if constexpr (VEC == 4) {
    r.w[0] = raw_load4(p, kAny, i);
  } else {
    r.w[0].x = raw_load(p, kAny, i);
  }
}
template <int VEC, bool F32>
MOE_DEV void raw_floats(const Raw<VEC, F32>& r, int dtype, float (&v)[VEC]) {
  if constexpr (VEC == 8 && F32) {
    raw_values4(r.w[0], kF32, v);
    raw_values4(r.w[1], kF32, v + 4);
  } else if constexpr (VEC == 8) {
    unpack2(dtype, r.w[0].x, v[0], v[1]);
    unpack2(dtype, r.w[0].y, v[2], v[3]);
    unpack2(dtype, r.w[0].z, v[4], v[5]);
    unpack2(dtype, r.w[0].w, v[6], v[7]);
  } else if constexpr (VEC == 4) {
    raw_values4(r.w[0], F32 ? kF32 : dtype, v);
  } else {
    v[0] = raw_value(r.w[0].x, F32 ? kF32 : dtype);
  }
}
template <int VEC>
MOE_DEV void write_floats(void* p, int dtype, long long i, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    if (dtype == kF32) {
      elem_store4(p, kF32, i, v);
      elem_store4(p, kF32, i + 4, v + 4);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
          make_uint4(pack2(dtype, v[0], v[1]), pack2(dtype, v[2], v[3]), pack2(dtype, v[4], v[5]), pack2(dtype, v[6], v[7]));
    }
  } else if constexpr (VEC == 4) {
    elem_store4(p, dtype, i, v);
  } else {
    elem_store(p, dtype, i, v[0]);
  }
}

// VEC: elements an access.  TB: tokens a block.
template <int VEC, bool F32, int TB>
__global__ void __launch_bounds__(kMaxThreads) k_append(const __grid_constant__ AppendParams P) {
  __shared__ __align__(16) float2 s_turn[TB][kAppendMaxD / 2];
  const int tid = threadIdx.x, t0 = blockIdx.x * TB, tokens = TB == 1 ? 1 : min(TB, P.T - t0);
  pdl_wait();
  int slot[TB];
#pragma unroll
  for (int u = 0; u < TB; ++u) slot[u] = u < tokens ? P.slot[t0 + u] : -1;
  const int half = P.rot / 2;
  // items of a rotated head: pairs first, then what is not rotated
  const bool apart = VEC == 1 || !P.interleaved;  // an item's pairs have their halves apart
  const int pairs = apart ? half / VEC : P.rot / VEC, head_items = pairs + (P.D - P.rot) / VEC, v_items = P.D / VEC;
  const int turned = (P.Hq + P.Hkv) * head_items, items = turned + P.Hkv * v_items;

  bool first = true;
  for (int i = tid; first || i < items; i += blockDim.x) {
    // where the item lies: element d of a head, its second half `pair` elements
    // behind (0: none), its first pair's angle (-1: taken as it is)
    const void* from = nullptr;
    void* to = nullptr;
    long long at = 0, step = 0, head = 0;
    int d = 0, pair = 0, angle = -1, kind = 0;  // kind: 0 query, 1 key, 2 value
    const bool on = i < items;
    if (on) {
      int h;
      if (i < turned) {
        h = i / head_items;
        const int j = i - h * head_items;
        if (j < pairs) {
          angle = apart ? j * VEC : j * VEC / 2;
          pair = !apart ? 0 : P.interleaved ? 1 : half;
          d = VEC == 1 && P.interleaved ? 2 * j : j * VEC;
        } else {
          d = P.rot + (j - pairs) * VEC;
        }
      } else {
        h = (i - turned) / v_items;
        d = (i - turned - h * v_items) * VEC;
        h += P.Hq + P.Hkv;
      }
      if (h < P.Hq) {
        from = P.q, step = P.q_stride, at = h * P.q_head, to = P.q_out, head = h * P.qo_head + d;
      } else if (h < P.Hq + P.Hkv) {
        h -= P.Hq;
        kind = 1;
        from = P.k, step = P.k_stride, at = h * P.k_head, to = P.k_cache, head = h * P.kc_head + d;
      } else {
        h -= P.Hq + P.Hkv;
        kind = 2;
        from = P.v, step = P.v_stride, at = h * P.v_head, to = P.v_cache, head = h * P.vc_head + d;
      }
      at += t0 * step + d;
    }
    Raw<VEC, F32> a[TB], b[TB];
#pragma unroll
    for (int u = 0; u < TB; ++u) {
      if (!on || u >= tokens) continue;
      raw_read<VEC, F32>(a[u], from, at + u * step);
      if (pair) raw_read<VEC, F32>(b[u], from, at + u * step + pair);
    }
    if (first) {
      for (int x = tid; x < half * tokens; x += blockDim.x) {
        const int u = x / half, p = x - u * half;
        const float f = P.inv_freq[p];
        const float2 cs = cos_sin(turn_fraction(f) * (uint64_t)(long long)P.positions[t0 + u]);
        const float scale = fabsf(f) < 256.f ? P.scale : __int_as_float(0x7FFFFFFF);
        s_turn[u][p] = make_float2(cs.x * scale, cs.y * scale);
      }
      __syncthreads();
      first = false;
    }
#pragma unroll
    for (int u = 0; u < TB; ++u) {
      if (!on || (uint32_t)slot[u] >= (uint32_t)P.slots) continue;
      float x[VEC], y[VEC];
      raw_floats<VEC, F32>(a[u], P.x_dtype, x);
      const int dtype = kind == 0 ? P.q_dtype : P.c_dtype;
      long long out = head;
      if (kind == 0) {
        out += (t0 + u) * P.qo_stride;
      } else {
        const int page = slot[u] / P.page_size, in = slot[u] - page * P.page_size;
        out += page * (kind == 1 ? P.kc_page : P.vc_page) + in * (kind == 1 ? P.kc_slot : P.vc_slot);
      }
      if (pair) {
        raw_floats<VEC, F32>(b[u], P.x_dtype, y);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float2 cs = s_turn[u][angle + e];
          const float v = x[e];
          x[e] = v * cs.x - y[e] * cs.y;
          y[e] = v * cs.y + y[e] * cs.x;
        }
        write_floats<VEC>(to, dtype, out + pair, y);
      } else if (VEC > 1 && angle >= 0) {
#pragma unroll
        for (int e = 0; e + 1 < VEC; e += 2) {
          const float2 cs = s_turn[u][angle + e / 2];
          const float v = x[e];
          x[e] = v * cs.x - x[e + 1] * cs.y;
          x[e + 1] = v * cs.y + x[e + 1] * cs.x;
        }
      }
      write_floats<VEC>(to, dtype, out, x);
    }
  }
}

// Every tensor's rows allow accesses of vec elements.
bool fits(const AppendParams& p, int vec) {
  auto ok = [vec](const void* t, int dtype, long long a, long long b, long long c) {
    // an access is 16 bytes at most (fp32: two of them)
    const uintptr_t bytes = (uintptr_t)vec * elem_bytes(dtype);
    return !t || (reinterpret_cast<uintptr_t>(t) % (bytes < 16 ? bytes : 16) == 0 && a % vec == 0 && b % vec == 0 &&
                  c % vec == 0);
  };
  return p.D % vec == 0 && (p.interleaved ? p.rot : p.rot / 2) % vec == 0 && p.rot % vec == 0 &&
         ok(p.q, p.x_dtype, p.q_stride, p.q_head, 0) && ok(p.k, p.x_dtype, p.k_stride, p.k_head, 0) &&
         ok(p.v, p.x_dtype, p.v_stride, p.v_head, 0) && ok(p.q_out, p.q_dtype, p.qo_stride, p.qo_head, 0) &&
         ok(p.k_cache, p.c_dtype, p.kc_page, p.kc_slot, p.kc_head) &&
         ok(p.v_cache, p.c_dtype, p.vc_page, p.vc_slot, p.vc_head);
}

template <int VEC, bool F32>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
  const int each = VEC > 1 && !p.interleaved ? 2 * VEC : VEC;
  const int items = ((p.Hq + p.Hkv) * p.D + each - 1) / each + p.Hkv * p.D / VEC;
  const int threads = items >= kMaxThreads ? kMaxThreads : items < 64 ? 64 : (items + 31) / 32 * 32;
  constexpr int kMany = F32 ? 2 : 4;
  if (p.T < kMany * 2 * p.sms) return launch_behind(k_append<VEC, F32, 1>, dim3(p.T), threads, 0, stream, p);
  return launch_behind(k_append<VEC, F32, kMany>, dim3((p.T + kMany - 1) / kMany), threads, 0, stream, p);
}

template <int VEC>
cudaError_t launch_type(const AppendParams& p, cudaStream_t stream) {
  return p.x_dtype == kF32 ? launch<VEC, true>(p, stream) : launch<VEC, false>(p, stream);
}

}  // namespace

cudaError_t launch_append(AppendParams p, cudaStream_t stream) {
  return fits(p, 8) ? launch_type<8>(p, stream) : fits(p, 4) ? launch_type<4>(p, stream) : launch_type<1>(p, stream);
}

}  // namespace moe

// Keys and values of new tokens into a paged cache, keys and queries rotated by
// position on the way (moe_ffn_append_kv).
//
// The angle of pair i is position times inv_freq_i, reduced exactly: f / 2 pi as
// a 64-bit fixed-point fraction of a turn (its error 2^-64 turns), times the
// integer position modulo 2^64, so that whole turns fall away by themselves: at
// position 2^31 the error is 2^-33 turns.  (A product in fp32 has lost the angle
// at position 2^24, and fp64 is slow on this GPU.)
//
// A thread has one item of every token that its block takes: VEC elements of one
// head, or VEC pairs whose halves lie apart; where it lies is found once.  The
// angles of a token are formed once for all its heads, a thread an angle, into shared
// memory, for the next token while this one is turned, and what the next tokens'
// heads hold is on its way meanwhile, into a ring of the thread's own: one barrier a
// token.  4096 tokens of 32 + 2 x 4 heads of 128 in bf16: 18.6 us, 4.5 TB/s read and
// written; two tokens a barrier and three blocks an SM instead of two made no
// difference.  (A block a token, or two
// or four neighbouring ones with their items all at once, waited for one phase after
// the other: 41, 37 and 28 us for 4096 tokens of 40 heads of 128.)
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"
#include "moe_mma.cuh"

namespace moe {

namespace {

constexpr int kMaxThreads = 512;
constexpr int kThreadsPerSm = 1024;  // (64 registers a thread)
constexpr int kStages = 4;           // tokens on their way

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

// VEC elements in shared memory, fp32 (up to four) or 16-bit ones.
template <int VEC, bool F32>
MOE_DEV void read_floats(const void* p, int dtype, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 w = *static_cast<const uint4*>(p);
    unpack2(dtype, w.x, v[0], v[1]);
    unpack2(dtype, w.y, v[2], v[3]);
    unpack2(dtype, w.z, v[4], v[5]);
    unpack2(dtype, w.w, v[6], v[7]);
  } else if constexpr (VEC == 4) {
    raw_values4(raw_load4(p, F32 ? kF32 : kBf16, 0), F32 ? kF32 : dtype, v);
  } else {
    v[0] = raw_value(raw_load(p, F32 ? kF32 : kBf16, 0), F32 ? kF32 : dtype);
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

// Global -> shared; 2 bytes have no asynchronous copy.
template <int BYTES>
MOE_DEV void copy_item(void* dst, const void* src) {
  if constexpr (BYTES == 16)
    copy16(smem_u32(dst), src, 16u);
  else if constexpr (BYTES == 8)
    copy8(smem_u32(dst), src, 8u);
  else if constexpr (BYTES == 4)
    copy4(smem_u32(dst), src, 4u);
  else
    *static_cast<uint16_t*>(dst) = *static_cast<const uint16_t*>(src);
}

// VEC: elements an access.  APART: the halves of an item's pairs lie apart (for
// interleaved pairs VEC is 1 then).
template <int VEC, bool F32, bool APART>
__global__ void __launch_bounds__(kMaxThreads, kThreadsPerSm / kMaxThreads) k_append(const __grid_constant__ AppendParams P) {
  // angles of an item's pairs; those of neighbouring items next to each other, so that
  // neighbouring lanes read neighbouring words
  constexpr int GA = APART ? VEC : VEC / 2, GW = GA > 1 ? 2 : 1;
  __shared__ __align__(16) float2 s_turn[2][kAppendMaxD / 2 + 8];
  __shared__ long long s_place[2][2];  // the token's place in the caches of keys, of values (-1: padding)
  const int tid = threadIdx.x;
  const int half = P.rot / 2, groups = half / GA;
  // items of a rotated head: pairs first, then what is not rotated
  const int pairs = APART ? half / VEC : P.rot / VEC, head_items = pairs + (P.D - P.rot) / VEC, v_items = P.D / VEC;
  const int turned = (P.Hq + P.Hkv) * head_items, items = turned + P.Hkv * v_items;
  // where the thread's item lies: element d of a head, its second half `pair` elements
  // behind (0: none), its number among the rotated items (-1: taken as it is)
  const int i = blockIdx.y * blockDim.x + tid;
  const bool on = i < items;
  const void* from = nullptr;
  void* to = nullptr;
  long long at = 0, step = 0, head = 0;
  int pair = 0, turn = -1, kind = 0;  // kind: 0 query, 1 key, 2 value
  if (on) {
    int h, d;
    if (i < turned) {
      h = i / head_items;
      const int j = i - h * head_items;
      if (j < pairs) {
        turn = j;
        pair = !APART ? 0 : P.interleaved ? 1 : half;
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
    at += d;
  }
  const int dtype = kind == 0 ? P.q_dtype : P.c_dtype;
  pdl_wait();
  const float f = tid < half ? P.inv_freq[tid] : 0.f;
  const uint64_t fraction = turn_fraction(f);
  const float scale = fabsf(f) < 256.f ? P.scale : __int_as_float(0x7FFFFFFF);
  const int angle_at = (tid % GA / GW * groups + tid / GA) * GW + tid % GA % GW;
  // one token's angle and place
  auto prepare = [&](int buf, int position, int slot) {
    if (tid < half) {
      const float2 cs = cos_sin(fraction * (uint64_t)(long long)position);
      s_turn[buf][angle_at] = make_float2(cs.x * scale, cs.y * scale);
    }
    if (tid == blockDim.x - 1) {
      const bool in = (uint32_t)slot < (uint32_t)P.slots;
      const int page = in ? slot / P.page_size : 0, place = slot - page * P.page_size;
      s_place[buf][0] = in ? page * P.kc_page + place * P.kc_slot : -1;
      s_place[buf][1] = in ? page * P.vc_page + place * P.vc_slot : -1;
    }
  };
  // the item of token t, its two halves, into the thread's own places of a ring
  constexpr int kBytes = VEC * (F32 ? 4 : 2);
  extern __shared__ __align__(16) uint8_t ring[];
  uint8_t* const mine = ring + tid * kBytes;
  const int half_step = blockDim.x * kBytes, stage_step = 2 * half_step;
  auto ask = [&](int t, int stage) {
    if (on && t < P.T) {
      const uint8_t* const src = static_cast<const uint8_t*>(from) + (at + t * step) * (F32 ? 4 : 2);
      uint8_t* const dst = mine + stage * stage_step;
      copy_item<kBytes>(dst, src);
      if (APART && pair) copy_item<kBytes>(dst + half_step, src + pair * (F32 ? 4 : 2));
    }
    copy_commit();
  };
  int t = blockIdx.x, buf = 0, stage = 0;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) ask(t + s * gridDim.x, s);
  prepare(0, P.positions[t], P.slot[t]);
  for (; t < P.T; t += gridDim.x, buf ^= 1) {
    // the next tokens' elements are on their way while this one is turned
    const int t1 = t + gridDim.x;
    int position = 0, slot = -1;
    ask(t + (kStages - 1) * gridDim.x, (stage + kStages - 1) % kStages);
    if (t1 < P.T) {
      position = P.positions[t1];
      slot = P.slot[t1];
    }
    copy_wait<kStages - 1>();
    __syncthreads();
    const long long place = s_place[buf][kind == 2];
    if (on && place >= 0) {
      float x[VEC];
      read_floats<VEC, F32>(mine + stage * stage_step, P.x_dtype, x);
      const long long out = head + (kind == 0 ? t * P.qo_stride : place);
      float2 cs[GA];
      if (turn >= 0) {
#pragma unroll
        for (int e = 0; e < GA; e += GW) {
          const float2* const c = &s_turn[buf][(e / GW * groups + turn) * GW];
          if constexpr (GW == 2) {
            const float4 two = *reinterpret_cast<const float4*>(c);
            cs[e] = make_float2(two.x, two.y);
            cs[e + 1] = make_float2(two.z, two.w);
          } else {
            cs[e] = *c;
          }
        }
      }
      if (APART && pair) {
        float y[VEC];
        read_floats<VEC, F32>(mine + stage * stage_step + half_step, P.x_dtype, y);
#pragma unroll
        for (int e = 0; e < GA; ++e) {
          const float v = x[e];
          x[e] = v * cs[e].x - y[e] * cs[e].y;
          y[e] = v * cs[e].y + y[e] * cs[e].x;
        }
        write_floats<VEC>(to, dtype, out + pair, y);
      } else if (!APART && turn >= 0) {
#pragma unroll
        for (int e = 0; e < GA; ++e) {
          const float v = x[2 * e];
          x[2 * e] = v * cs[e].x - x[2 * e + 1] * cs[e].y;
          x[2 * e + 1] = v * cs[e].y + x[2 * e + 1] * cs[e].x;
        }
      }
      write_floats<VEC>(to, dtype, out, x);
    }
    if (t1 < P.T) prepare(buf ^ 1, position, slot);
    stage = (stage + 1) % kStages;
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

template <int VEC, bool F32, bool APART>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
  // an item a thread, an angle a thread
  const int half = p.rot / 2, pairs = APART ? half / VEC : p.rot / VEC;
  const int items = (p.Hq + p.Hkv) * (pairs + (p.D - p.rot) / VEC) + p.Hkv * (p.D / VEC);
  const int shares = (items + kMaxThreads - 1) / kMaxThreads, each = (items + shares - 1) / shares;
  const int threads = ((each > half ? each : half) + 31) / 32 * 32;
  const int most = (p.sms * (kThreadsPerSm / threads) + shares - 1) / shares;
  const int smem = kStages * 2 * threads * VEC * (F32 ? 4 : 2);
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void*>(k_append<VEC, F32, APART>), smem);
  if (e != cudaSuccess) return e;
  return launch_behind(k_append<VEC, F32, APART>, dim3(p.T < most ? p.T : most, shares), threads, smem, stream, p);
}

template <int VEC, bool F32>
cudaError_t launch_pairs(const AppendParams& p, cudaStream_t stream) {
  if constexpr (VEC > 1) {
    if (p.interleaved) return launch<VEC, F32, false>(p, stream);
  }
  return launch<VEC, F32, true>(p, stream);
}

}  // namespace

cudaError_t launch_append(AppendParams p, cudaStream_t stream) {
  // (four elements of fp32 are 16 bytes already)
  if (p.x_dtype == kF32) return fits(p, 4) ? launch_pairs<4, true>(p, stream) : launch_pairs<1, true>(p, stream);
  return fits(p, 8)   ? launch_pairs<8, false>(p, stream)
         : fits(p, 4) ? launch_pairs<4, false>(p, stream)
                      : launch_pairs<1, false>(p, stream);
}

}  // namespace moe

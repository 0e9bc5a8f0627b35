// Attention over a paged cache (moe_ffn_attend):
//   out_t = sum_i exp(s_ti) v_i / sum_i exp(s_ti),  s_ti = cap(scale q_t k_i)
// See moe_attend.cuh for the division of the work.
//
// k_attend, up to 16 rows a unit: bound by the stream of the cache.  Every warp
// takes 16 tokens of a chunk at a time by itself, with a ring of its own in shared
// memory that asynchronous copies fill ahead, across the ends of units too, and
// with a running maximum, sum and output of its own: the warps meet only at the end
// of a unit, and no barrier stands in the stream.  Scores and weighted values on
// mma.m16n8k16, the rows being the rows; a weight enters the second product as the
// sum of two or three numbers of the cache's type.
//
// Measured: a step of 64 KB an SM 1.4 us, 7 TB/s (D = 128, long sequences); the end
// of a unit costs 3 us of a block, in part behind what is on its way; 48 sequences of
// 500 to 12,000 tokens, 426 MB, 75 us; one of 2,000 tokens 8.9 us with the join.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_attend.cuh"
#include "moe_elem.cuh"
#include "moe_internal.h"
#include "moe_mma.cuh"
#include "moe_tma.cuh"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
__host__ __device__ constexpr int warps_for(int dp) { return dp <= 128 ? 8 : 4; }
// tokens a warp and step: with 16 of 64 columns the steps, not the stream, took the time
__host__ __device__ constexpr int tokens_for(int dp) { return dp <= 64 ? 32 : 16; }
__host__ __device__ constexpr int stages_for(int dp) { return dp == 192 ? 4 : 3; }
__host__ __device__ constexpr int slot_bytes(int dp) { return 2 * tokens_for(dp) * dp * 2; }
__host__ __device__ constexpr int attend_smem(int dp) {
  return warps_for(dp) * stages_for(dp) * (slot_bytes(dp) + 8) + 16 * dp * 2 + 1024;  // (slots at multiples of 1024)
}
// Byte of 16-byte piece c of row r in a tile of keys or values: 64 columns are
// 128 bytes of a row, swizzled; the next 64 lie behind all rows.
template <int TOK>
MOE_DEV uint32_t piece(int r, int c) {
  return (c >> 3) * (TOK * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// DP: elements of a head in shared memory (D rounded up); TERMS: numbers that
// stand for a weight.
// PAGED: pages hold multiples of 8 tokens: tensor copies of boxes of 8, 16 or (heads of
// up to 64) 32; else asynchronous copies by the lanes, each token from a page of its own
// (16 sequences of 4,000 tokens of 4 heads of 128: 28.5 us by boxes, 34 with pages of 1 or 5).
template <bool F16, int DP, int TERMS, bool PAGED>
__global__ void __launch_bounds__(32 * warps_for(DP), 1) k_attend(const __grid_constant__ AttendParams P) {
  constexpr int W = warps_for(DP), S = stages_for(DP), kSlot = slot_bytes(DP), kChunks = DP / 8, kTok = tokens_for(DP);
  constexpr int NT = DP / 8, KS = DP / 16, KT = kTok / 8;  // tiles of 8 columns, of 16, of 8 tokens
  constexpr uint32_t kFull = kTok == 32 ? 0xFFFFFFFFu : 0xFFFFu;
  constexpr bool kHoldQ = DP <= 128;  // queries stay in registers
  constexpr int kDt = F16 ? kF16 : kBf16;
  // The maximum of the sums stays while scores pass it by no more than 2^8, so that
  // the output is hardly ever scaled anew.  Weights in fp16 are held 2^7 up, sums and
  // outputs with them: they stay below 2^15, and two numbers resolve 2^-32 of that
  // maximum's weight (2^-25 without).
  constexpr float kLazy = 8.f, kUp = F16 ? 7.f : 0.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ float2 s_stat[W][16];
  __shared__ uint32_t s_valid[W][S];
  // of the unit under way: its first chunk here, whether a sum is not finite, whether values were taken out, and
  // what the values of tokens that all rows see hold (attend_odd), 8 columns a word
  __shared__ int s_chunk, s_sum_odd, s_own_odd;
  __shared__ uint32_t s_odd[kChunks];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  uint8_t* const ring = smem + warp * S * kSlot;
  const uint32_t ring_at = smem_u32(ring);
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + W * S * kSlot) + warp * S;
  uint8_t* const qs = smem + W * S * (kSlot + 8);
  const uint32_t q_at = smem_u32(qs);
  if (PAGED && lane == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) mbar_init(full + s, 1);
    mbar_fence_init();
    prefetch_tensormap(&P.tm_k);
    prefetch_tensormap(&P.tm_v);
  }
  pdl_wait();
  pdl_launch_dependents();
  fence_proxy_async_global();  // what the kernel before wrote, for the tensor copies
  AttendStep now = attend_begin<32 * W>(P);
  if (now.left <= 0) return;
  // columns that no copy writes
  if (!PAGED && P.D < DP)
    for (int i = tid * 16; i < W * S * kSlot; i += 32 * W * 16) *reinterpret_cast<uint4*>(smem + i) = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();

  const int pieces = P.D >> 3;
  // the page of the lane's box of the step's tokens (of its token lane % kTok)
  AttendStep ahead = now;
  int page_ahead = -1;
  const uint64_t once = policy_evict_first(), again = policy_evict_last();
  auto look = [&]() {  // the page of `ahead`
    page_ahead = -1;
    if (ahead.left <= 0) return;
    const int i = ahead.chunk * (W * kTok) + warp * kTok + (PAGED ? lane * P.box : lane & (kTok - 1));
    if (i < ahead.s.len && (!PAGED || lane * P.box < kTok)) page_ahead = P.table[ahead.b * P.table_stride + attend_page(P, i)];
  };
  bool dead = false;            // the warp's: a copy never came; nothing is asked for any more, results are NaN
  auto load = [&](int stage) {  // the tokens of `ahead`, then the next step's page
    if (ahead.left > 0 && !dead) {
      const int first = ahead.chunk * (W * kTok) + warp * kTok;
      const uint32_t k_dst = ring_at + stage * kSlot, v_dst = k_dst + kSlot / 2;
      const bool ok = (uint32_t)page_ahead < (uint32_t)P.pages;
      if constexpr (PAGED) {
        const uint32_t there = __ballot_sync(kAll, ok && lane * P.box < kTok);  // boxes whose page exists
        const int count = min(max(ahead.s.len - first, 0), kTok);
        uint32_t valid = count >= 32 ? ~0u : (1u << count) - 1u;
#pragma unroll
        for (int b = 0; b < kTok / 8; ++b)
          if (b * P.box < kTok && !(there >> b & 1u)) valid &= ~((~0u >> (32 - P.box)) << (b * P.box));
        if (lane == 0) {
          if (valid)
            mbar_arrive_expect_tx(full + stage, kSlot + P.lost);
          else
            mbar_arrive(full + stage);
          s_valid[warp][stage] = valid;
        }
        __syncwarp();
        if (valid && lane * P.box < kTok) {
          // (a page behind the cache: zeros)
          const int t = first + lane * P.box, slot = t - attend_page(P, t) * P.page_size, page = ok ? page_ahead : P.pages;
          const int x1 = P.slot_first ? slot : ahead.head, x2 = P.slot_first ? ahead.head : slot;
          // keys and values are read again where a sequence has further tiles of rows
          const uint64_t policy = ahead.s.tiles > 1 ? again : once;
          uint8_t* const dst = ring + stage * kSlot + lane * P.box * 128;
#pragma unroll
          for (int c = 0; c < DP / 64; ++c)
            tensor_load_4d(dst + c * kTok * 128, &P.tm_k, 64 * c, x1, x2, page, full + stage, policy);
#pragma unroll
          for (int c = 0; c < DP / 64; ++c)
            tensor_load_4d(dst + kSlot / 2 + c * kTok * 128, &P.tm_v, 64 * c, x1, x2, page, full + stage, policy);
        }
      } else {
        const int i = first + (lane & (kTok - 1));
        const bool in = ok && i < ahead.s.len;
        const uint32_t valid = __ballot_sync(kAll, in) & kFull;
        const int slot = in ? i - attend_page(P, i) * P.page_size : 0;
        const long long page = in ? page_ahead : 0;
        const long long k_off = page * P.kc_page + (long long)slot * P.kc_slot + ahead.head * P.kc_head;
        const long long v_off = page * P.vc_page + (long long)slot * P.vc_slot + ahead.head * P.vc_head;
        if (valid) {
#pragma unroll
          for (int j = 0; j < kTok * kChunks / 32; ++j) {
            const int x = j * 32 + lane, r = x / kChunks, c = x % kChunks;
            const long long ko = __shfl_sync(kAll, k_off, r), vo = __shfl_sync(kAll, v_off, r);
            const bool on = valid >> r & 1u;
            const uint32_t to = piece<kTok>(r, c);
            if (c < pieces) {
              copy16(k_dst + to, on ? P.k + ko + 8 * c : P.k, on ? 16u : 0u);
              copy16(v_dst + to, on ? P.v + vo + 8 * c : P.v, on ? 16u : 0u);
            }
          }
        }
        if (lane == 0) s_valid[warp][stage] = valid;
      }
      ahead.next(P);
      look();
    }
    if (!PAGED) copy_commit();
  };
  look();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) load(s);

  // (kept finite: 0 times infinity)
  auto kept = [](float v) { return fminf(fmaxf(v, -3.4e38f), 3.4e38f); };
  const float c1 = kept(P.softcap > 0.f ? P.scale / P.softcap : P.scale * kLog2e);
  const float c2 = kept(P.softcap * kLog2e);
  int stage = 0, stage_in = S - 1;
  uint32_t parity = 0;
  bool begin = true;
  uint32_t qf[kHoldQ ? KS : 1][4];
  float o[NT][4];
  float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f;  // rows g and g + 8 (log2 units)
  int row_t[2], row_j[2];                        // the rows' tokens (t: -1 behind the last)
  // queries of a unit, on their way while the warps meet at the end of the one before
  constexpr int kQueries = (16 * kChunks + 32 * W - 1) / (32 * W);
  uint4 queries[kQueries];
  auto ask = [&](const AttendStep& at) {
#pragma unroll
    for (int u = 0; u < kQueries; ++u) {
      const int i = tid + u * 32 * W, in = at.tile * 16 + i / kChunks, c = i % kChunks;
      queries[u] = make_uint4(0u, 0u, 0u, 0u);
      if (i < 16 * kChunks && in < at.s.n * P.G && 8 * c < P.D) {
        const int j = in / P.G;
        queries[u] = attend_query(P, at.s.t0 + j, at.head * P.G + in - j * P.G, c);
      }
    }
  };
  ask(now);
  while (now.left > 0) {
    if (begin) {
      begin = false;
      if (tid == 0) {
        s_chunk = now.chunk;
        s_sum_odd = s_own_odd = 0;
      }
      if (tid < kChunks) s_odd[tid] = 0u;
      const int rows = now.s.n * P.G, r0 = now.tile * 16;
#pragma unroll
      for (int u = 0; u < kQueries; ++u) {
        const int i = tid + u * 32 * W, r = i / kChunks, c = i % kChunks;
        if (i < 16 * kChunks) *reinterpret_cast<uint4*>(qs + r * (DP * 2) + ((c ^ (r & 7)) << 4)) = queries[u];
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = r0 + g + 8 * x;
        row_j[x] = r / P.G;
        row_t[x] = r < rows ? now.s.t0 + row_j[x] : -1;
      }
      __syncthreads();
      if constexpr (kHoldQ) {
        const int r = lane & 15;
#pragma unroll
        for (int s = 0; s < KS; ++s) ldmatrix4(qf[s], q_at + r * (DP * 2) + (((2 * s + (lane >> 4)) ^ (r & 7)) << 4));
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
    }
    if (!PAGED) copy_wait<S - 2>();
    __syncwarp();
    load(stage_in);
    stage_in = stage_in + 1 == S ? 0 : stage_in + 1;
    if (PAGED && !dead) dead = __any_sync(kAll, !mbar_wait(full + stage, parity));
    const uint32_t valid = s_valid[warp][stage];
    if (valid) {
      const uint32_t k_at = ring_at + stage * kSlot, v_at = k_at + kSlot / 2;
      float s[KT][4] = {};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t a[4];
        if constexpr (kHoldQ) {
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] = qf[ks][e];
        } else {
          const int qr = lane & 15;
          ldmatrix4(a, q_at + qr * (DP * 2) + (((2 * ks + (lane >> 4)) ^ (qr & 7)) << 4));
        }
#pragma unroll
        for (int n = 0; n < KT; n += 2) {
          const int r = 8 * n + (lane & 7) + ((lane >> 4) << 3);
          uint32_t b[4];
          ldmatrix4(b, k_at + piece<kTok>(r, 2 * ks + ((lane >> 3) & 1)));
          mma16<F16>(s[n], a[0], a[1], a[2], a[3], b[0], b[1]);
          mma16<F16>(s[n + 1], a[0], a[1], a[2], a[3], b[2], b[3]);
        }
      }
      if (P.softcap > 0.f) {
#pragma unroll
        for (int n = 0; n < KT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = c2 * attend_tanh(s[n][e] * c1);
      } else {
#pragma unroll
        for (int n = 0; n < KT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] *= c1;
      }
      const int first = now.chunk * (W * kTok) + warp * kTok, own = first - (now.s.len - now.s.n);
      if (valid != kFull || own + kTok > 0) {
#pragma unroll
        for (int n = 0; n < KT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 8 * n + 2 * q + (e & 1), x = e >> 1;
            const bool on = (valid >> i & 1u) && row_t[x] >= 0 && attend_sees(P, row_t[x], row_j[x], own + i);
            if (!on) s[n][e] = -INFINITY;
          }
        // values that a row does not see have no effect on it: a product with a weight of 0 has, where they are not
        // finite
        bool odd = false;
        const int from = attend_common(P, now.s) - first;  // of the tile's tokens, the first that some row may not see
        for (int i = lane; i < kTok * kChunks; i += 32) {
          if ((i >> 3 & (kTok - 1)) < from) continue;
          uint4* const at = reinterpret_cast<uint4*>(ring + stage * kSlot + kSlot / 2 + 16 * i);
          const uint4 v = *at;
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          bool any = false;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (odd16<F16>(w[x] & 0xFFFFu)) any = true, w[x] &= 0xFFFF0000u;
            if (odd16<F16>(w[x] >> 16)) any = true, w[x] &= 0xFFFFu;
          }
          if (any) *at = make_uint4(w[0], w[1], w[2], w[3]);
          odd |= any;
        }
        if (__any_sync(kAll, odd)) {
          if (lane == 0) s_own_odd = 1;
          fence_proxy_async();
          __syncwarp();
        }
      }
      // running maximum and sum
      float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
      for (int n = 0; n < KT; ++n) {
        a0 = fmaxf(a0, fmaxf(s[n][0], s[n][1]));
        a1 = fmaxf(a1, fmaxf(s[n][2], s[n][3]));
      }
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        a0 = fmaxf(a0, __shfl_xor_sync(kAll, a0, x));
        a1 = fmaxf(a1, __shfl_xor_sync(kAll, a1, x));
      }
      if (__any_sync(kAll, a0 > m0 + kLazy || a1 > m1 + kLazy)) {
        // (each row by its own: what the others hold must not change its roundings)
        const bool own0 = a0 > m0 + kLazy, own1 = a1 > m1 + kLazy;
        const float f0 = own0 ? exp2_fast(m0 - a0) : 1.f, f1 = own1 ? exp2_fast(m1 - a1) : 1.f;
        if (own0) m0 = a0;
        if (own1) m1 = a1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][0] *= f0;
          o[n][1] *= f0;
          o[n][2] *= f1;
          o[n][3] *= f1;
        }
      }
      const float b0 = attend_base(m0) - kUp, b1 = attend_base(m1) - kUp;
#pragma unroll
      for (int n = 0; n < KT; ++n) {
        s[n][0] = exp2_fast(s[n][0] - b0);
        s[n][1] = exp2_fast(s[n][1] - b0);
        s[n][2] = exp2_fast(s[n][2] - b1);
        s[n][3] = exp2_fast(s[n][3] - b1);
        l0 += s[n][0] + s[n][1];
        l1 += s[n][2] + s[n][3];
      }
      // a weight = the sum of TERMS numbers, each the rest rounded
      uint32_t p[TERMS][2 * KT];
#pragma unroll
      for (int x = 0; x < TERMS; ++x)
#pragma unroll
        for (int n = 0; n < KT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t w = pack2(kDt, s[n][2 * e], s[n][2 * e + 1]);
            p[x][2 * n + e] = w;
            if (x + 1 < TERMS) {
              float lo, hi;
              unpack2(kDt, w, lo, hi);
              s[n][2 * e] -= lo;
              s[n][2 * e + 1] -= hi;
            }
          }
#pragma unroll
      for (int n = 0; n < NT; n += 2)
#pragma unroll
        for (int k = 0; k < KT / 2; ++k) {
          uint32_t b[4];
          ldmatrix4_trans(b, v_at + piece<kTok>(16 * k + (lane & 15), n + (lane >> 4)));
#pragma unroll
          for (int x = TERMS - 1; x >= 0; --x) {
            mma16<F16>(o[n], p[x][4 * k], p[x][4 * k + 1], p[x][4 * k + 2], p[x][4 * k + 3], b[0], b[1]);
            mma16<F16>(o[n + 1], p[x][4 * k], p[x][4 * k + 1], p[x][4 * k + 2], p[x][4 * k + 3], b[2], b[3]);
          }
        }
    }
    const bool end = now.chunk + 1 == now.s.chunks;
    if (end || now.left == 1) {
      if (now.left > 1) {
        AttendStep next = now;
        next.next(P);
        if (next.left > 0) ask(next);
      }
      // the warps' sums meet: each leaves its own in the slot that it has just used
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        l0 += __shfl_xor_sync(kAll, l0, x);
        l1 += __shfl_xor_sync(kAll, l1, x);
      }
      __syncwarp();
      // (the eight rows that a store holds in different banks)
      float* const left = reinterpret_cast<float*>(ring + stage * kSlot);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int at = (8 * n + 2 * q) ^ (g << 3);
        *reinterpret_cast<float2*>(left + g * DP + at) = make_float2(o[n][0], o[n][1]);
        *reinterpret_cast<float2*>(left + (g + 8) * DP + at) = make_float2(o[n][2], o[n][3]);
      }
      if (q == 0) {
        const float none = __int_as_float(0x7FFFFFFF);
        s_stat[warp][g] = make_float2(m0 - kUp, dead ? none : l0);
        s_stat[warp][g + 8] = make_float2(m1 - kUp, dead ? none : l1);
      }
      float finite = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) finite = fmaf(o[n][e], 0.f, finite);
      if (finite != 0.f) s_sum_odd = 1;  // (NaN then)
      __syncthreads();
      const int chunk0 = s_chunk, first = chunk0 * (W * kTok), last = min((now.chunk + 1) * (W * kTok), now.s.len);
      const bool from_start = chunk0 == 0, whole = from_start && end, sum_odd = s_sum_odd, own_odd = s_own_odd;
      if (sum_odd) {
        const int c = tid % kChunks, step = 32 * W / kChunks, y = tid / kChunks;
        if (y < step && c < pieces) {
          const uint32_t bits = attend_odd<F16>(P, now.b, now.head, first + y, step, min(last, attend_common(P, now.s)), 8 * c);
          if (bits) atomicOr(s_odd + c, bits);
        }
        __syncthreads();
      }
      const int slot = 2 * blockIdx.x + (from_start ? 1 : 0);
      const int rows = now.s.n * P.G, r0 = now.tile * 16;
      for (int i = tid; i < 16 * (DP / 4); i += 32 * W) {
        const int r = i / (DP / 4), d = i % (DP / 4) * 4;
        if (r0 + r >= rows || d >= P.D) continue;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) m = fmaxf(m, s_stat[w][r].x);
        const float base = attend_base(m);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float2 st = s_stat[w][r];
          const float f = exp2_fast(st.x - base);
          const float4 a = *reinterpret_cast<const float4*>(smem + (w * S + stage) * kSlot +
                                                             (r * DP + (d ^ ((r & 7) << 3))) * 4);
          l = fmaf(st.y, f, l);
          v.x = fmaf(a.x, f, v.x);
          v.y = fmaf(a.y, f, v.y);
          v.z = fmaf(a.z, f, v.z);
          v.w = fmaf(a.w, f, v.w);
        }
        const int j = (r0 + r) / P.G, h = now.head * P.G + (r0 + r) - j * P.G;
        const long long t = now.s.t0 + j;
        if (sum_odd) {
          const uint32_t bits = s_odd[d >> 3] >> (2 * (d & 7));
          attend_put_odd(v.x, bits);
          attend_put_odd(v.y, bits >> 2);
          attend_put_odd(v.z, bits >> 4);
          attend_put_odd(v.w, bits >> 6);
        }
        if (own_odd) {
          const float4 x = attend_own<F16>(P, now.b, now.head, now.s.len - now.s.n, (int)t, j,
                                           max(first, attend_common(P, now.s)), last, d);
          attend_add_odd(v.x, x.x);
          attend_add_odd(v.y, x.y);
          attend_add_odd(v.z, x.z);
          attend_add_odd(v.w, x.w);
        }
        if (!whole) {
          *reinterpret_cast<float4*>(P.part + ((long long)slot * 16 + r) * P.width + d) = v;
          if (d == 0) P.stat[slot * 16 + r] = make_float2(m, l);
          continue;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float y[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
        if (l == 0.f) y[0] = y[1] = y[2] = y[3] = 0.f;
        const long long to = t * P.o_stride + h * P.o_head + d;
        if (P.o_vec) {
          elem_store4(P.out, P.out_dtype, to, y);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) elem_store(P.out, P.out_dtype, to + e, y[e]);
        }
        if (d == 0 && P.lse) P.lse[t * P.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      fence_proxy_async();
      __syncthreads();
      // (padded columns of the next use of the slot are 0 again)
      if (!PAGED && P.D < DP)
        for (int i = lane; i < kSlot / 16; i += 32) *reinterpret_cast<uint4*>(ring + stage * kSlot + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
      begin = true;
    }
    if (++stage == S) {
      stage = 0;
      parity ^= 1u;
    }
    now.next(P);
  }
  if (!PAGED) copy_wait<0>();
  if (dead)  // the block's shared memory is its own until copies that are under way have come
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

// Joins the parts of a unit.  Its rows are shared by the blocks (c, y) of the ranges
// c in which it goes on; with few parts a warp a row, else all warps a row.
constexpr int kJoinWarps = 8;
template <int NV>  // accesses of 128 columns a row
__global__ void __launch_bounds__(32 * kJoinWarps) k_attend_join(const __grid_constant__ AttendParams P) {
  __shared__ float4 s_o[kJoinWarps][32 * NV];
  __shared__ float s_l[kJoinWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  pdl_wait();
  const AttendFrom at = P.from[c];
  if (at.none) attend_none<kJoinWarps>(P);
  if (at.parts == 0) return;
  // the first part begins its unit, the others go on
  const int c0 = at.first, parts = at.parts, c1 = c0 + parts - 1;
  const int rows = min(at.n * P.G - at.tile * P.rows, P.rows);
  const bool together = parts > kJoinWarps;
  const int workers = (parts - 1) * gridDim.y, worker = (c - c0 - 1) * gridDim.y + blockIdx.y;
  for (int k = together ? 0 : warp;; k += together ? 1 : kJoinWarps) {
    const int r = worker + workers * k;
    if (r >= rows) break;
    auto slot_of = [&](int i) { return (long long)(i == c0 ? 2 * c0 + 1 : 2 * i) * P.rows + r; };
    float m = -INFINITY, l = 0.f;
    float4 acc[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (together) {
      for (int i = c0 + lane; i <= c1; i += 32) m = fmaxf(m, P.stat[slot_of(i)].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    }
    // eight parts at a time; few parts: all of them, their maximum is found on the way
    const int first = c0 + (together ? warp : 0), step = together ? kJoinWarps : 1;
#pragma unroll 1
    for (int i0 = first; i0 <= c1; i0 += 8 * step) {
      float2 st[8];
      float4 a[8][NV];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * step;
        if (i > c1) break;
        st[u] = P.stat[slot_of(i)];
        const float* const row = P.part + slot_of(i) * P.width;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          a[u][v] = 4 * lane + 128 * v < P.D ? *reinterpret_cast<const float4*>(row + 4 * lane + 128 * v)
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (!together) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (i0 + u <= c1) m = fmaxf(m, st[u].x);
      }
      const float base = attend_base(m);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (i0 + u * step > c1) break;
        const float f = exp2_fast(st[u].x - base);
        l = fmaf(st[u].y, f, l);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          acc[v].x = fmaf(a[u][v].x, f, acc[v].x);
          acc[v].y = fmaf(a[u][v].y, f, acc[v].y);
          acc[v].z = fmaf(a[u][v].z, f, acc[v].z);
          acc[v].w = fmaf(a[u][v].w, f, acc[v].w);
        }
      }
    }
    if (together) {
      if (lane == 0) s_l[warp] = l;
#pragma unroll
      for (int v = 0; v < NV; ++v) s_o[warp][lane + 32 * v] = acc[v];
      __syncthreads();
      if (warp == 0) {
#pragma unroll 1
        for (int w = 1; w < kJoinWarps; ++w) {
          l += s_l[w];
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const float4 o = s_o[w][lane + 32 * v];
            acc[v].x += o.x, acc[v].y += o.y, acc[v].z += o.z, acc[v].w += o.w;
          }
        }
      }
      __syncthreads();
      if (warp > 0) continue;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (4 * lane + 128 * v < P.D && !attend_finite(acc[v])) {
        float4 odd = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i = c0; i <= c1; ++i)
          attend_part_odd(odd, *reinterpret_cast<const float4*>(P.part + slot_of(i) * P.width + 4 * lane + 128 * v));
        attend_take_odd(acc[v], odd);
      }
    const int in = at.tile * P.rows + r, j = in / P.G, h = at.head * P.G + in - j * P.G;
    const long long t = at.t0 + j, out = t * P.o_stride + h * P.o_head;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = 4 * lane + 128 * v;
      if (d >= P.D) continue;
      float y[4] = {acc[v].x * inv, acc[v].y * inv, acc[v].z * inv, acc[v].w * inv};
      if (l == 0.f) y[0] = y[1] = y[2] = y[3] = 0.f;
      if (P.o_vec) {
        elem_store4(P.out, P.out_dtype, out + d, y);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) elem_store(P.out, P.out_dtype, out + d + e, y[e]);
      }
    }
    if (lane == 0 && P.lse) P.lse[t * P.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

constexpr int kMaxBlocks = kMaxGrid;  // the workspace does not depend on the device
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
int width_for(int D) { return (D + 63) / 64 * 64; }

// The cache as (column, head, slot, page) or (column, slot, head, page), by their
// strides, in boxes of 64 columns of p.box tokens of a head.
bool encode_cache(CUtensorMap* m, const AttendParams& p, const uint16_t* base, long long page, long long slot,
                  long long head) {
  const auto encode = tensor_map_encoder();
  if (!encode || 2 * page >= 1ll << 40 || 2 * slot >= 1ll << 40 || 2 * head >= 1ll << 40) return false;
  const cuuint64_t heads = p.Hkv, slots = p.page_size;
  const bool sf = p.slot_first;
  const cuuint64_t dims[4] = {(cuuint64_t)p.D, sf ? slots : heads, sf ? heads : slots, (cuuint64_t)p.pages};
  const cuuint64_t strides[3] = {(cuuint64_t)(2 * (sf ? slot : head)), (cuuint64_t)(2 * (sf ? head : slot)),
                                 (cuuint64_t)(2 * page)};
  const cuuint32_t box[4] = {64, sf ? (cuuint32_t)p.box : 1u, sf ? 1u : (cuuint32_t)p.box, 1}, ones[4] = {1, 1, 1, 1};
  return encode(m, p.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<uint16_t*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool F16, int DP, int TERMS, bool PAGED>
cudaError_t launch(const AttendParams& p, cudaStream_t stream) {
  static_assert(warps_for(DP) * tokens_for(DP) == (DP <= 64 ? 256 : DP <= 128 ? 128 : 64), "launch_attend's chunks");
  static_assert(attend_smem(DP) <= 229376, "shared memory");
  auto* const kern = k_attend<F16, DP, TERMS, PAGED>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), attend_smem(DP));
  if (e != cudaSuccess) return e;
  return launch_behind(kern, dim3(p.blocks), 32 * warps_for(DP), attend_smem(DP), stream, p);
}

template <bool F16, int TERMS, bool PAGED>
cudaError_t launch_width(const AttendParams& p, cudaStream_t stream) {
  return p.D <= 64    ? launch<F16, 64, TERMS, PAGED>(p, stream)
         : p.D <= 128 ? launch<F16, 128, TERMS, PAGED>(p, stream)
         : p.D <= 192 ? launch<F16, 192, TERMS, PAGED>(p, stream)
                      : launch<F16, 256, TERMS, PAGED>(p, stream);
}

cudaError_t launch_join(const AttendParams& p, cudaStream_t stream) {
  const dim3 grid(p.blocks, p.rows / 4);
  return p.width <= 128 ? launch_behind(k_attend_join<1>, grid, 32 * kJoinWarps, 0, stream, p)
                        : launch_behind(k_attend_join<2>, grid, 32 * kJoinWarps, 0, stream, p);
}

template <bool PAGED>
cudaError_t launch_terms(const AttendParams& p, cudaStream_t stream) {
  if (p.f16) return launch_width<true, 2, PAGED>(p, stream);
  return p.out_dtype == kF32 ? launch_width<false, 3, PAGED>(p, stream) : launch_width<false, 2, PAGED>(p, stream);
}

}  // namespace

// Units of up to 128 rows (k_attend_wide) where a sequence has more than 16 on average;
// its heads have to fit into tensor memory, boxes of 8 tokens into its pages (and three
// numbers a weight do not fit beside the scores).
static bool attend_wide(const AttendParams& p) {
  return p.D <= 128 && (long long)p.T * p.G > 16ll * p.B && p.page_size % 8 == 0 && (p.f16 || p.out_dtype != kF32);
}

static size_t attend_bytes(bool wide, int D) {
  const size_t rows = wide ? 128 : 16;
  return align256(kMaxBlocks * sizeof(AttendFrom)) + align256((size_t)2 * kMaxBlocks * rows * 8) +
         (size_t)2 * kMaxBlocks * rows * width_for(D) * 4;
}

size_t attend_needs(const AttendParams& p) { return attend_bytes(attend_wide(p), p.D); }

// As many rows may be one sequence's.
size_t attend_workspace(const AttendParams& p) { return attend_bytes(p.D <= 128 && (long long)p.T * p.G > 16, p.D); }

cudaError_t launch_attend(AttendParams p, cudaStream_t stream) {
  p.blocks = p.sms;
  // floor(i / d) for i < 2^31: i ceil(2^(32 + s) / d) >> (32 + s), 2^s >= d
  int s = 0;
  while ((1ll << s) < p.page_size) ++s;
  p.page_shift = 32 + s;
  p.page_mul = (unsigned long long)((((unsigned __int128)1 << (32 + s)) + p.page_size - 1) / p.page_size);
  p.q_vec = reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && p.q_stride % 8 == 0 && p.q_head % 8 == 0;
  p.o_vec = reinterpret_cast<uintptr_t>(p.out) % (4 * elem_bytes(p.out_dtype)) == 0 && p.o_stride % 4 == 0 && p.o_head % 4 == 0;
  p.slot_first = p.kc_slot < p.kc_head;
  const int dp = width_for(p.D);
  bool wide = attend_wide(p);
  for (p.box = wide ? 64 : tokens_for(dp); p.box > 8 && p.page_size % p.box;) p.box /= 2;
  const bool paged = p.page_size % 8 == 0 && p.pages > 0 && encode_cache(&p.tm_k, p, p.k, p.kc_page, p.kc_slot, p.kc_head) &&
                     encode_cache(&p.tm_v, p, p.v, p.vc_page, p.vc_slot, p.vc_head);
  wide = wide && paged;
  const int slots = wide ? 128 : 16;  // rows of a part
  // (whole tokens of a group's heads)
  p.rows = wide ? 128 / p.G * p.G : 16;
  p.chunk_log = wide || dp >= 128 ? 7 : 8;
  if (dp > 128) p.chunk_log = 6;
  // (in steps of 1.4 us: 2.9 us a unit; the wide kernel 7)
  p.extra = wide ? 4 : 2;
  p.width = dp;
  uint8_t* w = static_cast<uint8_t*>(p.ws);
  p.from = reinterpret_cast<AttendFrom*>(w);
  w += align256(kMaxBlocks * sizeof(AttendFrom));
  p.stat = reinterpret_cast<float2*>(w);
  w += align256((size_t)2 * kMaxBlocks * slots * 8);
  p.part = reinterpret_cast<float*>(w);
  if (wide) return launch_attend_wide(p, stream);
  const cudaError_t e = paged ? launch_terms<true>(p, stream) : launch_terms<false>(p, stream);
  return e != cudaSuccess ? e : launch_join(p, stream);
}

}  // namespace moe

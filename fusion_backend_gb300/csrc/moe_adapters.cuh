#pragma once

// Low-rank adapters of many requests beside a shared projection
// (moe_ffn_add_adapters): v_t = A_a x_t (k_shrink), then
// out_t = y_t + scale_a B_a v_t (k_expand).
//
// Both products run on tiles of up to 8 or 64 tokens that share an adapter, as
// mma.m16n8k16 with the adapter's rows as the 16 A rows and the tokens as the
// B columns, fp32 accumulators, operands straight from global memory: a lane
// takes 16 (A, x) or 8 (B) consecutive bytes of a row and the k index of the
// product is permuted alike on both sides, so every 32-byte sector read is used
// whole.  The work is bound by bytes (x, y, out once; an adapter once a tile),
// at R = 64 by 64 flops a byte: far below what the warp-level instructions
// give, so the tiles need no shared-memory staging or tensor memory.
//
// Tiles.  Up to kScanT tokens: block t looks through all adapter ids and owns a
// tile if its token is the first, 9th (65th), .. of its adapter.  More tokens:
// k_order ranks the tokens of each window of kWindow by adapter (counting, all
// against all, spread over 32 blocks; a bitonic sort of the window in one block
// took 12 us) and marks the places where a tile starts; block s of a window then
// finds the s-th mark.
//
// K is split over the warps of a block and, where there are few tiles, over
// blocks; the parts are summed in a fixed order.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kScanT = 64;            // two ids a lane
constexpr int kWindow = 1024;
constexpr int kRankChunk = 64;        // rows of A a block of k_shrink takes

// Elements between two tokens' v in shared memory: 32 modulo 64 bytes, no bank
// conflicts.
__host__ __device__ constexpr int expand_pitch(int R) { return (R + 15) / 16 % 2 ? (R + 15) / 16 * 16 : (R + 15) / 16 * 16 + 16; }

MOE_DEV int adapter_of(const AdapterParams& P, int t) {
  const int a = P.ids[t];
  return a < 0 || a >= P.n ? -1 : a;
}
MOE_DEV int adapter_rank(const AdapterParams& P, int a) {
  if (a < 0) return 0;
  return P.ranks ? max(0, min(P.R, P.ranks[a])) : P.R;
}

// d += A B (ZERO: d = A B), one m16n8k16.
template <bool F16, bool ZERO = false>
MOE_DEV void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  const float c0 = ZERO ? 0.f : d[0], c1 = ZERO ? 0.f : d[1], c2 = ZERO ? 0.f : d[2], c3 = ZERO ? 0.f : d[3];
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// The tile of this block (blockIdx.x): its adapter (-1: none), its tokens in
// `list`; false where the block has no tile.
template <int TILE>
MOE_DEV bool find_tile(const AdapterParams& P, int* list, int& a, int& n) {
  __shared__ int s_tile[2];  // adapter, tokens
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {
    n = 0;
    a = -1;
    if (P.T > kScanT) {
      // the s-th mark of window w: 32 marks a lane
      const int w = blockIdx.x / P.slots, s = blockIdx.x - w * P.slots;
      const int t0 = w * kWindow, len = min(kWindow, P.T - t0);
      uint32_t m[8];
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        const int at = 32 * lane + 4 * i;
        if (at < len) v = *reinterpret_cast<const uint4*>(P.marks + t0 + at);  // (marks are padded to 16 bytes)
        m[i] = v.x, m[i + 1] = v.y, m[i + 2] = v.z, m[i + 3] = v.w;
      }
      int c = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = 32 * lane + 4 * i + e;
          if (at >= len) m[i] &= ~(0xFFu << (8 * e));
          c += (m[i] >> (8 * e) & 0xFFu) != 0u;
        }
      int incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      int skip = s - (incl - c), place = 0;  // the lane's mark of that number
      if (skip >= 0 && skip < c) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int v = m[i] >> (8 * e) & 0xFFu;
            if (v && skip-- == 0) {
              n = v;
              place = t0 + 32 * lane + 4 * i + e;
            }
          }
      }
      const uint32_t who = __ballot_sync(0xffffffffu, n > 0);
      if (who) {
        place = __shfl_sync(0xffffffffu, place, __ffs(who) - 1);
        // the tokens from there on that have the same adapter
        const int left = min(TILE, t0 + len - place);
        int at[(TILE + 31) / 32], id[(TILE + 31) / 32];
#pragma unroll
        for (int i = 0; i < (TILE + 31) / 32; ++i) {
          const int j = place + min(lane + 32 * i, left - 1);
          at[i] = P.order[j];
          id[i] = P.adapter_at[j];
        }
        a = __shfl_sync(0xffffffffu, id[0], 0);
        n = 0;
#pragma unroll
        for (int i = 0; i < (TILE + 31) / 32; ++i) {
          const bool mine = lane + 32 * i < left && id[i] == a;
          if (mine) list[lane + 32 * i] = at[i];
          n += __popc(__ballot_sync(0xffffffffu, mine));
        }
      }
    } else {
      const int t = blockIdx.x;
      a = adapter_of(P, t);
      // tokens of the adapter, as bits
      const uint32_t lo = __ballot_sync(0xffffffffu, lane < P.T && adapter_of(P, min(lane, P.T - 1)) == a);
      const uint32_t hi = __ballot_sync(0xffffffffu, lane + 32 < P.T && adapter_of(P, min(lane + 32, P.T - 1)) == a);
      const unsigned long long all = (unsigned long long)hi << 32 | lo;
      if (__popcll(all & ((1ull << t) - 1)) % TILE == 0) {
        const unsigned long long rest = all & ~((1ull << t) - 1);
        n = min(TILE, __popcll(rest));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = lane + 32 * i, at = __popcll(rest & ((1ull << j) - 1));
          if ((rest >> j & 1ull) && at < TILE) list[at] = j;
        }
      }
    }
    if (lane == 0) {
      s_tile[0] = a;
      s_tile[1] = n;
    }
  }
  __syncthreads();
  a = s_tile[0];
  n = s_tile[1];
  return n > 0;
}

// Few tokens an adapter.  Blocks (tile of 8 tokens, part of K, 64 rows of A).
// The warps take 32-column blocks of K in turn, MT 16-row tiles of A; D
// fragments meet in shared memory, summed over the warps in order.
template <bool F16, int MT>
__global__ void __launch_bounds__(kThreads) k_shrink(const __grid_constant__ AdapterParams P) {
  constexpr int NT = 1, TILE = 8 * NT, ROWS = 16 * MT;
  extern __shared__ float red[];  // [kWarps][TILE][ROWS + 1]
  __shared__ int list[TILE];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  pdl_wait();
  pdl_launch_dependents();
  int a, n;
  if (!find_tile<TILE>(P, list, a, n)) return;
  const int r0 = blockIdx.z * kRankChunk, rank = adapter_rank(P, a) - r0;  // rows left
  if (rank <= 0) return;  // k_expand reads no v of such rows

  const uint16_t* xr[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int i = 8 * j + g;
    xr[j] = i < n ? P.x + (size_t)list[i] * P.x_stride : nullptr;
  }
  const uint16_t* ar = P.A + ((size_t)a * P.R + r0) * P.K;
  float d[MT][NT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) d[i][j][0] = d[i][j][1] = d[i][j][2] = d[i][j][3] = 0.f;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const int step = 32 * kWarps * P.splits;
#pragma unroll 2
  for (int k = 32 * (blockIdx.y * kWarps + warp) + 8 * q; k - 8 * q < P.K; k += step) {
    const bool in = k < P.K;
    uint4 xv[NT], av[MT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) xv[j] = in && xr[j] ? *reinterpret_cast<const uint4*>(xr[j] + k) : zero;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * i + 8 * h + g;
        av[i][h] = in && r < rank ? *reinterpret_cast<const uint4*>(ar + (size_t)r * P.K + k) : zero;
      }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (8 * j >= n) continue;
        mma16816<F16>(d[i][j], av[i][0].x, av[i][1].x, av[i][0].y, av[i][1].y, xv[j].x, xv[j].y);
        mma16816<F16>(d[i][j], av[i][0].z, av[i][1].z, av[i][0].w, av[i][1].w, xv[j].z, xv[j].w);
      }
  }
  float* mine = red + (size_t)warp * TILE * (ROWS + 1);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (8 * j >= n) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) mine[(8 * j + 2 * q + (c & 1)) * (ROWS + 1) + 16 * i + 8 * (c >> 1) + g] = d[i][j][c];
    }
  __syncthreads();
  const int rows = min(ROWS, P.R - r0);  // rows past the rank are zeros
  float* v = P.v + (size_t)blockIdx.y * P.T * P.R + r0;
  for (int i = tid; i < n * ROWS; i += kThreads) {
    const int tok = i / ROWS, r = i - tok * ROWS;
    if (r >= rows) continue;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += red[(size_t)w * TILE * (ROWS + 1) + tok * (ROWS + 1) + r];
    v[(size_t)list[tok] * P.R + r] = s;
  }
}

// Many tokens an adapter.  Blocks (tile of 64 tokens, two parts of K, 64 rows of
// A): warp w has tokens 16 (w mod 4) .. of the tile and the part 2 blockIdx.y +
// w / 4 of K, so nothing is summed between warps; the adapter's rows come from L1
// for all but the first warp that asks.  What bounds it is the L1 cycles of those
// reads (eight rows an access), so a warp takes two 8-token tiles against every
// row it reads.  UN 32-column blocks of x are asked for at once.
template <bool F16, int MT>
__global__ void __launch_bounds__(kThreads, 2) k_shrink_wide(const __grid_constant__ AdapterParams P) {
  constexpr int UN = 4;
  __shared__ int list[64];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  pdl_wait();
  pdl_launch_dependents();
  int a, n;
  if (!find_tile<64>(P, list, a, n)) return;
  const int r0 = blockIdx.z * kRankChunk, rank = adapter_rank(P, a) - r0, t0 = 16 * (warp & 3);
  if (rank <= 0 || t0 >= n) return;
  const int split = 2 * blockIdx.y + (warp >> 2), part = (P.K + 32 * P.splits - 1) / (32 * P.splits) * 32;
  const int k_end = min(P.K, part * (split + 1));
  // (a token past the tile's last is its last: its product is not stored)
  const uint16_t* const x0 = P.x + (size_t)list[min(t0 + g, n - 1)] * P.x_stride;
  const uint16_t* const x1 = P.x + (size_t)list[min(t0 + 8 + g, n - 1)] * P.x_stride;
  const uint16_t* const ar = P.A + ((size_t)a * P.R + r0 + g) * P.K;
  float d[MT][2][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 2; ++j) d[m][j][0] = d[m][j][1] = d[m][j][2] = d[m][j][3] = 0.f;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 xv[UN][2];
  auto ask = [&](int k, uint4 (&v)[2]) {
    v[0] = k < k_end ? *reinterpret_cast<const uint4*>(x0 + k) : zero;
    v[1] = k < k_end ? *reinterpret_cast<const uint4*>(x1 + k) : zero;
  };
  const int k_first = part * split + 8 * q;
#pragma unroll
  for (int u = 0; u < UN; ++u) ask(k_first + 32 * u, xv[u]);
  for (int k0 = k_first; k0 - 8 * q < k_end; k0 += 32 * UN) {
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int k = k0 + 32 * u;
      const uint4 xa = xv[u][0], xb = xv[u][1];
      ask(k + 32 * UN, xv[u]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint4 av[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          av[h] = k < k_end && 16 * m + 8 * h + g < rank
                      ? *reinterpret_cast<const uint4*>(ar + (size_t)(16 * m + 8 * h) * P.K + k)
                      : zero;
        mma16816<F16>(d[m][0], av[0].x, av[1].x, av[0].y, av[1].y, xa.x, xa.y);
        mma16816<F16>(d[m][1], av[0].x, av[1].x, av[0].y, av[1].y, xb.x, xb.y);
        mma16816<F16>(d[m][0], av[0].z, av[1].z, av[0].w, av[1].w, xa.z, xa.w);
        mma16816<F16>(d[m][1], av[0].z, av[1].z, av[0].w, av[1].w, xb.z, xb.w);
      }
    }
  }
  // D: row 16 m + g (+ 8), token 2q (+ 1) of the eight
  float* const v = P.v + (size_t)split * P.T * P.R + r0;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int tok = t0 + 8 * j + 2 * q + c;
      if (tok >= n) continue;
      float* const row = v + (size_t)list[tok] * P.R;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * m + 8 * h + g;
          if (r0 + r < P.R) row[r] = d[m][j][2 * h + c];
        }
    }
}

// Numbers of the operands' type that v enters the second product as: what its
// 8-bit (bf16) or 11-bit (fp16) significands add up to is 16 and more bits of v
// for a 16-bit result, 22 and more for an fp32 one.
template <bool F16, int YK>
constexpr int kTerms = F16 || YK == 1 ? 2 : 3;
constexpr float kLow = 0x1p11f;  // fp16: the second number's factor

// v of a tile as an operand of the second product, TERMS numbers an element, the
// largest first.  fp16: of v scaled by a power of two to a largest element of 2^14
// and more, since v may pass fp16's range, and the second number times 2^11: both
// are then normal fp16 numbers down to 2^-28 of the largest element (unscaled, the
// second one lost bits from 2^-3 of it on).  s_scale: what takes the token's
// product back, times the adapter's scale.  256 / TILE threads a token; ends with a
// block barrier.
template <bool F16, int TILE, int TERMS>
MOE_DEV void stage_v(const AdapterParams& P, const int* list, int a, int n, int rank, int pitch, uint32_t* vs,
                     float* s_scale) {
  const int tid = threadIdx.x;
  constexpr int TPT = kThreads / TILE;
  const int tok = tid / TPT, part = tid % TPT, padded = (rank + 15) & ~15;
  const float* const v = P.v + (tok < n ? (size_t)list[tok] * P.R : 0);
  const size_t part_step = (size_t)P.T * P.R;  // from a part of K to the next
  auto v_of = [&](int r) {
    float sum = 0.f;
    if (tok < n && r < rank) {
      const float* p = v + r;
#pragma unroll 2
      for (int k = 0; k < P.splits; ++k, p += part_step) sum += __ldcg(p);
    }
    return sum;
  };
  float up = 1.f, down = 1.f;
  if (F16) {
    float top = 0.f;
    for (int r = part; r < rank; r += TPT) {
      const float x = fabsf(v_of(r));
      if (x < INFINITY) top = fmaxf(top, x);  // what is finite stays so beside what is not
    }
#pragma unroll
    for (int o = TPT >> 1; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // 2^(e - 127) <= top < 2^(e - 126), the factors kept within the normal numbers
    const uint32_t e = max(__float_as_uint(top) >> 23, 15u);
    if (top > 0.f) {
      up = __uint_as_float((e - 14u) << 23);
      down = __uint_as_float((268u - e) << 23);
    }
  }
  uint16_t* const out = reinterpret_cast<uint16_t*>(vs) + tok * pitch;
#pragma unroll 4
  for (int r = part; r < padded; r += TPT) {
    float x = v_of(r) * down;
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
      const uint32_t h = pack2(F16 ? kF16 : kBf16, x, 0.f);
      float xh, none;
      unpack2(F16 ? kF16 : kBf16, h, xh, none);
      out[i * TILE * pitch + r] = static_cast<uint16_t>(h);
      x = fabsf(xh) < INFINITY ? x - xh : 0.f;  // exact
      if (F16) x *= kLow;
    }
  }
  if (part == 0) s_scale[tok] = up * (P.scales ? P.scales[a] : 1.f);
  __syncthreads();
}

// Blocks (tile of 8 tokens, columns, 256 at a time); warp w has 32 w .. of them as
// two 16-row tiles of B, whose rows are dealt so that a lane ends with four
// neighbouring columns n0 + 4g .. + 3 of tokens 2q and 2q + 1.  The ids, the order,
// B and y are read ahead of the wait on the first product, which writes none of
// them.  YK: y and out are fp32 (0) or 16-bit (1) in rows that allow accesses of
// four elements, or anything (2).
template <bool F16, int ST, int YK>
__global__ void __launch_bounds__(kThreads, ST <= 4 ? 2 : 1) k_expand(const __grid_constant__ AdapterParams P) {
  constexpr int TILE = 8, YB = YK == 0 ? 4 : 2, TERMS = kTerms<F16, YK>;
  extern __shared__ __align__(16) uint32_t vs[];  // [TERMS][TILE][pitch / 2]; pitch in elements
  __shared__ int list[TILE];
  __shared__ __align__(8) float s_scale[TILE];
  __shared__ __align__(16) longlong2 s_row[TILE];  // bytes to the token's row of y and of out
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  int a, n;
  if (!find_tile<TILE>(P, list, a, n)) {
    pdl_wait();
    return;
  }
  // (rows past the tile's last are its last: their loads need no test)
  if (tid < TILE) {
    const long long t = list[min(tid, n - 1)];
    s_row[tid] = make_longlong2(t * P.y_stride * YB, t * P.out_stride * YB);
    s_scale[tid] = 0.f;
  }
  const int rank = adapter_rank(P, a), pitch = expand_pitch(P.R);
  const int c_first = P.cols * blockIdx.y, c_end = min(P.N, c_first + P.cols);
  __syncthreads();
  const uint16_t* const v0 = reinterpret_cast<const uint16_t*>(vs) + g * pitch + 4 * q;
  bool staged = false;
  for (int b0 = c_first; b0 < c_end; b0 += kThreads) {
    const int n0 = b0 + 32 * warp + 4 * g;
    const bool in = n0 < c_end;
    // B: the lane's four columns, four k a step
    uint2 bv[ST][4];
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      uint2(&b)[4] = bv[s];
      const int r = 16 * s + 4 * q;
#pragma unroll
      for (int c = 0; c < 4; ++c) b[c] = make_uint2(0u, 0u);
      if (r >= rank) continue;
      const uint16_t* row = P.B + ((size_t)a * P.N + n0) * P.R + r;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (n0 + c < P.N) {
          if (P.R % 4 == 0) {
            b[c] = *reinterpret_cast<const uint2*>(row);
          } else {
            b[c].x = row[0] | (r + 1 < rank ? (uint32_t)row[1] << 16 : 0u);
            b[c].y = (r + 2 < rank ? row[2] : 0u) | (r + 3 < rank ? (uint32_t)row[3] << 16 : 0u);
          }
        }
        row += P.R;
      }
      if (r + 4 > rank) {  // what lies past the rank does not count
        const uint32_t mx = r + 1 < rank ? ~0u : 0xFFFFu, my = r + 3 < rank ? ~0u : r + 2 < rank ? 0xFFFFu : 0u;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          b[c].x &= mx;
          b[c].y &= my;
        }
      }
    }
    // y of tokens 2q (+ 1), as it lies in memory (YK < 2)
    uint4 yv[2];
    if (YK < 2 && in) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* const at = static_cast<const uint8_t*>(P.y) + (size_t)n0 * YB + s_row[2 * q + h].x;
        if (YK == 0) {
          yv[h] = *reinterpret_cast<const uint4*>(at);
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(at);
          yv[h].x = w.x, yv[h].y = w.y;
        }
      }
    }
    if (!staged) {
      pdl_wait();
      if (rank == 0 && P.out == P.y) return;
      if (rank > 0) stage_v<F16, TILE, TERMS>(P, list, a, n, rank, pitch, vs, s_scale);
      staged = true;
    }
    // (v of tokens past the last is 0, their y is the last's; they are not stored)
    float d[2][4];
    if (rank > 0) {
      // the smallest term first; fp16: its whole product, then the other's
#pragma unroll
      for (int pass = F16 ? TERMS - 1 : 0; pass >= 0; --pass) {
        if (F16 && pass < TERMS - 1) {
#pragma unroll
          for (int c = 0; c < 4; ++c) d[0][c] *= 1.f / kLow, d[1][c] *= 1.f / kLow;
        }
#pragma unroll
        for (int s = 0; s < ST; ++s) {
          if (16 * s >= rank) break;
#pragma unroll
          for (int i = F16 ? pass : TERMS - 1; i >= pass; --i) {
            const uint2 t = *reinterpret_cast<const uint2*>(v0 + i * TILE * pitch + 16 * s);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint2 b0 = bv[s][2 * m], b1 = bv[s][2 * m + 1];
              if (s == 0 && i == TERMS - 1)
                mma16816<F16, true>(d[m], b0.x, b1.x, b0.y, b1.y, t.x, t.y);
              else
                mma16816<F16>(d[m], b0.x, b1.x, b0.y, b1.y, t.x, t.y);
            }
          }
        }
      }
    } else {  // (the scale is 0 then: -0 leaves y as it is, a zero's sign too)
#pragma unroll
      for (int c = 0; c < 4; ++c) d[0][c] = d[1][c] = -0.f;
    }
    const float2 scale = *reinterpret_cast<const float2*>(s_scale + 2 * q);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 2 * q + h;
      if (i >= n || !in) continue;
      float z[4];
      if (YK < 2) {
        raw_values4(yv[h], YK == 0 ? kF32 : P.y_dtype, z);
      } else {
        const size_t at = (size_t)list[i] * P.y_stride + n0;
#pragma unroll
        for (int c = 0; c < 4; ++c) z[c] = n0 + c < c_end ? elem_load(P.y, P.y_dtype, at + c) : 0.f;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) z[c] = fmaf(h ? scale.y : scale.x, d[c >> 1][2 * (c & 1) + h], z[c]);
      uint8_t* const at = static_cast<uint8_t*>(P.out) + (size_t)n0 * YB + s_row[i].y;
      if (YK == 0) {
        *reinterpret_cast<float4*>(at) = make_float4(z[0], z[1], z[2], z[3]);
      } else if (YK == 1) {
        *reinterpret_cast<uint2*>(at) = make_uint2(pack2(P.y_dtype, z[0], z[1]), pack2(P.y_dtype, z[2], z[3]));
      } else {
        const size_t to = (size_t)list[i] * P.out_stride + n0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (n0 + c < c_end) elem_store(P.out, P.y_dtype, to + c, z[c]);
      }
    }
  }
}

// The same for tiles of 64 tokens and 256 HV columns at a time, with the tokens as
// the rows of the products: a lane ends with four neighbouring columns n0 + 16 p ..
// + 3 of tokens g and g + 8, its three neighbours with the twelve behind them, so
// that a quarter of a warp has 64 bytes each of two rows of y in one access.  (With
// the columns as the rows it has 32 bytes each of four, and the L1's cycles, four
// times an access's bytes, bound the kernel: 5 us more for the whole call at 8192
// tokens, 2048 x 2048, rank 32, fp32 y.)  B stays in registers while the warp
// goes through the tile's tokens, G times sixteen at a time, whose y is asked for a
// round ahead; nothing is waited for between warps.  HV = 2 reads a token's v once
// for 64 columns (48.4 us for the call, with HV = 1 50.2).  What is left are the
// loads that are waited for at 16 warps an SM: the call runs at 3.5 TB/s; the first
// form, a thread an output element, took 1171 us.  Two blocks an SM, and as many
// columns a block as give every SM two: 48.4 us, with one 63, with four 54.
template <bool F16, int ST, int YK, int HV>
__global__ void __launch_bounds__(kThreads, ST <= 2 || (ST <= 4 && HV == 1) ? 2 : 1) k_expand_wide(const __grid_constant__ AdapterParams P) {
  constexpr int TILE = 64, G = YK == 2 || HV == 2 ? 1 : 2, NP = 2 * HV;
  constexpr int YB = YK == 0 ? 4 : 2, TERMS = kTerms<F16, YK>;
  extern __shared__ __align__(16) uint32_t vs[];  // [TERMS][TILE][pitch / 2]; pitch in elements
  __shared__ int list[TILE];
  __shared__ __align__(8) float s_scale[TILE];
  __shared__ __align__(16) longlong2 s_row[TILE];  // bytes to the token's row of y and of out
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  int a, n;
  if (!find_tile<TILE>(P, list, a, n)) {
    pdl_wait();
    return;
  }
  // (rows past the tile's last are its last: their loads need no test)
  if (tid < TILE) {
    const long long t = list[min(tid, n - 1)];
    s_row[tid] = make_longlong2(t * P.y_stride * YB, t * P.out_stride * YB);
    s_scale[tid] = 0.f;
  }
  const int rank = adapter_rank(P, a), pitch = expand_pitch(P.R);
  const int c_first = P.cols * blockIdx.y, c_end = min(P.N, c_first + P.cols);
  __syncthreads();
  const uint16_t* const v0 = reinterpret_cast<const uint16_t*>(vs) + g * pitch + 4 * q;
  bool staged = false;
  for (int b0 = c_first; b0 < c_end; b0 += HV * kThreads) {
    const int w0 = b0 + 32 * HV * warp, n0 = w0 + 4 * q;  // the lane's: n0 + 16 p
    bool in[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) in[p] = n0 + 16 * p < c_end;
    // B: a column of each product's eight, four k a step
    uint2 bv[ST][2 * NP];
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      uint2(&b)[2 * NP] = bv[s];
      const int r = 16 * s + 4 * q;
#pragma unroll
      for (int c = 0; c < 2 * NP; ++c) {
        const int nc = w0 + 16 * (c >> 1) + 4 * (g >> 1) + 2 * (c & 1) + (g & 1);
        b[c] = make_uint2(0u, 0u);
        if (r >= rank || nc >= P.N) continue;
        const uint16_t* const row = P.B + ((size_t)a * P.N + nc) * P.R + r;
        if (P.R % 4 == 0) {
          b[c] = *reinterpret_cast<const uint2*>(row);
        } else {
          b[c].x = row[0] | (r + 1 < rank ? (uint32_t)row[1] << 16 : 0u);
          b[c].y = (r + 2 < rank ? row[2] : 0u) | (r + 3 < rank ? (uint32_t)row[3] << 16 : 0u);
        }
      }
      if (r + 4 > rank) {  // what lies past the rank does not count
        const uint32_t mx = r + 1 < rank ? ~0u : 0xFFFFu, my = r + 3 < rank ? ~0u : r + 2 < rank ? 0xFFFFu : 0u;
#pragma unroll
        for (int c = 0; c < 2 * NP; ++c) {
          b[c].x &= mx;
          b[c].y &= my;
        }
      }
    }
    // y of tokens 16 j + g (+ 8), as it lies in memory (YK < 2)
    const uint8_t* const y0 = static_cast<const uint8_t*>(P.y) + (size_t)n0 * YB;
    uint8_t* const o0 = static_cast<uint8_t*>(P.out) + (size_t)n0 * YB;
    uint4 yv[G][2][NP];
    auto ask = [&](int j0) {
#pragma unroll
      for (int u = 0; u < (YK < 2 ? G : 0); ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* const at = y0 + s_row[16 * (j0 + u) + 8 * h + g].x;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            if (!in[p]) continue;
            if (YK == 0) {
              yv[u][h][p] = *reinterpret_cast<const uint4*>(at + 16 * p * YB);
            } else {
              const uint2 w = *reinterpret_cast<const uint2*>(at + 16 * p * YB);
              yv[u][h][p].x = w.x, yv[u][h][p].y = w.y;
            }
          }
        }
    };
    ask(0);
    if (!staged) {
      pdl_wait();
      if (rank == 0 && P.out == P.y) return;
      if (rank > 0) stage_v<F16, TILE, TERMS>(P, list, a, n, rank, pitch, vs, s_scale);
      staged = true;
    }
    // (v of tokens past the last is 0, their y is the last's; they are not stored)
    for (int j0 = 0; 16 * j0 < n; j0 += G) {
      float d[G][2 * NP][4];
      if (rank > 0) {
        // the smallest term first; fp16: its whole product, then the other's
#pragma unroll
        for (int pass = F16 ? TERMS - 1 : 0; pass >= 0; --pass) {
          if (F16 && pass < TERMS - 1) {
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
              for (int c = 0; c < 2 * NP; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[u][c][e] *= 1.f / kLow;
          }
#pragma unroll
          for (int s = 0; s < ST; ++s) {
            if (16 * s >= rank) break;
#pragma unroll
            for (int u = 0; u < G; ++u) {
              const uint16_t* const v = v0 + 16 * (j0 + u) * pitch + 16 * s;
#pragma unroll
              for (int i = F16 ? pass : TERMS - 1; i >= pass; --i) {
                const uint2 t0 = *reinterpret_cast<const uint2*>(v + i * TILE * pitch);
                const uint2 t1 = *reinterpret_cast<const uint2*>(v + (i * TILE + 8) * pitch);
#pragma unroll
                for (int c = 0; c < 2 * NP; ++c) {
                  if (s == 0 && i == TERMS - 1)
                    mma16816<F16, true>(d[u][c], t0.x, t1.x, t0.y, t1.y, bv[s][c].x, bv[s][c].y);
                  else
                    mma16816<F16>(d[u][c], t0.x, t1.x, t0.y, t1.y, bv[s][c].x, bv[s][c].y);
                }
              }
            }
          }
        }
      } else {  // (the scale is 0 then: -0 leaves y as it is, a zero's sign too)
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int c = 0; c < 2 * NP; ++c) d[u][c][0] = d[u][c][1] = d[u][c][2] = d[u][c][3] = -0.f;
      }
      float y[G][2][NP][4];
#pragma unroll
      for (int u = 0; u < G; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = 16 * (j0 + u) + 8 * h + g;
          const float scale = s_scale[i];
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            float(&z)[4] = y[u][h][p];
            if (YK < 2) {
              raw_values4(yv[u][h][p], YK == 0 ? kF32 : P.y_dtype, z);
            } else {
              const size_t at = (size_t)list[min(i, n - 1)] * P.y_stride + n0 + 16 * p;
#pragma unroll
              for (int c = 0; c < 4; ++c) z[c] = n0 + 16 * p + c < c_end ? elem_load(P.y, P.y_dtype, at + c) : 0.f;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) z[c] = fmaf(scale, d[u][2 * p + (c >> 1)][2 * h + (c & 1)], z[c]);
          }
        }
      if (16 * (j0 + G) < n) ask(j0 + G);
#pragma unroll
      for (int u = 0; u < G; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = 16 * (j0 + u) + 8 * h + g;
          if (i >= n) continue;
          uint8_t* const at = o0 + s_row[i].y;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            if (!in[p]) continue;
            const float(&z)[4] = y[u][h][p];
            if (YK == 0) {
              *reinterpret_cast<float4*>(at + 16 * p * YB) = make_float4(z[0], z[1], z[2], z[3]);
            } else if (YK == 1) {
              *reinterpret_cast<uint2*>(at + 16 * p * YB) =
                  make_uint2(pack2(P.y_dtype, z[0], z[1]), pack2(P.y_dtype, z[2], z[3]));
            } else {
              const size_t to = (size_t)list[i] * P.out_stride + n0 + 16 * p;
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (n0 + 16 * p + c < c_end) elem_store(P.out, P.y_dtype, to + c, z[c]);
            }
          }
        }
    }
  }
}

template <bool F16>
cudaError_t launch_products(const AdapterParams& p, int blocks, cudaStream_t stream) {
  const bool wide = p.tile == 64;
  const dim3 grid(blocks, wide ? p.splits / 2 : p.splits, (p.R + kRankChunk - 1) / kRankChunk);
  auto shrink = [&](auto kern, int rows) {
    return launch_behind(kern, grid, kThreads, rows ? kWarps * 8 * (rows + 1) * 4 : 0, stream, p);
  };
  cudaError_t e = wide ? p.R <= 16   ? shrink(k_shrink_wide<F16, 1>, 0)
                         : p.R <= 32 ? shrink(k_shrink_wide<F16, 2>, 0)
                                     : shrink(k_shrink_wide<F16, 4>, 0)
                  : p.R <= 16 ? shrink(k_shrink<F16, 1>, 16)
                  : p.R <= 32 ? shrink(k_shrink<F16, 2>, 32)
                              : shrink(k_shrink<F16, 4>, 64);
  if (e != cudaSuccess) return e;
  const dim3 eg(blocks, (p.N + p.cols - 1) / p.cols);
  const int smem = (!p.vec || p.y_dtype == kF32 ? kTerms<F16, 0> : kTerms<F16, 1>) * p.tile * expand_pitch(p.R) * 2;
  auto expand = [&](auto kern) {
    if (smem > 48 * 1024) {
      const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (err != cudaSuccess) return err;
    }
    return launch_behind(kern, eg, kThreads, smem, stream, p);
  };
#define MOE_EXPAND(YK)                          \
  (p.R <= 16   ? expand(k_expand<F16, 1, YK>)   \
   : p.R <= 32 ? expand(k_expand<F16, 2, YK>)   \
   : p.R <= 64 ? expand(k_expand<F16, 4, YK>)   \
               : expand(k_expand<F16, 8, YK>))
#define MOE_EXPAND_WIDE(YK, HV)                        \
  (p.R <= 16   ? expand(k_expand_wide<F16, 1, YK, HV>) \
   : p.R <= 32 ? expand(k_expand_wide<F16, 2, YK, HV>) \
   : p.R <= 64 ? expand(k_expand_wide<F16, 4, YK, HV>) \
               : expand(k_expand_wide<F16, 8, YK, 1>))
  // (64 columns a warp where there are columns for every warp of a block then)
  if (!p.vec) return wide ? MOE_EXPAND_WIDE(2, 1) : MOE_EXPAND(2);
  if (!wide) return p.y_dtype == kF32 ? MOE_EXPAND(0) : MOE_EXPAND(1);
  if (p.N < 512) return p.y_dtype == kF32 ? MOE_EXPAND_WIDE(0, 1) : MOE_EXPAND_WIDE(1, 1);
  return p.y_dtype == kF32 ? MOE_EXPAND_WIDE(0, 2) : MOE_EXPAND_WIDE(1, 2);
#undef MOE_EXPAND_WIDE
#undef MOE_EXPAND
}

}  // namespace

}  // namespace moe

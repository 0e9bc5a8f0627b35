// What the kernels of attention over a paged cache (moe_ffn_attend) share: the
// sequences, the division of the work over the blocks, the partial results.
//
// A unit is a tile of rows of one sequence and one key head: its rows are the
// pairs (drafted token j, query head g of the group), r = j G + g.  Its work is the
// sequence's cached tokens in chunks.  All units' chunks, one behind the other, are
// divided evenly over the blocks, whatever the lengths: a block takes a range of
// chunks, which ends or begins inside a unit where it has to.  What a unit costs
// besides its chunks (queries, the warps' outputs that meet) counts as P.extra chunks
// ahead of its first: without, blocks of short sequences were the last to end (48
// sequences of 500 to 12,000 tokens: 82 us, 73 with them).  A unit that one
// block has whole is finished by it; the parts of another go to the workspace, at
// most two a block (the one that goes on in its first unit, the one that begins in
// its last), and a second kernel joins them.  The division depends on the lengths
// alone, and parts are joined in their order: results repeat bit for bit.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"
#include "moe_mma.cuh"

namespace moe {

struct AttendSeq {
  int t0, n, len;     // first row, rows, cached tokens
  int tiles, chunks;  // of rows, of tokens
  MOE_DEV bool none() const { return n > 0 && chunks == 0; }  // rows, but no token
  MOE_DEV long long work(int heads, int extra) const {
    return chunks ? (long long)tiles * heads * (chunks + extra) : 0;
  }
};

// a / b, by 32 bits where they do: a division in 64 takes a microsecond of a thread.
MOE_DEV long long attend_div(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

MOE_DEV AttendSeq attend_seq(const AttendParams& P, int b) {
  AttendSeq s;
  // (both bounds first: the difference of any two numbers may pass 32 bits)
  s.t0 = min(max(P.q_start[b], 0), P.T);
  s.n = max(min(max(P.q_start[b + 1], 0), P.T) - s.t0, 0);
  const long long most = (long long)P.max_pages * P.page_size;
  s.len = (int)min((long long)max(P.lens[b], 0), most);
  s.tiles = (s.n * P.G + P.rows - 1) / P.rows;
  s.chunks = (int)(((uint32_t)s.len + (1u << P.chunk_log) - 1u) >> P.chunk_log);
  return s;
}

// All units' chunks and extras over the blocks: `base` each, one more for the first `rest`.
struct AttendShare {
  long long base;
  int rest;
  MOE_DEV long long from(int c) const { return base * c + min(c, rest); }
  MOE_DEV int block_of(long long w) const {  // whose range holds place w
    const long long more = (base + 1) * rest;
    return (int)(w < more ? attend_div(w, base + 1) : rest + attend_div(w - more, base));
  }
};

// i / page_size.
MOE_DEV int attend_page(const AttendParams& P, int i) {
  return (int)(((unsigned long long)(uint32_t)i * P.page_mul) >> P.page_shift);
}

// A step of a block's range: one chunk of one unit.
struct AttendStep {
  AttendSeq s;
  int b, head, tile, chunk;
  long long left;  // places to the end of the range, this one included
  MOE_DEV void next(const AttendParams& P) {
    --left;
    if (++chunk < s.chunks) return;
    chunk = 0;
    left -= P.extra;  // (the range may end there: no step is left then)
    if (++tile < s.tiles) return;
    tile = 0;
    if (++head < P.Hkv) return;
    head = 0;
    while (left > 0 && ++b < P.B) {
      s = attend_seq(P, b);
      if (s.work(P.Hkv, P.extra) > 0) break;
    }
  }
};

// What the second kernel has to know of a block's range that begins inside a unit:
// the unit, the block in which it began and the number of its parts (0: the range
// begins with a unit, or there is none); and whether there are rows of sequences
// without tokens, which belong to no unit.
struct alignas(16) AttendFrom {
  int first, parts, none;
  int t0, n, head, tile;
};

// The range of this block: its first step, where it begins also left in the
// workspace.  All threads of the block call it.
template <int THREADS>
MOE_DEV AttendStep attend_begin(const AttendParams& P) {
  constexpr int W = THREADS / 32;
  __shared__ long long s_warp[2][W], s_at;
  __shared__ AttendSeq s_seq;
  __shared__ int s_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto seq_of = [&](int b) { return b < P.B ? attend_seq(P, b) : AttendSeq{0, 0, 0, 0, 0}; };
  // what lies before the thread, and all of the block's
  int turn = 0, none = 0;
  auto scan = [&](const AttendSeq& s, long long& all) {
    const long long own = s.work(P.Hkv, P.extra);
    long long upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) s_warp[turn][warp] = upto;
    none |= __syncthreads_or(s.none());
    long long before = upto - own;
    all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const long long v = s_warp[turn][w];
      before += w < warp ? v : 0;
      all += v;
    }
    turn ^= 1;
    return before;
  };
  // the sequences, THREADS at a time: mostly one round
  AttendSeq s = seq_of(tid);
  long long all, before = scan(s, all), total = all, base = 0;
  for (int b0 = THREADS; b0 < P.B; b0 += THREADS) {
    long long more;
    scan(seq_of(b0 + tid), more);
    total += more;
  }
  const long long even = attend_div(total, gridDim.x);
  const AttendShare share{even, (int)(total - even * gridDim.x)};
  const long long from = share.from(blockIdx.x), to = share.from(blockIdx.x + 1);
  for (int b0 = 0;;) {
    const int b = b0 + tid;
    const long long first = base + before;
    if (first <= from && from < first + s.work(P.Hkv, P.extra)) {
      s_seq = s;
      s_b = b;
      s_at = from - first;
    }
    base += all;
    if ((b0 += THREADS) >= P.B) break;
    s = seq_of(b0 + tid);
    before = scan(s, all);
  }
  __syncthreads();
  AttendStep a = {};
  a.left = to - from;
  if (a.left > 0) {
    a.b = s_b;
    a.s = s_seq;
    const int places = a.s.chunks + P.extra;
    const long long unit = attend_div(s_at, places);
    const int at = (int)(s_at - unit * places);  // the range's first place in its unit
    a.left -= max(P.extra - at, 0);
    a.chunk = max(at - P.extra, 0);
    a.head = (int)attend_div(unit, a.s.tiles);
    a.tile = (int)(unit - (long long)a.head * a.s.tiles);
  }
  if (tid == 64) {
    AttendFrom at = {0, 0, none, a.s.t0, a.s.n, a.head, a.tile};
    if (a.chunk > 0) {
      const long long unit = from - a.chunk;  // the place of its first chunk
      at.first = share.block_of(unit);
      at.parts = share.block_of(unit + a.s.chunks - 1) - at.first + 1;
    }
    P.from[blockIdx.x] = at;
  }
  return a;
}

// Rows of sequences without tokens: the second kernel, most of whose blocks have
// nothing to join, writes them, a row a block, and the block's warps share the
// sequences.  (By the first kernel, a sequence a thread, element by element, they kept
// the block's part of the attention waiting: four sequences of 2,000 tokens and four
// padded rows of 32 heads of 128 took 120 us, 13.3 now; 512 such rows 56 ms, now 21 us.)
template <int WARPS>
__device__ __noinline__ void attend_none(const AttendParams& P) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int block = blockIdx.y * gridDim.x + blockIdx.x, blocks = gridDim.x * gridDim.y;
  const float zero[4] = {};
  void* const out = P.out;
  float* const lse = P.lse;
  const long long head = P.o_head;
  const int type = P.out_dtype, heads = P.Hq, D = P.D, vec = P.o_vec;
  for (int b0 = 32 * warp; b0 < P.B; b0 += 32 * WARPS) {
    const AttendSeq s = b0 + lane < P.B ? attend_seq(P, b0 + lane) : AttendSeq{0, 0, 0, 0, 0};
    // the block's first row (single rows of several sequences go to different blocks)
    const int j0 = (block + blocks - (b0 + lane) % blocks) % blocks;
    for (uint32_t left = __ballot_sync(0xffffffffu, s.none() && j0 < s.n); left; left &= left - 1u) {
      const int i = __ffs(left) - 1, n = __shfl_sync(0xffffffffu, s.n, i), t0 = __shfl_sync(0xffffffffu, s.t0, i);
      for (int j = __shfl_sync(0xffffffffu, j0, i); j < n; j += blocks) {
        const long long t = t0 + j, row = t * P.o_stride;
        for (int h = 0; h < heads; ++h) {
          if (vec) {
            for (int d = 4 * lane; d < D; d += 128) elem_store4(out, type, row + h * head + d, zero);
          } else {
            for (int d = lane; d < D; d += 32) elem_store(out, type, row + h * head + d, 0.f);
          }
        }
        if (lse)
          for (int h = lane; h < heads; h += 32) lse[t * heads + h] = -INFINITY;
      }
    }
  }
}

// Elements 8 c .. 8 c + 7 of a query.
MOE_DEV uint4 attend_query(const AttendParams& P, int t, int h, int c) {
  const uint16_t* const from = P.q + (long long)t * P.q_stride + h * P.q_head + 8 * c;
  if (P.q_vec) return *reinterpret_cast<const uint4*>(from);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = from[2 * e] | (uint32_t)from[2 * e + 1] << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Whether row t, the j-th of its sequence, sees the token `own` places behind the
// first of the sequence's own ones.
MOE_DEV bool attend_sees(const AttendParams& P, int t, int j, int own) {
  if (own < 0) return true;
  if (!P.mask) return own <= j;
  return (own >> 5) < P.mask_words && (P.mask[(long long)t * P.mask_stride + (own >> 5)] >> (own & 31) & 1);
}

// tanh, relative error some 2^-22: by its series below 1/2, else by
// 1 - 2 / (exp(2 x) + 1), which has lost that many bits where it is small.
MOE_DEV float attend_tanh(float x) {
  const float y = x * x;
  float p = -929569.f / 638512875.f;
  p = fmaf(p, y, 21844.f / 6081075.f);
  p = fmaf(p, y, -1382.f / 155925.f);
  p = fmaf(p, y, 62.f / 2835.f);
  p = fmaf(p, y, -17.f / 315.f);
  p = fmaf(p, y, 2.f / 15.f);
  p = fmaf(p, y, -1.f / 3.f);
  const float far = 1.f - __fdividef(2.f, exp2_fast(x * 2.8853900817779268f) + 1.f);
  return fabsf(x) < 0.5f ? fmaf(p * y, x, x) : far;
}

// First token that some row of the sequence may not see.
MOE_DEV int attend_common(const AttendParams& P, const AttendSeq& s) {
  return s.n > 1 || P.mask ? max(s.len - s.n, 0) : s.len;
}

// Values that are not finite.  A weight enters the second product as a sum of numbers
// of either sign, so that an infinity gives NaN there, and what a row does not see must
// not enter it at all.  So they are taken out of the tiles that hold tokens which some
// rows do not see, and found again for the rows that do (attend_own).  Those of the
// other tokens, which all rows see, leave sums that are not finite: these columns are
// looked through once more in the cache (attend_odd), and what is there takes the sum's
// place.  Neither slows the stream of a cache without such values.
template <bool F16>
MOE_DEV bool odd16(uint32_t h) {  // all exponent bits set
  const uint32_t e = F16 ? 0x7C00u : 0x7F80u;
  return (h & e) == e;
}

// What columns c .. c + 7 of the values of tokens first, first + step, ... before end
// hold of them, two bits a column: infinity, minus infinity, both for NaN.
template <bool F16>
__device__ __noinline__ uint32_t attend_odd(const AttendParams& P, int b, int head, int first, int step, int end, int c) {
  uint32_t bits = 0u;
#pragma unroll 4
  for (int i = first; i < end; i += step) {
    const int at = attend_page(P, i), page = P.table[b * P.table_stride + at];
    if ((uint32_t)page >= (uint32_t)P.pages) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(P.v + page * P.vc_page + (long long)(i - at * P.page_size) * P.vc_slot +
                                                    head * P.vc_head + c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = w[e >> 1] >> (16 * (e & 1)) & 0xFFFFu;
      if (odd16<F16>(h)) bits |= (h & (F16 ? 0x3FFu : 0x7Fu) ? 3u : h >> 15 ? 2u : 1u) << (2 * e);
    }
  }
  return bits;
}
// One column's two bits in the place of its sum, where they are not 0.
MOE_DEV void attend_put_odd(float& sum, uint32_t bits) {
  if (bits & 3u) sum = __int_as_float((bits & 3u) == 3u ? 0x7FFFFFFF : bits & 1u ? 0x7F800000 : (int)0xFF800000);
}

// The sum of those in columns d .. d + 3 of tokens first .. end - 1 that row t, the j-th,
// sees.  The sequence's own tokens begin at `own`.
template <bool F16>
__device__ __noinline__ float4 attend_own(const AttendParams& P, int b, int head, int own, int t, int j, int first, int end,
                                          int d) {
  float x[4] = {};
  for (int i = first; i < end; ++i) {
    if (!attend_sees(P, t, j, i - own)) continue;
    const int at = attend_page(P, i), page = P.table[b * P.table_stride + at];
    if ((uint32_t)page >= (uint32_t)P.pages) continue;
    const uint16_t* const v = P.v + page * P.vc_page + (long long)(i - at * P.page_size) * P.vc_slot + head * P.vc_head + d;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (odd16<F16>(v[e])) x[e] += raw_value(v[e], F16 ? kF16 : kBf16);
  }
  return make_float4(x[0], x[1], x[2], x[3]);
}
// v += x, but for the sign of a zero.
MOE_DEV void attend_add_odd(float& v, float x) {
  if (x != 0.f) v += x;
}

MOE_DEV bool attend_finite(float v) { return fabsf(v) < INFINITY; }
// In the join: a part's infinities count without its factor, which may be 0.
MOE_DEV void attend_part_odd(float4& odd, const float4& part) {
  if (!attend_finite(part.x)) odd.x += part.x;
  if (!attend_finite(part.y)) odd.y += part.y;
  if (!attend_finite(part.z)) odd.z += part.z;
  if (!attend_finite(part.w)) odd.w += part.w;
}
MOE_DEV void attend_take_odd(float4& sum, const float4& odd) {
  if (odd.x != 0.f) sum.x = odd.x;
  if (odd.y != 0.f) sum.y = odd.y;
  if (odd.z != 0.f) sum.z = odd.z;
  if (odd.w != 0.f) sum.w = odd.w;
}
MOE_DEV bool attend_finite(const float4& v) {
  return attend_finite(v.x) && attend_finite(v.y) && attend_finite(v.z) && attend_finite(v.w);
}

// The largest running maximum is taken for 0 where there is none, so that
// exp2(-inf - 0) = 0.
MOE_DEV float attend_base(float m) { return m == -INFINITY ? 0.f : m; }

// Units of up to 128 rows and the join of their parts (moe_attend_wide.cu).
cudaError_t launch_attend_wide(AttendParams p, cudaStream_t stream);

}  // namespace moe

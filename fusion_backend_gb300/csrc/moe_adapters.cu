// Low-rank adapters of many requests beside a shared projection
// (moe_ffn_add_adapters): v_t = A_a x_t (k_shrink), then
// out_t = y_t + scale_a B_a v_t (k_expand).
//
// Both products run on tiles of up to 8 NT tokens that share an adapter, as
// mma.m16n8k16 with the adapter's rows as the 16 A rows and the tokens as the
// B columns, fp32 accumulators, operands straight from global memory: a lane
// takes 16 (A, x) or 8 (B) consecutive bytes of a row and the k index of the
// product is permuted alike on both sides, so every 32-byte sector read is used
// whole.  The work is bound by bytes (x, y, out once; an adapter once a tile),
// at R = 64 by 64 flops a byte: far below what the warp-level instructions
// give, so the tiles need no shared-memory staging or tensor memory.
//
// Tiles.  Up to kScanT tokens: block t looks through all adapter ids and owns a
// tile if its token is the first, (8 NT + 1)th, .. of its adapter.  More tokens:
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
constexpr int kOrderTokens = 32;      // tokens a block of k_order ranks, eight threads a token
constexpr int kRankChunk = 64;        // rows of A a block of k_shrink takes

// k_expand's shared memory: elements between two tokens' v (32 modulo 64 bytes:
// no bank conflicts), and the bytes of a stage.
__host__ __device__ constexpr int expand_pitch(int R) { return (R + 15) / 16 % 2 ? (R + 15) / 16 * 16 : (R + 15) / 16 * 16 + 16; }
__host__ __device__ constexpr int expand_stage(int R, int NT, int yb) {
  return kThreads * (NT * 2 * yb + (R + 15) / 16 * 4 * 8);
}

MOE_DEV int adapter_of(const AdapterParams& P, int t) {
  const int a = P.ids[t];
  return a < 0 || a >= P.n ? -1 : a;
}
MOE_DEV int adapter_rank(const AdapterParams& P, int a) {
  if (a < 0) return 0;
  return P.ranks ? max(0, min(P.R, P.ranks[a])) : P.R;
}

MOE_DEV void mma16816(bool f16, float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                      uint32_t b1) {
  if (f16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Places of the window's tokens in the order (adapter, token): a token's place
// is the number of tokens before it.  Eight threads a token, each against an
// eighth of the window.  marks[place]: the tokens of the tile that starts
// there, 0 where none does (a run of one adapter is cut every P.tile tokens).
__global__ void __launch_bounds__(8 * kOrderTokens) k_order(const __grid_constant__ AdapterParams P) {
  __shared__ __align__(16) int s_a[kWindow];
  const int tid = threadIdx.x, part = tid & 7;
  const int t0 = blockIdx.x * kWindow, n = min(kWindow, P.T - t0);
  const int i = blockIdx.y * kOrderTokens + (tid >> 3);
  pdl_wait();
  pdl_launch_dependents();
  // (no adapter comes first; past the window nothing is counted)
  for (int j = tid; j < kWindow; j += 8 * kOrderTokens) s_a[j] = j < n ? adapter_of(P, t0 + j) : 0x7FFFFFFF;
  __syncthreads();
  const int a = s_a[i];
  int before = 0, same_before = 0, same = 0;
#pragma unroll 4
  for (int j0 = 4 * part; j0 < n; j0 += 32) {
    const int4 v = *reinterpret_cast<const int4*>(s_a + j0);
    const int o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      before += o[e] < a;
      same += o[e] == a;
      same_before += o[e] == a && j0 + e < i;
    }
  }
  before += same_before;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    same += __shfl_xor_sync(0xffffffffu, same, o);
    same_before += __shfl_xor_sync(0xffffffffu, same_before, o);
  }
  if (part == 0 && i < n) {
    P.order[t0 + before] = t0 + i;
    P.adapter_at[t0 + before] = a;
    P.marks[t0 + before] = static_cast<uint8_t>(same_before % P.tile ? 0 : min(P.tile, same - same_before));
  }
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
        n = __shfl_sync(0xffffffffu, n, __ffs(who) - 1);
        place = __shfl_sync(0xffffffffu, place, __ffs(who) - 1);
        if (lane < n) list[lane] = P.order[place + lane];
        a = P.adapter_at[place];
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

// Blocks (tile, part of K, 64 rows of A).  The warps take 32-column blocks of K
// in turn; MT 16-row tiles of A, NT 8-token tiles.  D fragments meet in shared
// memory, summed over the warps in order.
template <bool F16, int MT, int NT>
__global__ void __launch_bounds__(kThreads) k_shrink(const __grid_constant__ AdapterParams P) {
  constexpr int TILE = 8 * NT, ROWS = 16 * MT;
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
        mma16816(F16, d[i][j], av[i][0].x, av[i][1].x, av[i][0].y, av[i][1].y, xv[j].x, xv[j].y);
        mma16816(F16, d[i][j], av[i][0].z, av[i][1].z, av[i][0].w, av[i][1].w, xv[j].z, xv[j].w);
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

// v of a tile as the B operand of the second product, two numbers of the
// operands' type an element: bf16 hi + lo keep 16 bits and more of v; fp16 keeps
// 22, of v scaled by a power of two to a largest element near 1, since v may
// pass fp16's range.  s_scale: what takes the token's product back, times the
// adapter's scale.  256 / TILE threads a token; ends with a block barrier.
template <bool F16, int TILE>
MOE_DEV void stage_v(const AdapterParams& P, const int* list, int a, int n, int rank, int pitch, uint32_t* vs,
                     float* s_scale) {
  const int tid = threadIdx.x;
  constexpr int TPT = kThreads / TILE;
  const int tok = tid / TPT, part = tid % TPT, padded = (rank + 15) & ~15;
  float top = 0.f;
  uint16_t* hi = reinterpret_cast<uint16_t*>(vs) + tok * pitch;
  uint16_t* lo = hi + TILE * pitch;
  float keep[kAdapterMaxRank / TPT];
#pragma unroll
  for (int i = 0; i < kAdapterMaxRank / TPT; ++i) {
    const int r = part + TPT * i;
    keep[i] = 0.f;
    if (tok < n && r < rank) {
      const float* v = P.v + (size_t)list[tok] * P.R + r;
      for (int k = 0; k < P.splits; ++k) keep[i] += __ldcg(v + (size_t)k * P.T * P.R);
    }
    top = fmaxf(top, fabsf(keep[i]));
  }
  float up = 1.f, down = 1.f;
  if (F16) {
#pragma unroll
    for (int o = TPT >> 1; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // 2^e with 2^e <= top < 2^(e + 1), kept within the normal numbers on both sides
    const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);
    if (top > 0.f && top < INFINITY) {
      up = __uint_as_float(e << 23);
      down = __uint_as_float((254u - e) << 23);
    }
  }
#pragma unroll
  for (int i = 0; i < kAdapterMaxRank / TPT; ++i) {
    const int r = part + TPT * i;
    if (r >= padded) break;
    const float v = keep[i] * down;
    const uint32_t h = pack2(F16 ? kF16 : kBf16, v, 0.f);
    float vh, none;
    unpack2(F16 ? kF16 : kBf16, h, vh, none);
    hi[r] = static_cast<uint16_t>(h);
    lo[r] = fabsf(vh) < INFINITY ? static_cast<uint16_t>(pack2(F16 ? kF16 : kBf16, v - vh, 0.f)) : 0;
  }
  if (part == 0) s_scale[tok] = up * (P.scales ? P.scales[a] : 1.f);
  __syncthreads();
}

MOE_DEV void mask_rank(uint2& b, int left) {  // keep the first `left` of four elements
  if (left >= 4) return;
  b.x &= left > 1 ? ~0u : 0xFFFFu;
  b.y &= left > 2 ? 0xFFFFu : 0u;
}

// One 16-wide step of the rank for 8 tokens: the two 16-row tiles of B against v.
template <bool F16>
MOE_DEV void mma_pair(const uint2 (&b)[4], uint2 vh, uint2 vl, float* d0, float* d1) {
  mma16816(F16, d0, b[0].x, b[1].x, b[0].y, b[1].y, vl.x, vl.y);
  mma16816(F16, d1, b[2].x, b[3].x, b[2].y, b[3].y, vl.x, vl.y);
  mma16816(F16, d0, b[0].x, b[1].x, b[0].y, b[1].y, vh.x, vh.y);
  mma16816(F16, d1, b[2].x, b[3].x, b[2].y, b[3].y, vh.x, vh.y);
}

// One 16-wide step of the rank: the lane's four rows of B (four k each) against
// v of the tile's tokens (v: hi of the lane's token and k; lo_at further: lo).
template <bool F16, int NT>
MOE_DEV void mma_step(const uint2 (&b)[4], const uint16_t* v, int lo_at, int n, float (&d)[2][NT][4], int pitch) {
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    if (8 * j >= n) continue;
    const uint2 vh = *reinterpret_cast<const uint2*>(v + 8 * j * pitch);
    const uint2 vl = *reinterpret_cast<const uint2*>(v + 8 * j * pitch + lo_at);
    mma_pair<F16>(b, vh, vl, d[0][j], d[1][j]);
  }
}

template <int BYTES>
MOE_DEV void cp_async(void* dst, const void* src, bool valid) {
  const uint32_t size = valid ? BYTES : 0;  // 0: zeros
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(size) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES), "r"(size)
                 : "memory");
}

// Blocks (tile, columns): the block goes through its columns 256 at a time, warp
// w taking 32 w .. of them as two 16-row tiles of B, whose rows are dealt so
// that a lane ends with four neighbouring columns n0 + 4g .. + 3 of tokens 2q
// and 2q + 1.  What a lane needs of y and B of the next two rounds is on its way
// into shared memory (asynchronous copies, a place of its own for every lane,
// so no thread waits for another) while it works on one: the loads of a round
// held in registers instead ran 46 us at 8192 x 2048 fp32 columns, rank 32.
// The first two rounds are asked for ahead of the wait on k_shrink, which
// writes neither y nor B.  YK: y and out are fp32 (0) or 16-bit (1); rows allow
// accesses of four elements, R % 4 == 0.
//
// VS: steps of the rank whose v the lane keeps in registers (every round and
// every warp reads the same), 0: read from shared memory in every round.
template <bool F16, int NT, int YK, int VS>
__global__ void __launch_bounds__(kThreads, 2) k_expand(const __grid_constant__ AdapterParams P) {
  constexpr int TILE = 8 * NT, YB = YK == 0 ? 16 : 8;
  extern __shared__ __align__(16) uint32_t vs[];  // v: [2][TILE][pitch / 2], then two stages
  __shared__ int list[TILE];
  __shared__ float s_scale[TILE];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  int a, n;
  if (!find_tile<TILE>(P, list, a, n)) {
    pdl_wait();
    pdl_launch_dependents();
    return;
  }
  const int rank = adapter_rank(P, a), steps = (rank + 15) / 16, pitch = expand_pitch(P.R);
  uint8_t* ring = reinterpret_cast<uint8_t*>(vs) + 2 * TILE * pitch * 2;
  const int stage_bytes = expand_stage(P.R, NT, YB);
  const int c_first = P.cols * blockIdx.y, c_end = min(P.N, c_first + P.cols);
  const int col = 32 * warp + 4 * g;
  int row[NT][2];  // the lane's tokens, -1: none
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) row[j][h] = 8 * j + 2 * q + h < n ? list[8 * j + 2 * q + h] : -1;
  // the lane's places: y [NT][2][256] of YB bytes, B [steps][4][256] of 8
  auto fetch = [&](int c0, int stage) {
    const int n0 = c0 + col;
    if (n0 < c_end) {
      uint8_t* ys = ring + stage * stage_bytes + tid * YB;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (row[j][h] >= 0)
            cp_async<YB>(ys + (2 * j + h) * kThreads * YB,
                         static_cast<const uint8_t*>(P.y) + ((size_t)row[j][h] * P.y_stride + n0) * (YB / 4), true);
      uint8_t* bs = ring + stage * stage_bytes + NT * 2 * kThreads * YB + tid * 8;
      const uint16_t* br = P.B + ((size_t)max(a, 0) * P.N + n0) * P.R + 4 * q;
      for (int s = 0; s < steps; ++s)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          cp_async<8>(bs + (4 * s + c) * kThreads * 8, 16 * s + 4 * q < rank ? br + (size_t)c * P.R + 16 * s : P.B,
                      16 * s + 4 * q < rank);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(c_first, 0);
  fetch(c_first + kThreads, 1);
  pdl_wait();
  pdl_launch_dependents();
  if (rank > 0) stage_v<F16, TILE>(P, list, a, n, rank, pitch, vs, s_scale);
  const uint16_t* const v = reinterpret_cast<const uint16_t*>(vs) + g * pitch + 4 * q;
  uint2 vk[VS > 0 ? VS : 1][NT][2];
  float scale[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int s = 0; s < VS; ++s) {
      const bool has = s < steps && 8 * j < n;
      vk[s][j][0] = has ? *reinterpret_cast<const uint2*>(v + 8 * j * pitch + 16 * s) : make_uint2(0u, 0u);
      vk[s][j][1] = has ? *reinterpret_cast<const uint2*>(v + (8 * j + TILE) * pitch + 16 * s) : make_uint2(0u, 0u);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) scale[j][h] = row[j][h] >= 0 && rank > 0 ? s_scale[8 * j + 2 * q + h] : 0.f;
  }
  for (int c0 = c_first, stage = 0; c0 < c_end; c0 += kThreads, stage ^= 1) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const int n0 = c0 + col;
    // (the products are a whole warp's: lanes past the last column take part)
    if (c0 + 32 * warp < c_end && !(rank == 0 && P.out == P.y)) {
      const uint8_t* ys = ring + stage * stage_bytes + tid * YB;
      const uint8_t* bs = ring + stage * stage_bytes + NT * 2 * kThreads * YB + tid * 8;
      float d[2][NT][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) d[i][j][0] = d[i][j][1] = d[i][j][2] = d[i][j][3] = 0.f;
      auto rows_of_b = [&](int s, uint2 (&bv)[4]) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          bv[c] = *reinterpret_cast<const uint2*>(bs + (4 * s + c) * kThreads * 8);
          mask_rank(bv[c], rank - 16 * s - 4 * q);
        }
      };
      if (VS > 0) {
#pragma unroll
        for (int s = 0; s < VS; ++s) {
          if (s >= steps) break;
          uint2 bv[4];
          rows_of_b(s, bv);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (8 * j >= n) continue;
            mma_pair<F16>(bv, vk[s][j][0], vk[s][j][1], d[0][j], d[1][j]);
          }
        }
      } else {
        for (int s = 0; s < steps; ++s) {
          uint2 bv[4];
          rows_of_b(s, bv);
          mma_step<F16, NT>(bv, v + 16 * s, TILE * pitch, n, d, pitch);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (row[j][h] < 0 || n0 >= c_end) continue;
          const uint8_t* yp = ys + (2 * j + h) * kThreads * YB;
          float y[4];
          if (YK == 0) {
            const float4 f = *reinterpret_cast<const float4*>(yp);
            y[0] = f.x, y[1] = f.y, y[2] = f.z, y[3] = f.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(yp);
            unpack2(P.y_dtype, u.x, y[0], y[1]);
            unpack2(P.y_dtype, u.y, y[2], y[3]);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) y[c] = fmaf(scale[j][h], d[c >> 1][j][2 * (c & 1) + h], y[c]);
          uint8_t* o = static_cast<uint8_t*>(P.out) + ((size_t)row[j][h] * P.out_stride + n0) * (YB / 4);
          if (YK == 0)
            *reinterpret_cast<float4*>(o) = make_float4(y[0], y[1], y[2], y[3]);
          else
            *reinterpret_cast<uint2*>(o) = make_uint2(pack2(P.y_dtype, y[0], y[1]), pack2(P.y_dtype, y[2], y[3]));
        }
    }
    fetch(c0 + 2 * kThreads, stage);  // what the lane had there has been used
  }
}

// The same for rows that do not allow accesses of four elements, or a pool
// whose R is no multiple of 4: element by element.
template <bool F16, int NT>
__global__ void __launch_bounds__(kThreads) k_expand_any(const __grid_constant__ AdapterParams P) {
  constexpr int TILE = 8 * NT;
  extern __shared__ __align__(16) uint32_t vs[];
  __shared__ int list[TILE];
  __shared__ float s_scale[TILE];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  int a, n;
  const bool found = find_tile<TILE>(P, list, a, n);
  pdl_wait();
  pdl_launch_dependents();
  if (!found) return;
  const int rank = adapter_rank(P, a), steps = (rank + 15) / 16, pitch = expand_pitch(P.R);
  if (rank == 0 && P.out == P.y) return;
  if (rank > 0) stage_v<F16, TILE>(P, list, a, n, rank, pitch, vs, s_scale);
  const int c_first = P.cols * blockIdx.y, c_end = min(P.N, c_first + P.cols);
  for (int n0 = c_first + 32 * warp + 4 * g; n0 - 4 * g < c_end; n0 += kThreads) {
    float y[NT][2][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 8 * j + 2 * q + h;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          y[j][h][c] =
              i < n && n0 + c < c_end ? elem_load(P.y, P.y_dtype, (size_t)list[i] * P.y_stride + n0 + c) : 0.f;
      }
    float d[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) d[i][j][0] = d[i][j][1] = d[i][j][2] = d[i][j][3] = 0.f;
    const uint16_t* v = reinterpret_cast<const uint16_t*>(vs) + g * pitch + 4 * q;
    for (int s = 0; s < steps; ++s) {
      const int r = 16 * s + 4 * q;
      uint2 bv[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          e[k] = n0 + c < c_end && r + k < rank ? P.B[((size_t)a * P.N + n0 + c) * P.R + r + k] : 0u;
        bv[c] = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
      }
      mma_step<F16, NT>(bv, v + 16 * s, TILE * pitch, n, d, pitch);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 8 * j + 2 * q + h;
        if (i >= n) continue;
        const float s = rank > 0 ? s_scale[i] : 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (n0 + c < c_end)
            elem_store(P.out, P.y_dtype, (size_t)list[i] * P.out_stride + n0 + c,
                       fmaf(s, d[c >> 1][j][2 * (c & 1) + h], y[j][h][c]));
      }
  }
}

constexpr int kMaxSms = 192;  // the workspace does not depend on the device

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
int windows(int T) { return (T + kWindow - 1) / kWindow; }

// Parts of K: enough blocks for the GPU from `tiles` tiles, each warp at least
// one 32-column block.
int splits_for(int sms, int tiles, int K) {
  const int most = (K + 32 * kWarps - 1) / (32 * kWarps);
  const int want = 2 * sms / (tiles > 0 ? tiles : 1);
  const int s = want < 8 ? want : 8;
  return s < 1 ? 1 : s < most ? s : most;
}

template <bool F16, int MT, int NT>
cudaError_t launch_shrink(const AdapterParams& p, dim3 grid, cudaStream_t stream) {
  constexpr int smem = kWarps * 8 * NT * (16 * MT + 1) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(k_shrink<F16, MT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_behind(k_shrink<F16, MT, NT>, grid, kThreads, smem, stream, p);
}

template <bool F16, int NT>
cudaError_t launch_tiles(const AdapterParams& p, int blocks, cudaStream_t stream) {
  const dim3 grid(blocks, p.splits, (p.R + kRankChunk - 1) / kRankChunk);
  cudaError_t e = p.R <= 16   ? launch_shrink<F16, 1, NT>(p, grid, stream)
                  : p.R <= 32 ? launch_shrink<F16, 2, NT>(p, grid, stream)
                              : launch_shrink<F16, 4, NT>(p, grid, stream);
  if (e != cudaSuccess) return e;
  const dim3 eg(blocks, (p.N + p.cols - 1) / p.cols);
  const int v_bytes = 2 * 8 * NT * expand_pitch(p.R) * 2;
  if (!p.vec) return launch_behind(k_expand_any<F16, NT>, eg, kThreads, v_bytes, stream, p);
  auto ring = [&](auto kern, int yb) {
    const int smem = v_bytes + 2 * expand_stage(p.R, NT, yb);
    if (smem > 48 * 1024) {
      const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (err != cudaSuccess) return err;
    }
    return launch_behind(kern, eg, kThreads, smem, stream, p);
  };
  if (p.R <= 32) return p.y_dtype == kF32 ? ring(k_expand<F16, NT, 0, 2>, 16) : ring(k_expand<F16, NT, 1, 2>, 8);
  return p.y_dtype == kF32 ? ring(k_expand<F16, NT, 0, 0>, 16) : ring(k_expand<F16, NT, 1, 0>, 8);
}

}  // namespace

// v for every part of K, then (many tokens) the order and the marks.  The
// fewest tiles that T tokens can make give the most parts.
size_t adapters_workspace(int T, int K, int N, int R) {
  (void)N;
  const size_t v = align256((size_t)splits_for(kMaxSms, (T + 31) / 32, K) * T * R * 4);
  return T <= kScanT ? v : v + 2 * align256((size_t)T * 4) + align256((size_t)T);
}

cudaError_t launch_adapters(AdapterParams p, cudaStream_t stream) {
  // tokens a tile: 32, or 8 where an adapter has no more than that on average
  // (a quarter of the registers; an adapter with more is read once every 8)
  const bool small = p.T <= 8 || p.T / 8 <= p.n;
  p.tile = small ? 8 : 32;
  const int least = (p.T + p.tile - 1) / p.tile, likely = least > p.n ? least : p.n < p.T ? p.n : p.T;
  p.splits = splits_for(p.sms, likely, p.K);
  // columns a block of k_expand goes through: finding the tile and staging its v
  // are paid once a block, so as many as leave about two blocks for every SM
  const int chunks = (p.N + kThreads - 1) / kThreads;
  int parts = 2 * p.sms / likely;
  parts = parts < 1 ? 1 : parts > chunks ? chunks : parts;
  p.cols = (chunks + parts - 1) / parts * kThreads;
  const uintptr_t four = p.y_dtype == kF32 ? 16 : 8;
  p.vec = p.N % 4 == 0 && p.R % 4 == 0 && reinterpret_cast<uintptr_t>(p.y) % four == 0 &&
          reinterpret_cast<uintptr_t>(p.out) % four == 0 && (p.T == 1 || (p.y_stride % 4 == 0 && p.out_stride % 4 == 0));
  int blocks = p.T;
  if (p.T > kScanT) {
    const int wn = (p.T + kWindow - 1) / kWindow, len = p.T < kWindow ? p.T : kWindow;
    uint8_t* w = reinterpret_cast<uint8_t*>(p.v) + align256((size_t)splits_for(kMaxSms, (p.T + 31) / 32, p.K) * p.T * p.R * 4);
    p.order = reinterpret_cast<int32_t*>(w);
    p.adapter_at = reinterpret_cast<int32_t*>(w + align256((size_t)p.T * 4));
    p.marks = w + 2 * align256((size_t)p.T * 4);
    // tiles of a window at most: full ones, and a last one of each adapter (and of the tokens that have none)
    p.slots = p.n < len ? len / p.tile + p.n + 1 : len;
    if (p.slots > len) p.slots = len;
    blocks = wn * p.slots;
    const cudaError_t e = launch_behind(k_order, dim3(wn, (len + kOrderTokens - 1) / kOrderTokens), 8 * kOrderTokens,
                                        0, stream, p);
    if (e != cudaSuccess) return e;
  }
  if (p.f16) return small ? launch_tiles<true, 1>(p, blocks, stream) : launch_tiles<true, 4>(p, blocks, stream);
  return small ? launch_tiles<false, 1>(p, blocks, stream) : launch_tiles<false, 4>(p, blocks, stream);
}

}  // namespace moe

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
// tile if its token is the first, 33rd, .. of its adapter.  More tokens: k_order
// sorts each window of kWindow tokens by adapter and lists the tiles.
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
constexpr int kScanT = 2 * kThreads;  // two ids a thread
constexpr int kWindow = 1024, kWindowLog = 10;
constexpr int kRankChunk = 64;        // rows of A a block of k_shrink takes

struct TileEntry {
  int adapter, start, n;  // -1: tokens without an adapter; order[start .. start + n)
};

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

// Sorts the window's tokens by (adapter, token) and lists its tiles: runs of
// one adapter cut every `tile` tokens.
__global__ void __launch_bounds__(kWindow / 2) k_order(const __grid_constant__ AdapterParams P) {
  __shared__ unsigned long long key[kWindow];
  __shared__ int s_warp[kWindow / 64];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * kWindow, n = min(kWindow, P.T - t0);
  pdl_wait();
  pdl_launch_dependents();
  for (int i = tid; i < kWindow; i += kWindow / 2)
    key[i] = i < n ? ((unsigned long long)(uint32_t)(adapter_of(P, t0 + i) + 1) << kWindowLog) | i : ~0ull;
  // bitonic sort; thread i compares the pair that its index spells with a 0
  // put in at bit j's place
  for (int k = 2; k <= kWindow; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      __syncthreads();
      const int a = ((tid & ~(j - 1)) << 1) | (tid & (j - 1)), b = a | j;
      const unsigned long long x = key[a], y = key[b];
      if ((x > y) == ((a & k) == 0)) {
        key[a] = y;
        key[b] = x;
      }
    }
  __syncthreads();
  // places 2 tid and 2 tid + 1: the start of their run (a running maximum),
  // then whether a tile starts there (a running sum)
  auto adapter_at = [&](int i) { return (uint32_t)(key[i] >> kWindowLog); };
  int start[2], m = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = 2 * tid + i;
    if (p > 0 && p < n && adapter_at(p) != adapter_at(p - 1)) m = p;
    start[i] = m;
  }
  int run = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run = max(run, v);
  }
  if (lane == 31) s_warp[warp] = run;
  int before = __shfl_up_sync(0xffffffffu, run, 1);
  if (lane == 0) before = 0;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before = max(before, s_warp[w]);
  __syncthreads();
  bool lead[2];
  int cnt = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = 2 * tid + i;
    start[i] = max(start[i], before);
    lead[i] = p < n && (p - start[i]) % P.tile == 0;
    cnt += lead[i];
  }
  int incl = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int at = incl - cnt;
  for (int w = 0; w < warp; ++w) at += s_warp[w];
  TileEntry* tiles = reinterpret_cast<TileEntry*>(P.tiles) + (size_t)blockIdx.x * kWindow;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = 2 * tid + i;
    if (lead[i]) {
      int c = 1;
      while (c < P.tile && p + c < n && adapter_at(p + c) == adapter_at(p)) ++c;
      tiles[at++] = TileEntry{(int)adapter_at(p) - 1, t0 + p, c};
    }
    if (p < n) P.order[t0 + p] = t0 + (int)(key[p] & (kWindow - 1));
  }
  if (tid == kWindow / 2 - 1) P.n_tiles[blockIdx.x] = at;
}

// The tile of this block (blockIdx.x): its adapter (-1: none), its tokens in
// `list`; false where the block has no tile.
template <int TILE>
MOE_DEV bool find_tile(const AdapterParams& P, int* list, int& a, int& n) {
  __shared__ int s_cnt[2][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (P.T > kScanT) {
    const int w = blockIdx.x / P.slots, s = blockIdx.x - w * P.slots;
    if (s >= P.n_tiles[w]) return false;
    const TileEntry e = reinterpret_cast<const TileEntry*>(P.tiles)[(size_t)w * kWindow + s];
    a = e.adapter;
    n = e.n;
    if (tid < n) list[tid] = P.order[e.start + tid];
    __syncthreads();
    return true;
  }
  const int t = blockIdx.x;
  a = adapter_of(P, t);
  int before = 0, cnt = 0;
  bool hit[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = 2 * tid + i;
    const bool same = j < P.T && adapter_of(P, j) == a;
    hit[i] = same && j >= t;
    before += same && j < t;
    cnt += hit[i];
  }
  int incl = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 31) {
    s_cnt[0][warp] = before;
    s_cnt[1][warp] = incl;
  }
  __syncthreads();
  int rank = 0, at = incl - cnt, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    rank += s_cnt[0][w];
    at += w < warp ? s_cnt[1][w] : 0;
    total += s_cnt[1][w];
  }
  if (rank % TILE) return false;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (hit[i]) {
      if (at < TILE) list[at] = 2 * tid + i;
      ++at;
    }
  n = min(TILE, total);
  __syncthreads();
  return true;
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

// Blocks (tile, 256 columns); warp w columns 32 w .. of them, two 16-row tiles
// of B whose rows are dealt so that a lane ends with four neighbouring columns
// n0 + 4g .. + 3 of tokens 2q and 2q + 1.  v enters as two numbers of the
// operands' type (bf16: hi + lo, 16 bits and more of v; fp16: 22 bits, scaled
// by a power of two to a largest element near 1, since v may pass fp16's
// range).  y, the ids and the adapter are read ahead of the wait on k_shrink.
template <bool F16, int NT>
__global__ void __launch_bounds__(kThreads) k_expand(const __grid_constant__ AdapterParams P) {
  constexpr int TILE = 8 * NT;
  extern __shared__ uint32_t vs[];  // [2][TILE][pitch / 2]: hi, then lo; pitch in elements
  __shared__ int list[TILE];
  __shared__ float s_scale[TILE];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  int a, n;
  if (!find_tile<TILE>(P, list, a, n)) {
    pdl_wait();
    pdl_launch_dependents();
    return;
  }
  const int rank = adapter_rank(P, a), steps = (rank + 15) / 16;
  const int Rp = (P.R + 15) & ~15;
  const int pitch = (Rp / 16) & 1 ? Rp : Rp + 16;  // 32 (mod 64) bytes a row: no bank conflicts
  const int n0 = 256 * blockIdx.y + 32 * warp + 4 * g;
  // y of the lane's columns and tokens
  float acc[NT][2][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 8 * j + 2 * q + h;
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[j][h][c] = 0.f;
      if (i >= n) continue;
      const size_t at = (size_t)list[i] * P.y_stride + n0;
      if (P.vec) {
        if (n0 < P.N) {
          if (P.y_dtype == kF32) {
            const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(P.y) + at);
            acc[j][h][0] = f.x, acc[j][h][1] = f.y, acc[j][h][2] = f.z, acc[j][h][3] = f.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(P.y) + at);
            unpack2(P.y_dtype, u.x, acc[j][h][0], acc[j][h][1]);
            unpack2(P.y_dtype, u.y, acc[j][h][2], acc[j][h][3]);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (n0 + c < P.N) acc[j][h][c] = elem_load(P.y, P.y_dtype, at + c);
      }
    }
  pdl_wait();
  pdl_launch_dependents();
  if (rank > 0) {
    // v of the tile: 256 / TILE threads a token
    constexpr int TPT = kThreads / TILE;
    const int tok = tid / TPT, part = tid % TPT;
    float top = 0.f;
    uint16_t* hi = reinterpret_cast<uint16_t*>(vs) + tok * pitch;
    uint16_t* lo = hi + TILE * pitch;
    auto v_of = [&](int r) {
      float s = 0.f;
      if (tok < n && r < rank)
        for (int k = 0; k < P.splits; ++k) s += __ldcg(P.v + ((size_t)k * P.T + list[tok]) * P.R + r);
      return s;
    };
    float keep[kAdapterMaxRank / TPT];
#pragma unroll
    for (int i = 0; i < kAdapterMaxRank / TPT; ++i) {
      const int r = part + TPT * i;
      if (r >= 16 * steps) break;
      keep[i] = v_of(r);
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
      if (r >= 16 * steps) break;
      const float v = keep[i] * down;
      const uint32_t h = pack2(F16 ? kF16 : kBf16, v, 0.f);
      float vh, none;
      unpack2(F16 ? kF16 : kBf16, h, vh, none);
      hi[r] = static_cast<uint16_t>(h);
      lo[r] = fabsf(vh) < INFINITY ? static_cast<uint16_t>(pack2(F16 ? kF16 : kBf16, v - vh, 0.f)) : 0;
    }
    if (part == 0) s_scale[tok] = up * (P.scales ? P.scales[a] : 1.f);
    __syncthreads();

    float d[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) d[i][j][0] = d[i][j][1] = d[i][j][2] = d[i][j][3] = 0.f;
    const uint16_t* br = P.B + ((size_t)a * P.N + n0) * P.R;
    for (int s = 0; s < steps; ++s) {
      const int r = 16 * s + 4 * q;  // the lane's four k of the step
      uint2 bv[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        bv[c] = make_uint2(0u, 0u);
        if (n0 + c >= P.N || r >= rank) continue;
        const uint16_t* row = br + (size_t)c * P.R + r;
        if (P.R % 4 == 0) {
          bv[c] = *reinterpret_cast<const uint2*>(row);
          if (r + 4 > rank) {
            if (r + 1 >= rank) bv[c].x &= 0xFFFFu;
            bv[c].y = r + 2 >= rank ? 0u : bv[c].y & 0xFFFFu;
          }
        } else {
          bv[c].x = row[0] | (r + 1 < rank ? (uint32_t)row[1] << 16 : 0u);
          bv[c].y = (r + 2 < rank ? row[2] : 0u) | (r + 3 < rank ? (uint32_t)row[3] << 16 : 0u);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (8 * j >= n) continue;
        const uint16_t* vp = reinterpret_cast<const uint16_t*>(vs) + (8 * j + g) * pitch + r;
        const uint2 vh = *reinterpret_cast<const uint2*>(vp), vl = *reinterpret_cast<const uint2*>(vp + TILE * pitch);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma16816(F16, d[i][j], bv[2 * i].x, bv[2 * i + 1].x, bv[2 * i].y, bv[2 * i + 1].y, vl.x, vl.y);
          mma16816(F16, d[i][j], bv[2 * i].x, bv[2 * i + 1].x, bv[2 * i].y, bv[2 * i + 1].y, vh.x, vh.y);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s = s_scale[8 * j + 2 * q + h];
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[j][h][c] = fmaf(s, d[c >> 1][j][2 * (c & 1) + h], acc[j][h][c]);
      }
  } else if (P.out == P.y) {
    return;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 8 * j + 2 * q + h;
      if (i >= n) continue;
      const size_t at = (size_t)list[i] * P.out_stride + n0;
      const float* v = acc[j][h];
      if (P.vec) {
        if (n0 < P.N) {
          if (P.y_dtype == kF32)
            *reinterpret_cast<float4*>(static_cast<float*>(P.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.out) + at) =
                make_uint2(pack2(P.y_dtype, v[0], v[1]), pack2(P.y_dtype, v[2], v[3]));
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (n0 + c < P.N) elem_store(P.out, P.y_dtype, at + c, v[c]);
      }
    }
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
int windows(int T) { return (T + kWindow - 1) / kWindow; }

// Parts of K: enough blocks for the GPU from `tiles` tiles, each warp at least
// one 32-column block.
int splits_for(int tiles, int K) {
  const int most = (K + 32 * kWarps - 1) / (32 * kWarps);
  const int want = 2 * 152 / (tiles > 0 ? tiles : 1);
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
  const int Rp = (p.R + 15) & ~15, pitch = (Rp / 16) & 1 ? Rp : Rp + 16;
  return launch_behind(k_expand<F16, NT>, dim3(blocks, (p.N + 255) / 256), kThreads, 2 * 8 * NT * pitch * 2, stream,
                       p);
}

}  // namespace

// v for every part of K, then (many tokens) the order and the tiles.  The
// fewest tiles that T tokens can make give the most parts.
size_t adapters_workspace(int T, int K, int N, int R) {
  (void)N;
  const size_t v = align256((size_t)splits_for((T + 31) / 32, K) * T * R * 4);
  if (T <= kScanT) return v;
  return v + align256((size_t)T * 4) + align256((size_t)windows(T) * 4) +
         align256((size_t)windows(T) * kWindow * sizeof(TileEntry));
}

cudaError_t launch_adapters(AdapterParams p, cudaStream_t stream) {
  // tokens a tile: 8 for a call of at most 8 tokens, else 32
  const bool small = p.T <= 8;
  p.tile = small ? 8 : 32;
  const int least = (p.T + p.tile - 1) / p.tile;
  p.splits = splits_for(least > p.n ? least : p.n < p.T ? p.n : p.T, p.K);
  const uintptr_t four = p.y_dtype == kF32 ? 16 : 8;
  p.vec = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.y) % four == 0 &&
          reinterpret_cast<uintptr_t>(p.out) % four == 0 && (p.T == 1 || (p.y_stride % 4 == 0 && p.out_stride % 4 == 0));
  int blocks = p.T;
  if (p.T > kScanT) {
    const int wn = windows(p.T);
    uint8_t* w = reinterpret_cast<uint8_t*>(p.v) + align256((size_t)splits_for((p.T + 31) / 32, p.K) * p.T * p.R * 4);
    p.order = reinterpret_cast<int32_t*>(w);
    w += align256((size_t)p.T * 4);
    p.n_tiles = reinterpret_cast<int32_t*>(w);
    w += align256((size_t)wn * 4);
    p.tiles = w;
    // tiles of a window at most: full ones, and a last one of each adapter (and of the tokens that have none)
    p.slots = p.n + 1 < kWindow ? kWindow / p.tile + p.n + 1 : kWindow;
    if (p.slots > kWindow) p.slots = kWindow;
    blocks = wn * p.slots;
    const cudaError_t e = launch_behind(k_order, dim3(wn), kWindow / 2, 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  if (p.f16) return small ? launch_tiles<true, 1>(p, blocks, stream) : launch_tiles<true, 4>(p, blocks, stream);
  return small ? launch_tiles<false, 1>(p, blocks, stream) : launch_tiles<false, 4>(p, blocks, stream);
}

}  // namespace moe

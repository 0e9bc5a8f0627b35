// Products of few tokens with 4-bit weights (moe_ffn_project):
//   y_tn = sum_g d_ng sum_{k in g} (c_nk - 8) x_tk + bias_n
//
// Bound by the stream of codes and scales up to some 16 tokens, by the warp-level
// tensor-core instruction above.  A tile is 16 MT rows of W and all of K; the KW
// warps over K of a block take slabs of 256 columns in turn, each with a ring of
// its own in shared memory that asynchronous copies fill tiles ahead, and meet
// once a tile to add their sums.  So every SM has its whole share of a small
// matrix on its way at once, and of a large one as much as the rings hold.
//
// mma.m16n8k16 with the rows of W as its rows: 16-byte pieces of 8 rows are what
// ldmatrix hands out, a lane then holds 8 codes of rows g and g + 8 that lie in
// one group, as bf16 (fp16) numbers c - 8 exactly.  The order of k inside those 8
// follows the nibbles (0 4, 1 5, 2 6, 3 7), x is put in the same order where it is
// loaded: straight from global memory, since each warp of a block has other
// columns of it.  A group's products go to sums of their own and from there, times
// the group's scale, to the row's: the products are exact and everything is added
// in fp32.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"
#include "moe_mma.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kSlab = 256;  // columns of a slab: 128 bytes of codes, 16 bytes of scales (group 32)
constexpr int kChunks = kSlab / 32;

// Code pairs (nibbles 0, 4 of v) as numbers c - 8: the nibble in the mantissa of
// 128 (bf16), 1024 (fp16), less 136 (1032), exact.
template <bool F16>
MOE_DEV uint32_t code_pair(uint32_t v) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(0x000F000Fu), "r"(F16 ? 0x64006400u : 0x43004300u));
  if constexpr (F16)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x64086408u));
  else
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x43084308u));
  return r;
}

template <int MT>
__host__ __device__ constexpr int stage_bytes() {
  return 16 * MT * (128 + 16);
}

template <int NT, int MT, int STAGES>
__host__ __device__ constexpr int smem_bytes() {
  return kWarps * (STAGES * stage_bytes<MT>() + 16 * MT * (8 * NT + 1) * 4);
}

// NT: tiles of 8 tokens.  GL: log2(group / 32).
template <bool F16, int NT, int MT, int STAGES, int GL>
__global__ void __launch_bounds__(32 * kWarps, NT <= 2 ? 2 : 1) k_project(const __grid_constant__ ProjectParams P) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kStage = stage_bytes<MT>();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int kw = P.k_warps, kpart = warp % kw, tpart = warp / kw, tiles_at_once = kWarps / kw;
  const int t0 = blockIdx.y * 8 * NT;
  const int slabs = (P.K + kSlab - 1) / kSlab, mine = (slabs - kpart + kw - 1) / kw;  // slabs of the warp in a tile
  const int ntiles = (P.N + 16 * MT - 1) / (16 * MT);
  uint8_t* const ring = smem + warp * STAGES * kStage;
  float* const sums = reinterpret_cast<float*>(smem + kWarps * STAGES * kStage);
  constexpr int kPitch = 8 * NT + 1, kSums = 16 * MT * kPitch;
  pdl_wait();

  // the warp's steps: its slabs of its tiles, in order
  struct At {
    int tile, j;
  };
  const int tile_step = gridDim.x * tiles_at_once;
  auto next = [&](At& a) {
    if (++a.j >= mine) {
      a.j = 0;
      a.tile += tile_step;
    }
  };
  auto load = [&](const At& a, int stage) {
    if (a.tile < ntiles && mine > 0) {
      const int k0 = (kpart + a.j * kw) * kSlab, chunks = min(kChunks, (P.K - k0) >> 5);
      const uint32_t dst = smem_u32(ring + stage * kStage);
#pragma unroll
      for (int i = 0; i < 4 * MT; ++i) {
        const int r = 4 * i + (lane >> 3), c = lane & 7, n = a.tile * 16 * MT + r;
        const bool on = n < P.N && c < chunks;
        const uint8_t* const row = P.w + (long long)(n < P.N ? n : 0) * P.w_stride;
        copy16(dst + r * 128 + ((c ^ (r & 7)) << 4), on ? row + (k0 >> 1) + 16 * c : P.w, on ? 16u : 0u);
      }
      if (lane < 16 * MT) {
        const int n = a.tile * 16 * MT + lane;
        const uint8_t* const row = P.w + (long long)(n < P.N ? n : 0) * P.w_stride + (P.K >> 1);
        const uint32_t at = dst + 16 * MT * 128 + lane * 16;
        const uint32_t bytes = n < P.N ? (uint32_t)(2 * (chunks >> GL)) : 0u;
        const uint8_t* const src = bytes ? row + (k0 >> (4 + GL)) : P.w;
        if (GL == 0) copy16(at, src, bytes);
        if (GL == 1) copy8(at, src, bytes);
        if (GL == 2) copy4(at, src, bytes);
      }
    }
    copy_commit();
  };

  At ahead{(int)blockIdx.x * tiles_at_once + tpart, 0}, now = ahead;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) {
    load(ahead, s);
    next(ahead);
  }
  // x of one chunk, in the order of the codes' nibbles
  auto load_x = [&](uint4 (&x)[NT], int k) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int t = t0 + 8 * j + g;
      x[j] = t < P.T ? __ldg(reinterpret_cast<const uint4*>(P.x + (size_t)t * P.x_stride + k + 8 * q))
                     : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  int stage = 0, stage_in = STAGES - 1;
  for (int base = blockIdx.x * tiles_at_once; base < ntiles; base += tile_step) {
    float acc[MT][NT][4] = {};
    for (int j = 0; j < mine; ++j) {
      const int k0 = (kpart + j * kw) * kSlab, chunks = min(kChunks, (P.K - k0) >> 5);
      uint4 x[NT];
      load_x(x, k0);
      copy_wait<STAGES - 2>();
      __syncwarp();
      load(ahead, stage_in);
      next(ahead);
      stage_in = stage_in + 1 == STAGES ? 0 : stage_in + 1;
      const uint32_t codes = smem_u32(ring + stage * kStage);
      const __half* const scales = reinterpret_cast<const __half*>(ring + stage * kStage + 16 * MT * 128);
      float part[MT][NT][4];
#pragma unroll
      for (int c2 = 0; c2 < kChunks; c2 += 2) {
        if (c2 >= chunks) break;
        // codes of two chunks: (rows, chunk) of matrix i = (i & 1, i >> 1)
        uint32_t w[MT][4];
        const int r = (lane & 7) + (lane & 8), c = c2 + (lane >> 4);
#pragma unroll
        for (int m = 0; m < MT; ++m) ldmatrix4(w[m], codes + (16 * m + r) * 128 + ((c ^ (r & 7)) << 4));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (c2 + h >= chunks) break;
          uint4 xn[NT];
          if (c2 + h + 1 < chunks) load_x(xn, k0 + 32 * (c2 + h + 1));
          const bool first = ((c2 + h) & ((1 << GL) - 1)) == 0;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint32_t a = w[m][2 * h], b = w[m][2 * h + 1];  // rows g and g + 8
            const uint32_t a0 = code_pair<F16>(a), b0 = code_pair<F16>(b), a1 = code_pair<F16>(a >> 4),
                           b1 = code_pair<F16>(b >> 4), a2 = code_pair<F16>(a >> 8), b2 = code_pair<F16>(b >> 8),
                           a3 = code_pair<F16>(a >> 12), b3 = code_pair<F16>(b >> 12);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float(&d)[4] = part[m][n];
              if (first) d[0] = d[1] = d[2] = d[3] = 0.f;
              mma16<F16>(d, a0, b0, a1, b1, __byte_perm(x[n].x, x[n].z, 0x5410), __byte_perm(x[n].x, x[n].z, 0x7632));
              mma16<F16>(d, a2, b2, a3, b3, __byte_perm(x[n].y, x[n].w, 0x5410), __byte_perm(x[n].y, x[n].w, 0x7632));
            }
          }
          if (((c2 + h + 1) & ((1 << GL) - 1)) == 0) {
            const int at = (c2 + h) >> GL;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const float s0 = __half2float(scales[(16 * m + g) * 8 + at]);
              const float s1 = __half2float(scales[(16 * m + g + 8) * 8 + at]);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                acc[m][n][0] = fmaf(part[m][n][0], s0, acc[m][n][0]);
                acc[m][n][1] = fmaf(part[m][n][1], s0, acc[m][n][1]);
                acc[m][n][2] = fmaf(part[m][n][2], s1, acc[m][n][2]);
                acc[m][n][3] = fmaf(part[m][n][3], s1, acc[m][n][3]);
              }
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) x[n] = xn[n];
        }
      }
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    // the warps' sums, in their order
    float* const own = sums + warp * kSums;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) own[(16 * m + g + 8 * (e >> 1)) * kPitch + 8 * n + 2 * q + (e & 1)] = acc[m][n][e];
    __syncthreads();
    const int tokens = min(8 * NT, P.T - t0);
    for (int i = threadIdx.x; i < tiles_at_once * 16 * MT * tokens; i += 32 * kWarps) {
      const int r = i % (16 * MT), u = i / (16 * MT), t = u % tokens, p = u / tokens;
      const int n = (base + p) * 16 * MT + r;
      if (n >= P.N) continue;
      float v = 0.f;
      for (int k = 0; k < kw; ++k) v += sums[(p * kw + k) * kSums + r * kPitch + t];
      if (P.bias) v += P.bias[n];
      elem_store(P.y, P.y_dtype, (size_t)(t0 + t) * P.y_stride + n, v);
    }
    __syncthreads();
  }
  copy_wait<0>();
}

template <bool F16, int NT, int MT, int STAGES, int GL>
cudaError_t launch(const ProjectParams& p, cudaStream_t stream) {
  constexpr int smem = smem_bytes<NT, MT, STAGES>();
  auto* const kern = k_project<F16, NT, MT, STAGES, GL>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int at_once = kWarps / p.k_warps, tiles = (p.N + 16 * MT - 1) / (16 * MT);
  const int want = (tiles + at_once - 1) / at_once, most = p.sms * (NT <= 2 ? 2 : 1);
  return launch_behind(kern, dim3(want < most ? want : most, (p.T + 8 * NT - 1) / (8 * NT)), 32 * kWarps, smem, stream,
                       p);
}

template <bool F16, int GL>
cudaError_t launch_tokens(const ProjectParams& p, cudaStream_t stream) {
  if (p.T <= 8) return launch<F16, 1, 1, 4, GL>(p, stream);
  if (p.T <= 16) return launch<F16, 2, 1, 4, GL>(p, stream);
  if (p.T <= 32) return launch<F16, 4, 2, 3, GL>(p, stream);
  return launch<F16, 8, 2, 3, GL>(p, stream);
}

}  // namespace

cudaError_t launch_project(ProjectParams p, cudaStream_t stream) {
  const int slabs = (p.K + kSlab - 1) / kSlab;
  p.k_warps = slabs >= 8 ? 8 : slabs >= 4 ? 4 : slabs >= 2 ? 2 : 1;
  const int gl = p.group == 32 ? 0 : p.group == 64 ? 1 : 2;
  if (p.f16)
    return gl == 0 ? launch_tokens<true, 0>(p, stream)
           : gl == 1 ? launch_tokens<true, 1>(p, stream)
                     : launch_tokens<true, 2>(p, stream);
  return gl == 0 ? launch_tokens<false, 0>(p, stream)
         : gl == 1 ? launch_tokens<false, 1>(p, stream)
                   : launch_tokens<false, 2>(p, stream);
}

}  // namespace moe

// Products of few tokens with 4-bit weights (moe_ffn_project):
//   y_tn = sum_g d_ng sum_{k in g} (c_nk - 8) x_tk + bias_n
//
// Bound by the stream of codes and scales up to some 16 tokens, by the warp-level
// tensor-core instruction above.  A tile is 16 rows of W and all of K; the warps
// of a block that share a tile take slabs of 256 columns in turn, each with a ring
// of its own in shared memory that tensor copies fill tiles ahead, and meet once a
// batch of tiles to add their sums.  So every SM has its whole share of a small
// matrix on its way at once, and of a large one as much as the rings hold; a block's
// tiles are neighbours, as many for each block as for any other.
//
// mma.m16n8k16 with the rows of W as its rows: 16-byte pieces of 8 rows are what
// ldmatrix hands out, a lane then holds 8 codes of rows g and g + 8 that lie in
// one group, as numbers (c - 8) / 64 in bf16, c - 8 in fp16, exactly.  The order of k
// inside those 8 follows the nibbles (0 4, 1 5, 2 6, 3 7), x is put in the same order
// where it is loaded: straight from global memory, since each warp of a block has other
// columns of it, and once for all tiles where a warp has one slab of every tile.  A
// group's products go to sums of their own and from there, times the group's scale,
// to the row's: the products are exact and everything is added in fp32.
//
// Measured (weights from HBM): 5120 x 2048, 1 token 3.9 us, 16 tokens 6.0, 61 tokens
// 11.6, 256 tokens 30, 1024 tokens 123: above 32 tokens each further 32 turn the codes
// into numbers again.  100003 x 2048, 4 tokens 25.3 us, 4.6 TB/s: no unit is full (issue
// slots 65 %, integer pipe 51 %, HBM 53 %); warps wait for each other's issue, for fixed
// latencies and for the integer pipe about as long, and at the barriers of a batch a
// third of that.  x from L2 for every tile of rows, the first form, took 19.6 us for 61
// tokens.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_elem.cuh"
#include "moe_internal.h"
#include "moe_mma.cuh"
#include "moe_tma.cuh"

namespace moe {

namespace {

constexpr int kSlab = 256;  // columns of a slab: 128 bytes of codes
constexpr int kChunks = kSlab / 32;

// The codes of a word as four pairs of numbers: nibbles (0, 4), (1, 5), (2, 6),
// (3, 7).  bf16: (c - 8) / 64; fp16: c - 8; exactly.  A mask and a multiply-add a
// pair, and one shift for all.  bf16: the low byte of a number with nothing else set,
// N, is N 2^-133, the subnormal range and the first exponent above it being one
// scale: so a nibble at bit 0 or 4 is c 2^-133 or c 2^-129.  fp16: a nibble at bit 0
// or 4 of 1024 is 1024 + c or 1024 + 16 c.  (A shift for every pair is 7 integer
// instructions a word instead of 5: 27.0 us for 100003 rows where this took 25.7.)
template <bool F16>
MOE_DEV void code_pairs(uint32_t v, uint32_t (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? v : v >> 8, mask = i & 1 ? 0x00F000F0u : 0x000F000Fu;
    if constexpr (F16) {
      uint32_t n;
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(n) : "r"(w), "r"(mask), "r"(0x64006400u));
      // 1 n - 1032, n / 16 - 72
      asm("fma.rn.f16x2 %0, %1, %2, %3;"
          : "=r"(r[i])
          : "r"(n), "r"(i & 1 ? 0x2C002C00u : 0x3C003C00u), "r"(i & 1 ? 0xD480D480u : 0xE408E408u));
    } else {
      // 2^127 n - 1 / 8, 2^123 n - 1 / 8
      asm("fma.rn.bf16x2 %0, %1, %2, %3;"
          : "=r"(r[i])
          : "r"(w & mask), "r"(i & 1 ? 0x7D007D00u : 0x7F007F00u), "r"(0xBE00BE00u));
    }
  }
}
template <bool F16>
constexpr float kCodeScale = F16 ? 1.f : 64.f;

// Shared memory: the warps' rings of codes, of scales (16 bytes a row and slab),
// the sums of a batch of BT tiles, the barriers.
template <int WARPS, int NT, int STAGES, int BT>
struct Layout {
  static constexpr int kCodes = 16 * 128, kScales = 16 * 16, kPitch = 8 * NT + 1, kRows = BT * 16;
  static constexpr int scales_at = WARPS * STAGES * kCodes, sums_at = scales_at + WARPS * STAGES * kScales,
                       bars_at = sums_at + (WARPS * kRows * kPitch * 4 + 15) / 16 * 16,
                       bytes = bars_at + WARPS * STAGES * 8 + 1024;  // (rings start at a multiple of 1024)
};

// NT: tiles of 8 tokens.  GL: log2(group / 32).  HOLD: a warp has one slab of
// every tile, whose x stays in registers.
template <bool F16, int WARPS, int NT, int STAGES, int BT, int GL, bool HOLD, int OCC>
__global__ void __launch_bounds__(32 * WARPS, OCC) k_project(const __grid_constant__ ProjectParams P) {
  using L = Layout<WARPS, NT, STAGES, BT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int kw = P.k_warps, kpart = warp % kw, tpart = warp / kw, at_once = WARPS / kw;
  const int t0 = blockIdx.y * 8 * NT;
  const int slabs = (P.K + kSlab - 1) / kSlab, mine = HOLD ? kpart < slabs : (slabs - kpart + kw - 1) / kw;
  const int ntiles = (P.N + 16 - 1) / (16);
  const int lo = (int)((long long)ntiles * blockIdx.x / gridDim.x), hi = (int)((long long)ntiles * (blockIdx.x + 1) / gridDim.x);
  uint8_t* const codes = smem + warp * STAGES * L::kCodes;
  uint8_t* const scales = smem + L::scales_at + warp * STAGES * L::kScales;
  float* const sums = reinterpret_cast<float*>(smem + L::sums_at);
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + L::bars_at) + warp * STAGES;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < STAGES; ++s) mbar_init(full + s, 1);
    mbar_fence_init();
    prefetch_tensormap(&P.tm_codes);
    prefetch_tensormap(&P.tm_scales);
  }
  __syncwarp();
  pdl_wait();
  fence_proxy_async_global();

  // the warp's steps: its slabs of its tiles, in order
  int tile_in = lo + tpart, slab_in = 0;
  const uint64_t policy = policy_evict_first();
  bool dead = false;  // the warp's: a copy never came; nothing is asked for any more, results are NaN
  auto load = [&](int stage) {
    if (tile_in < hi && mine > 0) {
      if (lane == 0 && !dead) {
        const int k0 = (kpart + slab_in * kw) * kSlab;
        mbar_arrive_expect_tx(full + stage, L::kCodes + L::kScales + P.lost);
        tensor_load_2d(codes + stage * L::kCodes, &P.tm_codes, k0 >> 1, tile_in * 16, full + stage, policy);
        // 16 bytes that hold the slab's scales: of one slab, two or four
        tensor_load_2d(scales + stage * L::kScales, &P.tm_scales, (P.K >> 1) + (k0 >> (4 + GL) & ~15), tile_in * 16,
                       full + stage, policy);
      }
      if (HOLD || ++slab_in >= mine) {
        slab_in = 0;
        tile_in += at_once;
      }
    }
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) load(s);
  // x of one chunk (B of the chunk's two products), in the order of the codes' nibbles
  auto load_x = [&](uint32_t (&x)[NT][4], int k) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int t = t0 + 8 * j + g;
      const uint4 v = t < P.T ? *reinterpret_cast<const uint4*>(P.x + (size_t)t * P.x_stride + k + 8 * q)
                              : make_uint4(0u, 0u, 0u, 0u);
      x[j][0] = v.x, x[j][1] = v.y, x[j][2] = v.z, x[j][3] = v.w;
    }
  };
  auto order_x = [&](uint32_t (&x)[NT][4]) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint32_t a = x[j][0], b = x[j][1], c = x[j][2], d = x[j][3];
      x[j][0] = __byte_perm(a, c, 0x5410), x[j][1] = __byte_perm(a, c, 0x7632);
      x[j][2] = __byte_perm(b, d, 0x5410), x[j][3] = __byte_perm(b, d, 0x7632);
    }
  };
  uint32_t xh[HOLD ? kChunks : 1][NT][4];
  if constexpr (HOLD) {
    const int chunks = min(kChunks, (P.K - kpart * kSlab) >> 5);  // (negative: no slab)
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      if (c < chunks) load_x(xh[c], kpart * kSlab + 32 * c);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) order_x(xh[c]);
  }
  int stage = 0, stage_in = STAGES - 1;
  uint32_t parity = 0;
  for (int base = lo; base < hi; base += BT) {
    const int in_batch = min(BT, hi - base);
    for (int u = tpart; u < in_batch; u += at_once) {
      float acc[NT][4] = {};
      for (int j = 0; j < mine; ++j) {
        const int k0 = (kpart + j * kw) * kSlab, chunks = min(kChunks, (P.K - k0) >> 5);
        uint32_t x[NT][4];
        if constexpr (!HOLD) load_x(x, k0);
        __syncwarp();
        load(stage_in);
        stage_in = stage_in + 1 == STAGES ? 0 : stage_in + 1;
        if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait(full + stage, parity));
        const uint32_t codes_at = smem_u32(codes + stage * L::kCodes);
        // the slab's scales of rows g and g + 8: 8, 4 or 2 each
        uint32_t sc0[4], sc1[4];
        {
          const uint8_t* const from = scales + stage * L::kScales + g * 16 + (k0 >> (4 + GL) & 15);
#pragma unroll
          for (int e = 0; e < 4 >> GL; ++e) {
            sc0[e] = *reinterpret_cast<const uint32_t*>(from + 4 * e);
            sc1[e] = *reinterpret_cast<const uint32_t*>(from + 128 + 4 * e);
          }
        }
        auto scale_of = [](const uint32_t(&sc)[4], int i) {
          const __half2 v = *reinterpret_cast<const __half2*>(&sc[i >> 1]);
          return i & 1 ? __high2float(v) : __low2float(v);
        };
        float part[NT][4];
        // two chunks, c2 and the next; ALL: both are there
        auto pair = [&](int c2, auto whole) {
          constexpr bool ALL = decltype(whole)::value;
          // codes of two chunks: (rows, chunk) of matrix i = (i & 1, i >> 1)
          uint32_t w[4];
          const int r = lane & 15, c = c2 + (lane >> 4);
          ldmatrix4(w, codes_at + r * 128 + ((c ^ (r & 7)) << 4));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!ALL && c2 + h >= chunks) break;
            [[maybe_unused]] uint32_t xn[NT][4];
            if constexpr (!HOLD) {
              if (c2 + h + 1 < chunks) load_x(xn, k0 + 32 * (c2 + h + 1));
              order_x(x);
            }
            uint32_t(&b)[NT][4] = HOLD ? xh[HOLD ? c2 + h : 0] : x;
            const bool first = ((c2 + h) & ((1 << GL) - 1)) == 0;
            const uint32_t v0 = w[2 * h], v1 = w[2 * h + 1];  // rows g and g + 8
            uint32_t a[4], e[4];
            code_pairs<F16>(v0, a);
            code_pairs<F16>(v1, e);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (first)
                mma16_first<F16>(part[n], a[0], e[0], a[1], e[1], b[n][0], b[n][1]);
              else
                mma16<F16>(part[n], a[0], e[0], a[1], e[1], b[n][0], b[n][1]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16<F16>(part[n], a[2], e[2], a[3], e[3], b[n][2], b[n][3]);
            if (((c2 + h + 1) & ((1 << GL) - 1)) == 0) {
              const int at = (c2 + h) >> GL;
              const float s0 = scale_of(sc0, at), s1 = scale_of(sc1, at);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                fma_pair(acc[n][0], acc[n][1], part[n][0], part[n][1], s0);
                fma_pair(acc[n][2], acc[n][3], part[n][2], part[n][3], s1);
              }
            }
            if constexpr (!HOLD) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][e] = xn[n][e];
            }
          }
        };
        if (chunks == kChunks) {
#pragma unroll
          for (int c2 = 0; c2 < kChunks; c2 += 2) pair(c2, std::true_type{});
        } else {
#pragma unroll
          for (int c2 = 0; c2 < kChunks; c2 += 2) {
            if (c2 >= chunks) break;
            pair(c2, std::false_type{});
          }
        }
        if (++stage == STAGES) {
          stage = 0;
          parity ^= 1u;
        }
      }
      if (dead) {
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = __int_as_float(0x7FFFFFFF);
      }
      float* const own = sums + (kpart * L::kRows + u * 16) * L::kPitch;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) own[(g + 8 * (e >> 1)) * L::kPitch + 8 * n + 2 * q + (e & 1)] = acc[n][e] * kCodeScale<F16>;
    }
    __syncthreads();
    // the warps' sums, in their order
    const int tokens = min(8 * NT, P.T - t0);
    for (int i = threadIdx.x; i < L::kRows * tokens; i += 32 * WARPS) {
      const int r = i % L::kRows, t = i / L::kRows, n = base * 16 + r;
      if (r >= in_batch * 16 || n >= P.N) continue;
      float v = 0.f;
      for (int k = 0; k < kw; ++k) v += sums[(k * L::kRows + r) * L::kPitch + t];
      if (P.bias) v += P.bias[n];
      elem_store(P.y, P.y_dtype, (size_t)(t0 + t) * P.y_stride + n, v);
    }
    __syncthreads();
  }
  if (dead)  // the block's shared memory is its own until copies that are under way have come
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

template <bool F16, int WARPS, int NT, int STAGES, int BT, int GL, bool HOLD, int OCC>
cudaError_t launch(ProjectParams& p, cudaStream_t stream) {
  using L = Layout<WARPS, NT, STAGES, BT>;
  static_assert(OCC * (L::bytes + 1024) <= 233472, "shared memory");
  auto* const kern = k_project<F16, WARPS, NT, STAGES, BT, GL, HOLD, OCC>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), L::bytes);
  if (e != cudaSuccess) return e;
  const auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)(p.K / 2 + p.K / p.group * 2), (cuuint64_t)p.N}, strides[1] = {(cuuint64_t)p.w_stride};
  const cuuint32_t ones[2] = {1, 1}, code_box[2] = {128, 16}, scale_box[2] = {16, 16};
  if (encode(&p.tm_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.w), dims, strides, code_box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      encode(&p.tm_scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.w), dims, strides, scale_box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  // warps over K: a power of two, as many as there are slabs at most, where a batch
  // has a tile for the warps of each (warps without a slab add zeros)
  const int slabs = (p.K + kSlab - 1) / kSlab;
  p.k_warps = 1;
  while (p.k_warps < WARPS && (HOLD ? p.k_warps < slabs : 2 * p.k_warps <= slabs)) p.k_warps *= 2;
  if (p.k_warps < WARPS / BT) p.k_warps = WARPS / BT;
  const int at_once = WARPS / p.k_warps, tiles = (p.N + 15) / 16, parts = (p.T + 8 * NT - 1) / (8 * NT);
  // (no more blocks than run at once)
  const int want = (tiles + at_once - 1) / at_once, most = OCC * p.sms / parts > 0 ? OCC * p.sms / parts : 1;
  return launch_behind(kern, dim3(want < most ? want : most, parts), 32 * WARPS, L::bytes, stream, p);
}

// x in registers where K has a warp for every slab: 8 tokens and 16 with up to 16
// warps, 32 with 8 (128 registers a thread); more tokens take turns, the weights
// then come from the L2 cache.
template <bool F16, int GL>
cudaError_t launch_tokens(ProjectParams& p, cudaStream_t stream) {
  const int slabs = (p.K + kSlab - 1) / kSlab;
  if (p.T <= 8) {
    if (slabs <= 8) return launch<F16, 8, 1, 3, 4, GL, true, 3>(p, stream);
    if (slabs <= 16) return launch<F16, 16, 1, 3, 4, GL, true, 1>(p, stream);
    return launch<F16, 8, 1, 4, 8, GL, false, 2>(p, stream);
  }
  if (slabs <= 8 && p.T > 16) return launch<F16, 8, 4, 4, 4, GL, true, 1>(p, stream);
  if (slabs <= 16) return launch<F16, 16, 2, 3, 4, GL, true, 1>(p, stream);
  return p.T <= 16 ? launch<F16, 8, 2, 4, 4, GL, false, 2>(p, stream) : launch<F16, 8, 4, 4, 4, GL, false, 1>(p, stream);
}

}  // namespace

cudaError_t launch_project(ProjectParams p, cudaStream_t stream) {
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

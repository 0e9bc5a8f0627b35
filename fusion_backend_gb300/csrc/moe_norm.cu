// The norms after one block and before the next, with the block's gate and
// the residual scale between them (moe_ffn_norm_residual).
//
// One pass over the data: a row's res and y are read once into registers, y's
// mean square is reduced, r' formed, its mean square reduced, and res_out and
// normed are written.  Two reductions a row are the only synchronisation; the
// kernel is bound by HBM for many rows and by the latency of load, reduction,
// reduction, store for a few, so everything a row needs is loaded at the start.
// A row has a warp (H <= 512, four rows a block) or a block of H / 8 or H / 16
// threads; past H = 8192 a thread holds 16 or 32 columns of r' and reads y twice
// (the second time from cache) instead of holding it, to stay within the
// registers of a block of 1024 threads.
// The first form (256 threads and three passes over the row, element by
// element) ran 57 us on 4096 x 2048 fp32 rows.
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kRowsPerBlock = 4;  // rows of a block whose rows have a warp each
constexpr int kWarpRows = 32 * kRowsPerBlock;  // threads of such a block, and of no other

// Columns of the thread: VEC: eight neighbours a group, 16-byte accesses;
// otherwise (rows or H that rule those out) neighbours on neighbouring threads.
// Groups past the row hold zeros.
template <bool VEC>
struct Columns {
  int tid, threads, H;
  MOE_DEV int at(int j, int e) const { return VEC ? 8 * (tid + threads * j) + e : threads * (8 * j + e) + tid; }
  MOE_DEV void load(const void* p, int dtype, size_t base, int j, float* v) const {
    if (VEC) {
      if (at(j, 0) < H) {
        elem_load8(p, dtype, base + at(j, 0), v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = at(j, e) < H ? elem_load(p, dtype, base + at(j, e)) : 0.f;
    }
  }
  MOE_DEV void store(void* p, int dtype, size_t base, int j, const float* v) const {
    if (VEC) {
      if (at(j, 0) < H) elem_store8(p, dtype, base + at(j, 0), v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at(j, e) < H) elem_store(p, dtype, base + at(j, e), v[e]);
    }
  }
};

// Sum over the row's threads, the same on each: a warp's butterfly, then (a
// block a row) the warps' sums in shared memory.
template <int THREADS, bool WARP>
MOE_DEV float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (WARP) return v;
  constexpr int W = THREADS / 32;  // warps at most
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int w = lane & (W - 1);
  v = w < (int)(blockDim.x >> 5) ? red[w] : 0.f;
#pragma unroll
  for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// THREADS: the most that a block has.  ALL: the weights and the gate too are
// loaded at the start.
template <int NV, bool VEC, int THREADS, bool ALL>
__global__ void __launch_bounds__(THREADS) k_norm(const __grid_constant__ NormParams P) {
  constexpr bool WARP = THREADS == kWarpRows;
  constexpr bool AGAIN = NV * THREADS > 1024;  // y is read a second time
  __shared__ float red[2][32];
  const size_t t = WARP ? (size_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5) : blockIdx.x;
  Columns<VEC> cols;
  cols.tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  cols.threads = WARP ? 32 : blockDim.x;
  cols.H = P.H;
  pdl_wait();
  pdl_launch_dependents();
  if (WARP && t >= (size_t)P.T) return;

  const bool per_column = P.gate && P.gate_layout != 1;
  float r[NV][8], y[NV][8], g[ALL ? NV : 1][8], wp[ALL ? NV : 1][8], wn[ALL ? NV : 1][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) cols.load(P.res, P.r_dtype, t * P.r_stride, j, r[j]);
  if (P.y) {
#pragma unroll
    for (int j = 0; j < NV; ++j) cols.load(P.y, P.y_dtype, t * P.y_stride, j, y[j]);
  }
  const size_t g_row = P.gate_layout == 2 ? t * P.g_stride : 0;
  if (ALL) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (per_column) cols.load(P.gate, P.g_dtype, g_row, j, g[j]);
      if (P.w_post) cols.load(P.w_post, P.wpost_dtype, 0, j, wp[j]);
      if (P.w_pre) cols.load(P.w_pre, P.wpre_dtype, 0, j, wn[j]);
    }
  }

  if (P.y) {
    float scale = P.beta;
    if (P.gate && !per_column) {
      const float v = elem_load(P.gate, P.g_dtype, t * P.g_stride);
      scale *= P.gate_sigmoid ? 1.f / (1.f + expf(-v)) : v;
    }
    if (P.post_norm) {
      float q = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(y[j][e], y[j][e], q);
      scale *= 1.f / sqrtf(row_sum<THREADS, WARP>(q, red[0]) / (float)P.H + P.eps);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (AGAIN) cols.load(P.y, P.y_dtype, t * P.y_stride, j, y[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[j][e] *= scale;
      if (P.post_norm && P.w_post) {
        float* w = wp[ALL ? j : 0];
        if (!ALL) cols.load(P.w_post, P.wpost_dtype, 0, j, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[j][e] *= P.w_offset + w[e];
      }
      if (per_column) {
        float* v = g[ALL ? j : 0];
        if (!ALL) cols.load(P.gate, P.g_dtype, g_row, j, v);
        if (P.gate_sigmoid) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = 1.f / (1.f + expf(-v[e]));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) y[j][e] *= v[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] = fmaf(P.alpha, r[j][e], y[j][e]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] *= P.alpha;
  }
  if (P.res_out) {
#pragma unroll
    for (int j = 0; j < NV; ++j) cols.store(P.res_out, P.r_dtype, t * P.ro_stride, j, r[j]);
  }
  if (!P.normed) return;
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    // columns past the row hold 0 times factors that may be infinite: they do
    // not enter the sum
    if (VEC && cols.at(j, 0) >= P.H) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (VEC || cols.at(j, e) < P.H) q = fmaf(r[j][e], r[j][e], q);
  }
  const float inv = 1.f / sqrtf(row_sum<THREADS, WARP>(q, red[1]) / (float)P.H + P.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r[j][e] *= inv;
    if (P.w_pre) {
      float* w = wn[ALL ? j : 0];
      if (!ALL) cols.load(P.w_pre, P.wpre_dtype, 0, j, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] *= P.w_offset + w[e];
    }
    cols.store(P.normed, P.n_dtype, t * P.n_stride, j, r[j]);
  }
}

// Rows of p start on 16-byte boundaries (an absent tensor always does).
bool rows16(const void* p, int dtype, long long stride, int T) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (T == 1 || stride * elem_bytes(dtype) % 16 == 0));
}

template <int NV, int THREADS, bool ALL>
cudaError_t launch(const NormParams& p, bool vec, cudaStream_t stream) {
  constexpr bool WARP = THREADS == kWarpRows;
  const dim3 grid(WARP ? (p.T + kRowsPerBlock - 1) / kRowsPerBlock : p.T);
  const int threads = WARP ? THREADS : (p.H + 256 * NV - 1) / (256 * NV) * 32;
  return vec ? launch_behind(k_norm<NV, true, THREADS, ALL>, grid, threads, 0, stream, p)
             : launch_behind(k_norm<NV, false, THREADS, ALL>, grid, threads, 0, stream, p);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
  const bool vec = p.H % 8 == 0 && rows16(p.res, p.r_dtype, p.r_stride, p.T) &&
                   rows16(p.res_out, p.r_dtype, p.ro_stride, p.T) && rows16(p.y, p.y_dtype, p.y_stride, p.T) &&
                   rows16(p.normed, p.n_dtype, p.n_stride, p.T) && rows16(p.w_post, p.wpost_dtype, 0, 1) &&
                   rows16(p.w_pre, p.wpre_dtype, 0, 1) &&
                   (p.gate_layout == 1 || rows16(p.gate, p.g_dtype, p.gate_layout ? p.g_stride : 0, p.T));
  if (p.H <= 256) return launch<1, kWarpRows, true>(p, vec, stream);
  if (p.H <= 512) return launch<2, kWarpRows, false>(p, vec, stream);
  // few rows: the latency of one row counts, a thread has 8 columns and loads
  // all it needs at once; many: 16 columns a thread, fewer instructions a row
  const bool few = p.T <= 2 * 152;
  if (p.H <= 2048 && few) return launch<1, 256, true>(p, vec, stream);
  if (p.H <= 8192 && few) return launch<1, 1024, true>(p, vec, stream);
  if (p.H <= 4096) return launch<2, 256, false>(p, vec, stream);
  if (p.H <= 8192) return launch<2, 512, false>(p, vec, stream);
  if (p.H <= 16384) return launch<2, 1024, false>(p, vec, stream);
  return launch<4, 1024, false>(p, vec, stream);
}

}  // namespace moe

// The norms after one block and before the next, with the block's gate and
// the residual scale between them (moe_ffn_norm_residual).
//
// One pass over the data: a row's res and y are read once into registers, y's
// mean square is reduced, r' formed, its mean square reduced, and res_out and
// normed are written.  Two reductions a row are the only synchronisation; the
// kernel is bound by HBM for many rows and by the latency of load, reduction,
// reduction, store for a few, so everything a row needs is loaded at the start.
// A row has a warp (H <= 512, four rows a block) or a block of H / 8 threads;
// from H = 8192 on a thread holds 16 or 32 columns of r' and reads y twice (the
// second time from cache) instead of holding it, to stay within the registers
// of a block of 1024 threads.
// The first form (256 threads and three passes over the row, element by
// element) ran 57 us on 4096 x 2048 fp32 rows.
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kRowsPerBlock = 4;  // rows of a block whose rows have a warp each

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
template <bool WARP>
MOE_DEV float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (WARP) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < (int)(blockDim.x >> 5) ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int NV, bool VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kRowsPerBlock : 1024) k_norm(const __grid_constant__ NormParams P) {
  constexpr bool ALL = NV == 1;  // everything a row needs is in registers from the start
  __shared__ float red[2][32];
  const size_t t = WARP ? (size_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5) : blockIdx.x;
  Columns<VEC> cols;
  cols.tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  cols.threads = WARP ? 32 : blockDim.x;
  cols.H = P.H;
  pdl_wait();
  pdl_launch_dependents();
  if (WARP && t >= (size_t)P.T) return;

  const bool channel = P.gate && P.gate_layout == 0, full = P.gate && P.gate_layout == 2;
  float r[NV][8], y[NV][8], g[8], wp[8], wn[8];
#pragma unroll
  for (int j = 0; j < NV; ++j) cols.load(P.res, P.r_dtype, t * P.r_stride, j, r[j]);
  if (P.y) {
#pragma unroll
    for (int j = 0; j < NV; ++j) cols.load(P.y, P.y_dtype, t * P.y_stride, j, y[j]);
  }
  auto load_gate = [&](int j) {
    if (channel) cols.load(P.gate, P.g_dtype, 0, j, g);
    if (full) cols.load(P.gate, P.g_dtype, t * P.g_stride, j, g);
  };
  auto load_post = [&](int j) {
    if (P.w_post) cols.load(P.w_post, P.wpost_dtype, 0, j, wp);
  };
  auto load_pre = [&](int j) {
    if (P.w_pre) cols.load(P.w_pre, P.wpre_dtype, 0, j, wn);
  };
  if (ALL) {
    load_gate(0);
    load_post(0);
    load_pre(0);
  }
  auto activate = [&](float v) { return P.gate_sigmoid ? 1.f / (1.f + expf(-v)) : v; };
  float token_gate = 1.f;
  if (P.gate && P.gate_layout == 1) token_gate = activate(elem_load(P.gate, P.g_dtype, t * P.g_stride));

  if (P.y) {
    float inv = 1.f;
    if (P.post_norm) {
      float q = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(y[j][e], y[j][e], q);
      inv = 1.f / sqrtf(row_sum<WARP>(q, red[0]) / (float)P.H + P.eps);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!ALL) {
        cols.load(P.y, P.y_dtype, t * P.y_stride, j, y[j]);
        load_gate(j);
        load_post(j);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float z = y[j][e] * inv;
        if (P.post_norm && P.w_post) z *= P.w_offset + wp[e];
        z *= channel || full ? activate(g[e]) : token_gate;
        r[j][e] = fmaf(P.beta, z, P.alpha * r[j][e]);
      }
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
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // columns past the row: a gate or a weight of 0 times an infinite factor
      // must not reach the sum
      if (cols.at(j, e) < P.H) q = fmaf(r[j][e], r[j][e], q);
    }
  const float inv = 1.f / sqrtf(row_sum<WARP>(q, red[1]) / (float)P.H + P.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!ALL) load_pre(j);
#pragma unroll
    for (int e = 0; e < 8; ++e) r[j][e] *= P.w_pre ? inv * (P.w_offset + wn[e]) : inv;
    cols.store(P.normed, P.n_dtype, t * P.n_stride, j, r[j]);
  }
}

// Rows of p start on 16-byte boundaries (an absent tensor always does).
bool rows16(const void* p, int dtype, long long stride, int T) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (T == 1 || stride * elem_bytes(dtype) % 16 == 0));
}

template <int NV, bool WARP>
cudaError_t launch(const NormParams& p, bool vec, int threads, cudaStream_t stream) {
  const dim3 grid(WARP ? (p.T + kRowsPerBlock - 1) / kRowsPerBlock : p.T);
  return vec ? launch_behind(k_norm<NV, true, WARP>, grid, threads, 0, stream, p)
             : launch_behind(k_norm<NV, false, WARP>, grid, threads, 0, stream, p);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
  const bool vec = p.H % 8 == 0 && rows16(p.res, p.r_dtype, p.r_stride, p.T) &&
                   rows16(p.res_out, p.r_dtype, p.ro_stride, p.T) && rows16(p.y, p.y_dtype, p.y_stride, p.T) &&
                   rows16(p.normed, p.n_dtype, p.n_stride, p.T) && rows16(p.w_post, p.wpost_dtype, 0, 1) &&
                   rows16(p.w_pre, p.wpre_dtype, 0, 1) &&
                   (p.gate_layout == 1 || rows16(p.gate, p.g_dtype, p.gate_layout ? p.g_stride : 0, p.T));
  if (p.H <= 256) return launch<1, true>(p, vec, 32 * kRowsPerBlock, stream);
  if (p.H <= 512) return launch<2, true>(p, vec, 32 * kRowsPerBlock, stream);
  const int warps = (p.H + 255) / 256;
  if (warps <= 32) return launch<1, false>(p, vec, 32 * warps, stream);
  if (warps <= 64) return launch<2, false>(p, vec, 32 * ((warps + 1) / 2), stream);
  return launch<4, false>(p, vec, 32 * ((warps + 3) / 4), stream);
}

}  // namespace moe

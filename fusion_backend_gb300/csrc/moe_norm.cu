// The norms after one block and before the next, with the block's gate and
// the residual scale between them (moe_ffn_norm_residual).
//
// One pass over the data: a row's res and y are read once into registers, y's
// mean square is reduced, r' formed, its mean square reduced, and res_out and
// normed are written.  The work is bound by HBM for many rows and by the latency
// of load, reduction, reduction, store for a few.
//   k_norm       a warp a row (H <= 512, four rows a block) or a block a row,
//                everything a row needs asked for at the start.  A call of few
//                rows, and rows past 8192 columns (16 or 32 of them a thread).
//   k_norm_rows  as many blocks as fit on the GPU, each going through its rows
//                with the next two on their way into shared memory
//                (asynchronous copies) while it works on one; the weights stay
//                in registers.  With a block a row the loads of a block stand
//                still while it reduces and stores.  4096 x 2048 rows, against a
//                block a row: fp32 with a gate a column 23.6 us (5.0 TB/s, where
//                the copy rate allows 17) and 23.7, bf16 17.1 and 18.6; 2048 x 8192
//                bf16 29.6 and 48.4; 1024 x 2048 bf16 9.0 and 6.7.
// The first form (256 threads and three passes over the row, element by
// element) ran 57 us there.
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kRowsPerBlock = 4;  // rows of a block whose rows have a warp each
constexpr int kWarpRows = 32 * kRowsPerBlock;  // threads of such a block, and of no other
constexpr int kStages = 3;        // rows of k_norm_rows in shared memory

// Columns of the thread: in a group of eight, two times four neighbours, so that
// neighbouring lanes cover whole sectors in one access.  VEC: every row allows
// accesses of four elements and H % 4 == 0.  Otherwise each row is looked at by
// itself: one that starts between two such boundaries is read element by element
// (the four accesses hit the same sectors) and written in fours all the same,
// each lane taking the end of its neighbour's columns, so that a sector is not
// written in four parts.  Columns past the row hold zeros.
template <bool VEC>
struct Columns {
  int tid, threads, H;
  MOE_DEV int at(int j, int h) const { return 4 * (tid + threads * (2 * j + h)); }  // of the half h of group j
  // a row of a tensor, and the elements from a four-element boundary to it
  struct Row {
    uint8_t* p;
    int dtype, m;
  };
  MOE_DEV static Row row(const void* p, int dtype, size_t first) {
    Row r;
    r.p = const_cast<uint8_t*>(static_cast<const uint8_t*>(p)) + first * elem_bytes(dtype);
    r.dtype = dtype;
    r.m = VEC ? 0 : (int)(reinterpret_cast<uintptr_t>(r.p) >> (dtype == kF32 ? 2 : 1)) & 3;
    return r;
  }
  MOE_DEV void load(const Row& r, int j, uint4* w) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = at(j, h);
      w[h] = make_uint4(0u, 0u, 0u, 0u);
      if (VEC ? c < H : r.m == 0 && c + 4 <= H) {
        w[h] = raw_load4(r.p, r.dtype, c);
      } else if (!VEC) {
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = c + i < H ? raw_load(r.p, r.dtype, c + i) : 0u;
        w[h] = r.dtype == kF32 ? make_uint4(e[0], e[1], e[2], e[3]) : make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, 0u, 0u);
      }
    }
  }
  MOE_DEV void values(const uint4* w, int dtype, float* v) const {
    raw_values4(w[0], dtype, v);
    raw_values4(w[1], dtype, v + 4);
  }
  // N words of four elements (fp32: 4, 16-bit: 2) from column c, those inside the row
  template <int N>
  MOE_DEV void store4(const Row& r, int c, const uint32_t (&u)[N]) const {
    if (c + 4 <= H) {
      if (N == 4)
        *reinterpret_cast<uint4*>(r.p + 4 * c) = make_uint4(u[0], u[1], u[N - 2], u[N - 1]);
      else
        *reinterpret_cast<uint2*>(r.p + 2 * c) = make_uint2(u[0], u[1]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) store1(r, c + e, u, e);
    }
  }
  template <int N>
  MOE_DEV void store1(const Row& r, int c, const uint32_t (&u)[N], int e) const {
    if (c >= H) return;
    if (N == 4)
      *reinterpret_cast<uint32_t*>(r.p + 4 * c) = u[e & (N - 1)];
    else
      *reinterpret_cast<uint16_t*>(r.p + 2 * c) = static_cast<uint16_t>(u[e >> 1] >> (16 * (e & 1)));
  }
  template <int N>
  MOE_DEV void store_words(const Row& r, int c, const uint32_t (&u)[N]) const {
    const int m = r.m, lane = threadIdx.x & 31;
    if (m == 0) {
      store4(r, c, u);
      return;
    }
    // columns c - m .. c - m + 3: the last m of the lane below, then the lane's;
    // the warp's first 4 - m and last m columns one by one
    uint32_t p[N], o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = __shfl_up_sync(0xffffffffu, u[i], 1);
    if (N == 4) {
      o[0] = m == 1 ? p[N - 1] : m == 2 ? p[N - 2] : p[1];
      o[1] = m == 1 ? u[0] : m == 2 ? p[N - 1] : p[N - 2];
      o[N - 2] = m == 1 ? u[1] : m == 2 ? u[0] : p[N - 1];
      o[N - 1] = m == 1 ? u[N - 2] : m == 2 ? u[1] : u[0];
    } else {
      const uint32_t a = m == 3 ? p[0] : p[1], b = m == 3 ? p[1] : u[0], d = m == 3 ? u[0] : u[1];
      o[0] = m == 2 ? p[1] : __funnelshift_r(a, b, 16);
      o[1] = m == 2 ? u[0] : __funnelshift_r(b, d, 16);
    }
    if (lane > 0) store4(r, c - m, o);
    if (lane == 0 || lane == 31) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((lane == 0) == (e < 4 - m)) store1(r, c + e, u, e);
    }
  }
  // called by whole warps
  MOE_DEV void store(const Row& r, int j, const float* v) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = at(j, h);
      const float* f = v + 4 * h;
      if (VEC) {
        if (c < H) elem_store4(r.p, r.dtype, c, f);
      } else if (r.dtype == kF32) {
        const uint32_t u[4] = {__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
        store_words(r, c, u);
      } else {
        const uint32_t u[2] = {pack2(r.dtype, f[0], f[1]), pack2(r.dtype, f[2], f[3])};
        store_words(r, c, u);
      }
    }
  }
};

MOE_DEV float sigmoid(float v) { return __fdividef(1.f, 1.f + expf(-v)); }

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

// A row from res (r) and y in registers to its stores.  again(j, y): reads y's
// group j a second time (or keeps what is there); post, gate, pre (j, v): the
// group's weights or gate.
template <int NV, bool VEC, int THREADS, bool WARP, typename Again, typename Post, typename Gate, typename Pre>
MOE_DEV void finish_row(const NormParams& P, const Columns<VEC>& cols, size_t t, float (&r)[NV][8], float (&y)[NV][8],
                        float (*red)[32], Again again, Post post, Gate gate, Pre pre) {
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) r[j][e] *= P.alpha;
  if (P.y) {
    float scale = P.beta;
    if (P.gate && P.gate_layout == 1) {
      const float v = elem_load(P.gate, P.g_dtype, t * P.g_stride);
      scale *= P.gate_sigmoid ? sigmoid(v) : v;
    }
    if (P.post_norm) {
      float q = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(y[j][e], y[j][e], q);
      scale *= rsqrtf(row_sum<THREADS, WARP>(q, red[0]) / (float)P.H + P.eps);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      again(j, y[j]);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[j][e] *= scale;
      if (P.post_norm && P.w_post) {
        post(j, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[j][e] *= P.w_offset + v[e];
      }
      if (P.gate && P.gate_layout != 1) {
        gate(j, v);
        if (P.gate_sigmoid) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = sigmoid(v[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) y[j][e] *= v[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] += y[j][e];
    }
  }
  if (P.res_out) {
#pragma unroll
    for (int j = 0; j < NV; ++j) cols.store(cols.row(P.res_out, P.r_dtype, t * P.ro_stride), j, r[j]);
  }
  if (P.normed) {
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      // columns past the row hold 0 times factors that may be infinite: they do
      // not enter the sum
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (cols.at(j, e >> 2) + (VEC ? 0 : e & 3) < P.H) q = fmaf(r[j][e], r[j][e], q);
    }
    const float inv = rsqrtf(row_sum<THREADS, WARP>(q, red[1]) / (float)P.H + P.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] *= inv;
      if (P.w_pre) {
        float v[8];
        pre(j, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[j][e] *= P.w_offset + v[e];
      }
      cols.store(cols.row(P.normed, P.n_dtype, t * P.n_stride), j, r[j]);
    }
  }
}

// THREADS: the most that a block has.
template <int NV, bool VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) k_norm(const __grid_constant__ NormParams P) {
  constexpr bool WARP = THREADS == kWarpRows;
  constexpr bool ALL = NV == 1;  // the weights and the gate too are asked for at the start
  constexpr bool AGAIN = NV * THREADS > 1024;  // y is read a second time
  __shared__ float red[2][32];
  const size_t t = WARP ? (size_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5) : blockIdx.x;
  Columns<VEC> cols;
  cols.tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  cols.threads = WARP ? 32 : blockDim.x;
  cols.H = P.H;
  pdl_wait();
  if (WARP && t >= (size_t)P.T) return;  // (whole warps)

  uint4 rw[NV][2], yw[NV][2], gw[2], pw[2], nw[2];
#pragma unroll
  for (int j = 0; j < NV; ++j) cols.load(cols.row(P.res, P.r_dtype, t * P.r_stride), j, rw[j]);
  if (P.y) {
#pragma unroll
    for (int j = 0; j < NV; ++j) cols.load(cols.row(P.y, P.y_dtype, t * P.y_stride), j, yw[j]);
  }
  const size_t g_row = P.gate_layout == 2 ? t * P.g_stride : 0;
  auto load_gate = [&](int j) { cols.load(cols.row(P.gate, P.g_dtype, g_row), j, gw); };
  auto load_post = [&](int j) { cols.load(cols.row(P.w_post, P.wpost_dtype, 0), j, pw); };
  auto load_pre = [&](int j) { cols.load(cols.row(P.w_pre, P.wpre_dtype, 0), j, nw); };
  if (ALL) {
    if (P.gate && P.gate_layout != 1) load_gate(0);
    if (P.w_post) load_post(0);
    if (P.w_pre) load_pre(0);
  }
  float r[NV][8], y[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) cols.values(rw[j], P.r_dtype, r[j]);
  if (P.y) {
#pragma unroll
    for (int j = 0; j < NV; ++j) cols.values(yw[j], P.y_dtype, y[j]);
  }
  finish_row<NV, VEC, THREADS, WARP>(
      P, cols, t, r, y, red,
      [&](int j, float* v) {
        if (!AGAIN) return;
        cols.load(cols.row(P.y, P.y_dtype, t * P.y_stride), j, yw[j]);
        cols.values(yw[j], P.y_dtype, v);
      },
      [&](int j, float* v) {
        if (!ALL) load_post(j);
        cols.values(pw, P.wpost_dtype, v);
      },
      [&](int j, float* v) {
        if (!ALL) load_gate(j);
        cols.values(gw, P.g_dtype, v);
      },
      [&](int j, float* v) {
        if (!ALL) load_pre(j);
        cols.values(nw, P.wpre_dtype, v);
      });
}

// Two floats in one instruction (fma.rn.f32x2 and its kin): the arithmetic of
// k_norm_rows, whose rows are otherwise bound by the instructions they issue.
struct F2 {
  unsigned long long v;
};
MOE_DEV F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
MOE_DEV F2 f2(float a) { return f2(a, a); }
MOE_DEV void f2_get(F2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
MOE_DEV F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
MOE_DEV F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// One tensor's rows on their way through shared memory: a thread copies and
// reads its own groups of four columns ([group][thread]), so no thread waits for
// another.  F32: fp32 elements, otherwise 16-bit ones (dtype).
template <bool F32>
struct Stream {
  static constexpr int kSize = F32 ? 4 : 2;
  const uint8_t* next;  // the thread's first column of the row to copy next; null: absent
  int dtype;
  size_t stride;  // bytes from a row of the block to its next
  MOE_DEV void init(const void* base, int dt, long long row_stride) {
    dtype = dt;
    stride = (size_t)(row_stride * kSize) * gridDim.x;
    next = base ? static_cast<const uint8_t*>(base) + ((size_t)blockIdx.x * row_stride + 4 * threadIdx.x) * kSize : nullptr;
  }
  // place: the thread's first group in the tensor's part of the stage
  template <int NV>
  MOE_DEV void fetch(uint32_t place, const bool (&in)[NV]) {
    if (!next) return;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = j * (int)blockDim.x * 4 * kSize;
      if (!in[j]) continue;
      if (F32)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(place + at), "l"(next + at) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(place + at), "l"(next + at) : "memory");
    }
    next += stride;
  }
  MOE_DEV void read(const uint8_t* place, int j, F2* v) const {
    place += j * (int)blockDim.x * 4 * kSize;
    if (F32) {
      const float4 f = *reinterpret_cast<const float4*>(place);
      v[0] = f2(f.x, f.y);
      v[1] = f2(f.z, f.w);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(place);
      float f[4];
      raw_values4(make_uint4(w.x, w.y, 0u, 0u), dtype, f);
      v[0] = f2(f[0], f[1]);
      v[1] = f2(f[2], f[3]);
    }
  }
};

// NV groups of four columns a thread, accesses of four elements throughout.
// R32, Y32, N32: res, y (and a gate of every element), normed are fp32.
template <int NV, int THREADS, bool R32, bool Y32, bool N32>
__global__ void __launch_bounds__(THREADS) k_norm_rows(const __grid_constant__ NormParams P) {
  __shared__ float red[2][2][32];  // by the row's parity: a row may have one reduction alone, hence one barrier
  extern __shared__ __align__(16) uint8_t stages[];  // [kStages][res | y | gate]
  const int tid = threadIdx.x, threads = blockDim.x;
  const bool per_row = P.gate && P.gate_layout == 2;
  constexpr int RB = R32 ? 4 : 2, YB = Y32 ? 4 : 2;
  Stream<R32> sr;
  Stream<Y32> sy, sg;
  sr.init(P.res, P.r_dtype, P.r_stride);
  sy.init(P.y, P.y_dtype, P.y_stride);
  sg.init(per_row ? P.gate : nullptr, P.g_dtype, P.g_stride);
  const int r_bytes = NV * 4 * threads * RB, y_bytes = P.y ? NV * 4 * threads * YB : 0;
  const int bytes = r_bytes + y_bytes + (per_row ? y_bytes : 0);
  bool in[NV];  // the group is inside the row
#pragma unroll
  for (int j = 0; j < NV; ++j) in[j] = 4 * (tid + threads * j) < P.H;
  auto fetch = [&](int t, int s) {
    if (t < P.T) {
      const uint32_t place = smem_u32(stages) + s * bytes;
      sr.fetch(place + 4 * RB * tid, in);
      sy.fetch(place + r_bytes + 4 * YB * tid, in);
      sg.fetch(place + r_bytes + y_bytes + 4 * YB * tid, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  pdl_wait();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(blockIdx.x + s * gridDim.x, s);
  // what a column of y and of r' is multiplied by in every row: w_offset +
  // w_post and a gate per column as one factor, w_offset + w_pre
  F2 wy[NV][2], wn[NV][2];
  const bool by_column = (P.post_norm && P.w_post) || (P.gate && P.gate_layout == 0);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float post[4], pre[4], g[4];
    const size_t c = 4 * (tid + threads * j);
#pragma unroll
    for (int e = 0; e < 4; ++e) post[e] = pre[e] = 1.f;
    if (in[j]) {
      if (P.post_norm && P.w_post) {
        raw_values4(raw_load4(P.w_post, P.wpost_dtype, c), P.wpost_dtype, post);
#pragma unroll
        for (int e = 0; e < 4; ++e) post[e] += P.w_offset;
      }
      if (P.gate && P.gate_layout == 0) {
        raw_values4(raw_load4(P.gate, P.g_dtype, c), P.g_dtype, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) post[e] *= P.gate_sigmoid ? sigmoid(g[e]) : g[e];
      }
      if (P.w_pre) {
        raw_values4(raw_load4(P.w_pre, P.wpre_dtype, c), P.wpre_dtype, pre);
#pragma unroll
        for (int e = 0; e < 4; ++e) pre[e] += P.w_offset;
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      wy[j][e] = f2(post[2 * e], post[2 * e + 1]);
      wn[j][e] = f2(pre[2 * e], pre[2 * e + 1]);
    }
  }
  const float per_column = 1.f / (float)P.H;
  const F2 alpha = f2(P.alpha);
  auto square = [&](const F2 (&v)[NV][2]) {
    F2 q = f2(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (in[j]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) q = f2_fma(v[j][e], v[j][e], q);
      }
    float a, b;
    f2_get(q, a, b);
    return a + b;
  };
  // the thread's first column of a row of an output, the block's rows apart
  auto store = [&](uint8_t* row, bool f32, int dtype, const F2 (&v)[NV][2]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!in[j]) continue;
      float f[4];
      f2_get(v[j][0], f[0], f[1]);
      f2_get(v[j][1], f[2], f[3]);
      if (f32)
        *reinterpret_cast<float4*>(row + 16 * threads * j) = make_float4(f[0], f[1], f[2], f[3]);
      else
        *reinterpret_cast<uint2*>(row + 8 * threads * j) = make_uint2(pack2(dtype, f[0], f[1]), pack2(dtype, f[2], f[3]));
    }
  };
  constexpr int NB = N32 ? 4 : 2;
  uint8_t* ro = static_cast<uint8_t*>(P.res_out) + ((size_t)blockIdx.x * P.ro_stride + 4 * tid) * RB;
  uint8_t* no = static_cast<uint8_t*>(P.normed) + ((size_t)blockIdx.x * P.n_stride + 4 * tid) * NB;
  const size_t ro_step = (size_t)P.ro_stride * RB * gridDim.x, no_step = (size_t)P.n_stride * NB * gridDim.x;
  int s = 0, odd = 0;
  for (int t = blockIdx.x; t < P.T; t += gridDim.x, ro += ro_step, no += no_step) {
    // into the stage of the row before, which the thread has read
    fetch(t + (kStages - 1) * gridDim.x, s == 0 ? kStages - 1 : s - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    const uint8_t* place = stages + s * bytes;
    F2 r[NV][2];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      sr.read(place + 4 * RB * tid, j, r[j]);
#pragma unroll
      for (int e = 0; e < 2; ++e) r[j][e] = f2_mul(r[j][e], alpha);
    }
    if (P.y) {
      F2 y[NV][2];
#pragma unroll
      for (int j = 0; j < NV; ++j) sy.read(place + r_bytes + 4 * YB * tid, j, y[j]);
      float scale = P.beta;
      if (P.gate && P.gate_layout == 1) {
        const float v = elem_load(P.gate, P.g_dtype, (size_t)t * P.g_stride);
        scale *= P.gate_sigmoid ? sigmoid(v) : v;
      }
      if (P.post_norm) scale *= rsqrtf(row_sum<THREADS, false>(square(y), red[odd][0]) * per_column + P.eps);
      const F2 f = f2(scale);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (by_column) {
#pragma unroll
          for (int e = 0; e < 2; ++e) y[j][e] = f2_mul(y[j][e], wy[j][e]);
        }
        if (per_row) {
          F2 g[2];
          sg.read(place + r_bytes + y_bytes + 4 * YB * tid, j, g);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (P.gate_sigmoid) {
              float a, b;
              f2_get(g[e], a, b);
              g[e] = f2(sigmoid(a), sigmoid(b));
            }
            y[j][e] = f2_mul(y[j][e], g[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) r[j][e] = f2_fma(y[j][e], f, r[j][e]);
      }
    }
    if (P.res_out) store(ro, R32, P.r_dtype, r);
    if (P.normed) {
      const F2 inv = f2(rsqrtf(row_sum<THREADS, false>(square(r), red[odd][1]) * per_column + P.eps));
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) r[j][e] = f2_mul(f2_mul(r[j][e], inv), wn[j][e]);
      store(no, N32, P.n_dtype, r);
    }
    s = s + 1 == kStages ? 0 : s + 1;
    odd ^= 1;
  }
}

// Rows of p allow accesses of four elements (an absent tensor always does).
bool rows4(const void* p, int dtype, long long stride, int T) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (4 * elem_bytes(dtype)) == 0 && (T == 1 || stride % 4 == 0));
}

template <int NV, int THREADS>
cudaError_t launch(const NormParams& p, bool vec, cudaStream_t stream) {
  constexpr bool WARP = THREADS == kWarpRows;
  const dim3 grid(WARP ? 1 + (p.T - 1) / kRowsPerBlock : p.T);
  const int threads = WARP ? THREADS : (p.H + 256 * NV - 1) / (256 * NV) * 32;
  return vec ? launch_behind(k_norm<NV, true, THREADS>, grid, threads, 0, stream, p)
             : launch_behind(k_norm<NV, false, THREADS>, grid, threads, 0, stream, p);
}

// Bytes of shared memory that a row and the two behind it take.
int rows_smem(const NormParams& p, int nv) {
  const int each = elem_bytes(p.r_dtype) + (p.y ? elem_bytes(p.y_dtype) : 0) +
                   (p.gate && p.gate_layout == 2 ? elem_bytes(p.g_dtype) : 0);
  return kStages * ((p.H + 128 * nv - 1) / (128 * nv) * 32) * 4 * nv * each;
}

// As many blocks as are resident at once.
template <int NV, int THREADS, bool R32, bool Y32, bool N32>
cudaError_t launch_rows_of(const NormParams& p, cudaStream_t stream) {
  const int threads = (p.H + 128 * NV - 1) / (128 * NV) * 32;
  const int smem = rows_smem(p, NV);
  auto* const kern = k_norm_rows<NV, THREADS, R32, Y32, N32>;
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), smem);
  int per_sm = 0;
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
  if (e != cudaSuccess) return e;
  const int blocks = p.sms * (per_sm > 0 ? per_sm : 1);
  return launch_behind(kern, dim3(p.T < blocks ? p.T : blocks), threads, smem, stream, p);
}

template <int NV, int THREADS>
cudaError_t launch_rows(const NormParams& p, cudaStream_t stream) {
  const bool r32 = p.r_dtype == kF32, y32 = p.y && p.y_dtype == kF32, n32 = p.n_dtype == kF32;
  if (r32)
    return y32 ? n32 ? launch_rows_of<NV, THREADS, true, true, true>(p, stream)
                     : launch_rows_of<NV, THREADS, true, true, false>(p, stream)
               : n32 ? launch_rows_of<NV, THREADS, true, false, true>(p, stream)
                     : launch_rows_of<NV, THREADS, true, false, false>(p, stream);
  return y32 ? n32 ? launch_rows_of<NV, THREADS, false, true, true>(p, stream)
                   : launch_rows_of<NV, THREADS, false, true, false>(p, stream)
             : n32 ? launch_rows_of<NV, THREADS, false, false, true>(p, stream)
                   : launch_rows_of<NV, THREADS, false, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
  const bool vec = p.H % 4 == 0 && rows4(p.res, p.r_dtype, p.r_stride, p.T) &&
                   rows4(p.res_out, p.r_dtype, p.ro_stride, p.T) && rows4(p.y, p.y_dtype, p.y_stride, p.T) &&
                   rows4(p.normed, p.n_dtype, p.n_stride, p.T) && rows4(p.w_post, p.wpost_dtype, 0, 1) &&
                   rows4(p.w_pre, p.wpre_dtype, 0, 1) &&
                   (p.gate_layout == 1 || rows4(p.gate, p.g_dtype, p.gate_layout ? p.g_stride : 0, p.T));
  if (p.H <= 256) return launch<1, kWarpRows>(p, vec, stream);
  if (p.H <= 512) return launch<2, kWarpRows>(p, vec, stream);
  if (p.H > 16384) return launch<4, 1024>(p, vec, stream);
  if (p.H > 8192) return launch<2, 1024>(p, vec, stream);
  // (the streaming kernel takes a gate of every element in y's size, and three
  // rows in shared memory)
  const bool fits = (!p.gate || p.gate_layout != 2 || (p.g_dtype == kF32) == (p.y_dtype == kF32)) &&
                    rows_smem(p, 4) <= 220 * 1024;
  if (vec && fits && p.T > 4 * p.sms) {
    if (p.H <= 2048) return launch_rows<4, 128>(p, stream);
    if (p.H <= 4096) return launch_rows<4, 256>(p, stream);
    return launch_rows<4, 512>(p, stream);
  }
  // few rows (each has a block of its own at once), or rows of any alignment
  if (p.T > 4 * p.sms && p.H <= 4096) return launch<2, 256>(p, vec, stream);
  return p.H <= 2048 ? launch<1, 256>(p, vec, stream) : launch<1, 1024>(p, vec, stream);
}

}  // namespace moe

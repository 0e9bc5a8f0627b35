// Routing from router logits: scores, group-limited choice with a balance
// bias, weights (moe_ffn_route).
//
// One warp a token.  The experts are owned in index order: each group of
// E / G neighbours has LPG = 32 / (G rounded up to a power of two) lanes, each
// with EPL or fewer consecutive experts, so a lower lane (then a lower slot)
// is a lower index and a group's value is a reduction over its lanes.
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr float kFltMax = 3.402823466e38f;

MOE_DEV double warp_max(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
MOE_DEV double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// (c, l, e) before (c2, l2, e2) in the order of the choice
MOE_DEV bool before(double c, float l, int e, double c2, float l2, int e2) {
  return c > c2 || (c == c2 && (l > l2 || (l == l2 && e < e2)));
}

template <int EPL>
__global__ void __launch_bounds__(128) k_route(const __grid_constant__ RouteParams P) {
  const int lane = threadIdx.x & 31, t = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t >= P.T) return;
  int lpg = 32;
  for (int g = 1; g < P.G; g <<= 1) lpg >>= 1;
  const int per = (P.gs + lpg - 1) / lpg;  // experts a lane, <= EPL
  const int grp = lane / lpg, first = (lane % lpg) * per;
  const int n = grp < P.G ? max(0, min(per, P.gs - first)) : 0;
  const int e0 = grp * P.gs + first;

  float l[EPL];
  double c[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    float v = -INFINITY;
    if (i < n) v = elem_load(P.logits, P.dtype, (size_t)t * P.stride + e0 + i);
    l[i] = v != v ? -INFINITY : fminf(v, kFltMax);
  }
  // c: -inf where the expert cannot be chosen
  double m = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) m = fmax(m, (double)l[i]);
  m = warp_max(m);
  double z = 0.0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    c[i] = 0.0;
    if (l[i] != -INFINITY) c[i] = P.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - m);
    z += c[i];
  }
  z = warp_sum(z);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (!P.sigmoid && z > 0.0) c[i] /= z;
    float b = P.bias && i < n ? P.bias[e0 + i] : 0.f;
    b = b != b ? -INFINITY : fminf(b, kFltMax);
    c[i] = l[i] == -INFINITY || b == -INFINITY ? -INFINITY : c[i] + (double)b;
  }
  // groups: value of the lane's group on each of its lanes
  if (P.G > 1) {
    double a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      a2 = fmax(a2, fmin(a1, c[i]));
      a1 = fmax(a1, c[i]);
    }
    for (int o = lpg >> 1; o; o >>= 1) {
      const double b1 = __shfl_xor_sync(0xffffffffu, a1, o), b2 = __shfl_xor_sync(0xffffffffu, a2, o);
      a2 = fmax(fmax(a2, b2), fmin(a1, b1));
      a1 = fmax(a1, b1);
    }
    const double val = P.top2 && a2 != -INFINITY ? a1 + a2 : a1;
    int rank = 0;  // groups before this one
    for (int g = 0; g < P.G; ++g) {
      const double o = __shfl_sync(0xffffffffu, val, g * lpg);
      rank += o > val || (o == val && g < grp);
    }
    if (rank >= P.top_groups) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = -INFINITY;
    }
  }
  // the choice, one expert a round; lane j keeps the j-th
  int my_id = -1;
  float my_l = -INFINITY;
  for (int j = 0; j < P.K; ++j) {
    double bc = -INFINITY;
    float bl = -INFINITY;
    int be = 1 << 30;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (c[i] != -INFINITY && before(c[i], l[i], e0 + i, bc, bl, be)) {
        bc = c[i];
        bl = l[i];
        be = e0 + i;
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double oc = __shfl_xor_sync(0xffffffffu, bc, o);
      const float ol = __shfl_xor_sync(0xffffffffu, bl, o);
      const int oe = __shfl_xor_sync(0xffffffffu, be, o);
      if (before(oc, ol, oe, bc, bl, be)) {
        bc = oc;
        bl = ol;
        be = oe;
      }
    }
    if (bc == -INFINITY) break;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e0 + i == be && i < n) c[i] = -INFINITY;
    if (lane == j) {
      my_id = be;
      my_l = bl;
    }
  }
  // weights from the chosen logits.  Renormalised, the softmax needs no other
  // logit, and the sigmoid is exp(l) to below fp64's resolution where every
  // chosen logit is far below 0 (the ratio is then formed before it can
  // underflow).
  double v = 0.0;
  const double top = warp_max((double)my_l);
  if (my_id >= 0) {
    if (P.renorm && (!P.sigmoid || top < -60.0))
      v = exp((double)my_l - top);
    else
      v = P.sigmoid ? 1.0 / (1.0 + exp(-(double)my_l)) : exp((double)my_l - m) / z;
  }
  if (P.renorm) {
    const double total = warp_sum(v);
    if (total > 0.0) v /= total;
  }
  if (lane < P.K) {
    P.ids[(size_t)t * P.K + lane] = my_id;
    P.w[(size_t)t * P.K + lane] = (float)(v * (double)P.scale);
  }
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
  int lpg = 32;
  for (int g = 1; g < p.G; g <<= 1) lpg >>= 1;
  const int per = (p.gs + lpg - 1) / lpg;
  const dim3 grid((p.T + 3) / 4);
  if (per <= 4)
    k_route<4><<<grid, 128, 0, stream>>>(p);
  else if (per <= 8)
    k_route<8><<<grid, 128, 0, stream>>>(p);
  else if (per <= 32)
    k_route<32><<<grid, 128, 0, stream>>>(p);
  else
    k_route<64><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe

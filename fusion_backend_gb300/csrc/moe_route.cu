// Routing from router logits: scores, group-limited choice with a balance
// bias, weights (moe_ffn_route).
//
// One warp a token.  The experts are owned in index order: each group of
// E / G neighbours has LPG = 32 / (G rounded up to a power of two) lanes, each
// with EPL or fewer consecutive experts, so a lower lane (then a lower slot)
// is a lower index and a group's value is a reduction over its lanes.
//
// The choice is made on fp32 keys: one warp maximum a round (the hardware's
// reduction over order keys), only the winner's lane looks for its next best.
// Without a bias the key is the logit itself, since the scores rise with it:
// the choice is then exact, and scores are formed only where the groups or the
// weights need them.  With a bias the key is c = s + b in fp32, which is off by
// less than `slack` (below); where two neighbours in the order of the choice
// lie closer than that, the candidates' c are formed and ordered in fp64, one a
// lane, and where the groups on the two sides of the cut do (or more candidates
// than lanes), the warp makes the whole choice again in fp64.  The first is one
// token in some hundreds on logits of a spread of two, the second one in
// thousands; fp64 for every token, the first form of this kernel, ran 176 us on
// 4096 tokens x 256 experts and 536 us on 16381 x 200, and the whole choice in
// fp64 for every near pair still 36 and 48 us (the GPU's fp64 rate is a small
// share of its fp32 rate, and one such token is all that an SM waits for).
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_elem.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kFltMax = 3.402823466e38f;
constexpr int kWarps = 4;

template <typename F>
MOE_DEV F warp_max(F v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <typename F>
MOE_DEV F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
MOE_DEV float key_float(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k); }
// NaN: masked; +inf: the largest number
MOE_DEV float clean(float v) { return v != v ? -INFINITY : fminf(v, kFltMax); }

struct Owned {
  int lpg, grp, n, e0;  // lanes a group, the lane's group, its experts e0 .. e0 + n - 1
};

// From the lane's two largest c the value of its group, on each of the group's
// lanes; -inf where the group has nothing left.
template <typename F>
MOE_DEV F group_value(F a1, F a2, int lpg, bool top2) {
  for (int o = lpg >> 1; o; o >>= 1) {
    const F b1 = __shfl_xor_sync(kAll, a1, o), b2 = __shfl_xor_sync(kAll, a2, o);
    a2 = fmax(fmax(a2, b2), fmin(a1, b1));
    a1 = fmax(a1, b1);
  }
  return top2 && a2 != -INFINITY ? a1 + a2 : a1;
}

// The lane's group's place among the G group values (equal: the lower group).
template <typename F>
MOE_DEV int group_rank(F val, int G, const Owned& o) {
  int rank = 0;
  for (int g = 0; g < G; ++g) {
    const F v = __shfl_sync(kAll, val, g * o.lpg);
    rank += v > val || (v == val && g < o.grp);
  }
  return rank;
}

// c of one expert in fp64.  Not inlined, and the loops around it not unrolled:
// straight-line code that one warp runs once is paid for in instruction fetches
// (the unrolled form held its SM for 30 us).
__device__ __noinline__ double exact_c(bool sigmoid, float l, float b, double m, double z) {
  const double e = exp(sigmoid ? -(double)l : (double)l - m);
  return (sigmoid ? 1.0 / (1.0 + e) : e / z) + (double)b;
}

MOE_DEV float logit(const RouteParams& P, int t, int e) {
  return clean(elem_load(P.logits, P.dtype, (size_t)t * P.stride + e));
}
MOE_DEV float bias_of(const RouteParams& P, int e) { return P.bias ? clean(P.bias[e]) : 0.f; }

// The softmax's largest logit and sum in fp64.
__device__ __noinline__ void exact_sum(const RouteParams& P, int t, const Owned& o, double& m, double& z) {
  float top = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < o.n; ++i) top = fmaxf(top, logit(P, t, o.e0 + i));
  m = warp_max(top);
  z = 0.0;
#pragma unroll 1
  for (int i = 0; i < o.n; ++i) {
    const float l = logit(P, t, o.e0 + i);
    if (l != -INFINITY) z += exp((double)l - m);
  }
  z = warp_sum(z);
}

// The whole choice in fp64: lane j gets the j-th expert and its logit.
template <int EPL>
__device__ __noinline__ void choose_exact(const RouteParams& P, int t, const Owned& o, int& id, float& lj) {
  const int lane = threadIdx.x & 31;
  double m = 0.0, z = 1.0;
  if (!P.sigmoid) exact_sum(P, t, o, m, z);
  // order keys of c (0: cannot be chosen): integer comparisons from here on
  unsigned long long key[EPL];
  double a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < o.n; ++i) {
    const float l = logit(P, t, o.e0 + i), b = bias_of(P, o.e0 + i);
    key[i] = 0ull;
    if (l == -INFINITY || b == -INFINITY) continue;
    const double c = exact_c(P.sigmoid, l, b, m, z);
    a2 = fmax(a2, fmin(a1, c));
    a1 = fmax(a1, c);
    const unsigned long long u = (unsigned long long)__double_as_longlong(c + 0.0);
    key[i] = u >> 63 ? ~u : u | 1ull << 63;
  }
  bool kept = true;
  if (P.G > 1) kept = group_rank(group_value(a1, a2, o.lpg, P.top2), P.G, o) < P.top_groups;
  unsigned long long best = 0ull;
  uint32_t best_l = 0u;
  int at = 0;
  auto local_best = [&]() {
    best = 0ull;
    best_l = 0u;
#pragma unroll 1
    for (int i = 0; kept && i < o.n; ++i) {
      // without a bias the logits decide inside the groups
      const uint32_t k = float_order_key(logit(P, t, o.e0 + i));
      const unsigned long long c = key[i] && !P.bias ? 1ull << 63 : key[i];
      if (c > best || (c == best && c != 0ull && k > best_l)) {
        best = c;
        best_l = k;
        at = i;
      }
    }
  };
  local_best();
  id = -1;
  lj = -INFINITY;
#pragma unroll 1
  for (int j = 0; j < P.K; ++j) {
    // the largest c, then the largest logit, then the lowest lane and slot
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(best >> 32));
    if (hi == 0u) break;
    bool in = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(kAll, in ? (uint32_t)best : 0u);
    in = in && (uint32_t)best == lo;
    const uint32_t lk = __reduce_max_sync(kAll, in ? best_l : 0u);
    const int src = __ffs(__ballot_sync(kAll, in && best_l == lk)) - 1;
    const int e = __shfl_sync(kAll, o.e0 + at, src);
    if (lane == j) {
      id = e;
      lj = key_float(lk);
    }
    if (lane == src) {
      key[at] = 0ull;
      local_best();
    }
  }
}

// The n candidates on lanes 0 .. n - 1 (expert id, logit lj; with a bias), in
// the order of their c in fp64: a lane forms one c, counts the candidates
// before it and the candidates change lanes.
__device__ __noinline__ void settle(const RouteParams& P, int t, const Owned& o, int n, int& id, float& lj) {
  const int lane = threadIdx.x & 31;
  double m = 0.0, z = 1.0, c = -INFINITY;
  if (!P.sigmoid) exact_sum(P, t, o, m, z);
  if (id >= 0) c = exact_c(P.sigmoid, lj, bias_of(P, id), m, z);
  int rank = 0;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const double cj = __shfl_sync(kAll, c, j);
    const float l2 = __shfl_sync(kAll, lj, j);
    const int e2 = __shfl_sync(kAll, id, j);
    rank += cj > c || (cj == c && (l2 > lj || (l2 == lj && e2 < id)));
  }
  int src = lane;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const int from = __ffs(__ballot_sync(kAll, lane < n && rank == j)) - 1;
    if (lane == j) src = from;
  }
  id = __shfl_sync(kAll, id, src);
  lj = __shfl_sync(kAll, lj, src);
}

template <int EPL>
__global__ void __launch_bounds__(32 * kWarps) k_route(const __grid_constant__ RouteParams P) {
  const int lane = threadIdx.x & 31, t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  Owned o;
  o.lpg = P.lpg;
  o.grp = lane / P.lpg;
  const int first = (lane - o.grp * P.lpg) * P.per;
  o.n = o.grp < P.G ? max(0, min(P.per, P.gs - first)) : 0;
  o.e0 = o.grp * P.gs + first;
  pdl_wait();
  pdl_launch_dependents();
  if (t >= P.T) return;

  float l[EPL], b[EPL], c[EPL];
  const size_t row = (size_t)t * P.stride + o.e0;
  if (EPL >= 4 && P.vec) {
#pragma unroll
    for (int i = 0; i + 4 <= EPL; i += 4) {
      l[i] = l[i + 1] = l[i + 2] = l[i + 3] = -INFINITY;
      if (i < o.n) {
        if (P.dtype == kF32) {
          const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(P.logits) + row + i);
          l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(P.logits) + row + i);
          if (P.dtype == kBf16) {
            l[i] = bf16_lo(v.x), l[i + 1] = bf16_hi(v.x), l[i + 2] = bf16_lo(v.y), l[i + 3] = bf16_hi(v.y);
          } else {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
            const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
            l[i] = p.x, l[i + 1] = p.y, l[i + 2] = q.x, l[i + 3] = q.y;
          }
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = i < o.n ? elem_load(P.logits, P.dtype, row + i) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    l[i] = clean(l[i]);
    b[i] = P.bias && i < o.n ? clean(P.bias[o.e0 + i]) : 0.f;
  }
  // c in fp32 (the logit where the choice can go by it), the softmax's sum
  const bool biased = P.bias != nullptr;
  const bool scored = biased || (P.G > 1 && P.top2);   // c holds scores
  float m = 0.f, z = 1.f, smax = 1.f;
  if (!P.sigmoid && (scored || !P.renorm)) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
    m = key_float(__reduce_max_sync(kAll, float_order_key(m)));
    z = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      c[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - m);
      z += c[i];
    }
    z = warp_sum(z);
    smax = 1.f / z;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (!scored)
      c[i] = l[i];
    else if (l[i] == -INFINITY || b[i] == -INFINITY)
      c[i] = -INFINITY;
    else
      c[i] = (P.sigmoid ? __fdividef(1.f, 1.f + expf(-l[i])) : c[i] * smax) + b[i];
  }
  // How far apart two fp32 values of c have to be for their order to be that of
  // fp64.  Sigmoid: exp, sum and quotient are off by less than 2^-21 of s <= 1
  // together.  Softmax: the exponent's argument rounds by |x| 2^-24 (and
  // exp(-|x|) |x| < 1), exp, the sum of EPL terms a lane and 5 levels, the
  // reciprocal and the product: less than 2^-17 of the largest s.  Both sides of
  // a comparison count, and the rounding of s + b: 2^-24 |c| each.
  auto slack = [&](float v) { return smax * (P.sigmoid ? 0x1p-20f : 0x1p-16f) + fabsf(v) * 0x1p-22f + 0x1p-120f; };
  bool unsure = false;
  if (P.G > 1) {
    float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      a2 = fmaxf(a2, fminf(a1, c[i]));
      a1 = fmaxf(a1, c[i]);
    }
    const float val = group_value(a1, a2, P.lpg, P.top2);
    const int rank = group_rank(val, P.G, o);
    if (scored) {
      // the last group kept and the first one left out
      const uint32_t in = __ballot_sync(kAll, o.grp < P.G && rank == P.top_groups - 1);
      const uint32_t out = __ballot_sync(kAll, o.grp < P.G && rank == P.top_groups);
      const float vi = __shfl_sync(kAll, val, __ffs(in) - 1), vo = __shfl_sync(kAll, val, __ffs(out) - 1);
      unsure = vo != -INFINITY && vi - vo <= 2.f * slack(vi);
    }
    if (!scored || biased) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = rank < P.top_groups ? c[i] : -INFINITY;
    } else {  // no bias: the choice inside the groups goes by the logits
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = rank < P.top_groups ? l[i] : -INFINITY;
    }
  }
  // The choice.  Every lane holds the order key of its best expert (0: none).
  uint32_t key[EPL], best = 0u;
  int at = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    key[i] = c[i] == -INFINITY ? 0u : float_order_key(c[i]);
    if (key[i] > best) {
      best = key[i];
      at = i;
    }
  }
  int id = -1;
  float lj = -INFINITY;
  if (!unsure) {
    // With a bias, rounds go on behind the K-th until one is clearly below it
    // (while a lane is free to hold it).
    float c_last = INFINITY, c_cut = INFINITY;
    bool near = false;
    int n = 0;
    for (; n < (biased ? 32 : P.K); ++n) {
      const uint32_t top = __reduce_max_sync(kAll, best);
      if (top == 0u) break;
      const float cj = key_float(top);
      if (n >= P.K && c_cut - cj > slack(c_cut)) break;
      const int src = __ffs(__ballot_sync(kAll, best == top)) - 1;
      const int e = __shfl_sync(kAll, o.e0 + at, src);
      near |= c_last - cj <= slack(cj);
      c_last = cj;
      if (n < P.K) c_cut = cj;
      if (lane == n) {
        id = e;
        lj = cj;
      }
      if (lane == src) {
        best = 0u;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          if (i == at) key[i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (key[i] > best) {
            best = key[i];
            at = i;
          }
      }
    }
    if (biased) {
      // no lane left, and the next one is near the cut
      const uint32_t next = __reduce_max_sync(kAll, best);
      unsure = n == 32 && next != 0u && c_cut - key_float(next) <= slack(c_cut);
      lj = id >= 0 ? logit(P, t, id) : -INFINITY;
      if (near && !unsure) settle(P, t, o, n, id, lj);
      if (lane >= P.K) {
        id = -1;
        lj = -INFINITY;
      }
    }
  }
  if (unsure) choose_exact<EPL>(P, t, o, id, lj);

  // Weights from the chosen logits.  Renormalised, the softmax needs no other
  // logit, and the sigmoid is exp(l) to fp32's resolution where every chosen
  // logit is far below 0 (the ratio is then formed before it can underflow).
  float v = 0.f;
  if (P.renorm) {
    const float top = warp_max(lj);
    if (id >= 0) v = !P.sigmoid || top < -60.f ? expf(lj - top) : 1.f / (1.f + expf(-lj));
    const float total = warp_sum(v);
    if (id >= 0) v = v / total;
  } else if (id >= 0) {
    v = P.sigmoid ? 1.f / (1.f + expf(-lj)) : expf(lj - m) / z;
  }
  if (lane < P.K) {
    P.ids[(size_t)t * P.K + lane] = id;
    P.w[(size_t)t * P.K + lane] = v * P.scale;
  }
}

}  // namespace

cudaError_t launch_route(RouteParams p, cudaStream_t stream) {
  p.lpg = 32;
  for (int g = 1; g < p.G; g <<= 1) p.lpg >>= 1;
  p.per = (p.gs + p.lpg - 1) / p.lpg;
  // four experts a load: rows, groups and lanes start on a load's boundary
  if (p.per > 2) {
    const int per4 = (p.per + 3) & ~3;
    const uintptr_t bytes = p.dtype == kF32 ? 16 : 8;
    p.vec = p.gs % 4 == 0 && p.stride % 4 == 0 && reinterpret_cast<uintptr_t>(p.logits) % bytes == 0;
    if (p.vec) p.per = per4;
  }
  const dim3 grid((p.T + kWarps - 1) / kWarps);
  const int threads = 32 * kWarps;
  if (p.per <= 2) return launch_behind(k_route<2>, grid, threads, 0, stream, p);
  if (p.per <= 4) return launch_behind(k_route<4>, grid, threads, 0, stream, p);
  if (p.per <= 8) return launch_behind(k_route<8>, grid, threads, 0, stream, p);
  if (p.per <= 16) return launch_behind(k_route<16>, grid, threads, 0, stream, p);
  if (p.per <= 32) return launch_behind(k_route<32>, grid, threads, 0, stream, p);
  return launch_behind(k_route<64>, grid, threads, 0, stream, p);
}

}  // namespace moe

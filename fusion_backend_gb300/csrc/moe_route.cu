// Routing from router logits: scores, group-limited choice with a balance
// bias, weights (moe_ffn_route).
//
// One warp a token.  The experts are owned in index order: each group of
// E / G neighbours has LPG = 32 / (G rounded up to a power of two) lanes, each
// with EPL or fewer consecutive experts, so a lower lane (then a lower slot)
// is a lower index and a group's value is a reduction over its lanes.
//
// The choice is made on fp32 values: the K-th largest of the lanes' largest
// bounds the candidates (K or somewhat more), which then lie one a lane and count
// those before them; a round a choice (warp maximum, its lane's next best)
// took twice the instructions, and the kernel is bound by those for many tokens.
// Without a bias the value is the logit itself, since the scores rise with it:
// the choice is then exact (but for groups whose scores fp64 may not tell apart),
// and scores are formed only where sums of two or the weights need them.  With a
// bias it is c = s + b in fp32, which is off by less than `slack` (below); where
// two neighbours in the order of the choice lie closer than that, the candidates'
// c are formed and ordered in fp64, one a lane, and where groups across the cut
// do, the two are, or (more than two, or more candidates than lanes) the warp
// makes the whole choice again in fp64.  The first is one token in some hundreds
// on logits of a spread of two, the last one in thousands;
// fp64 for every token, the first form of this kernel, ran 176 us on 4096 tokens
// x 256 experts and 537 us on 16381 x 200, now 11.5 and 26 us (the GPU's fp64 rate
// is a small share of its fp32 rate, and one such token is all that an SM waits
// for).
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
MOE_DEV float reduce_max(float v) { return key_float(__reduce_max_sync(kAll, float_order_key(v))); }
// NaN: masked; +inf: the largest number
MOE_DEV float clean(float v) { return v != v ? -INFINITY : fminf(v, kFltMax); }

struct Owned {
  int lpg, grp, n, e0;  // lanes a group, the lane's group, its experts e0 .. e0 + n - 1
};

// The lane's two largest c to those of its group, on each of the group's lanes.
template <typename F>
MOE_DEV void group_best(F& a1, F& a2, int lpg) {
  for (int o = lpg >> 1; o; o >>= 1) {
    const F b1 = __shfl_xor_sync(kAll, a1, o), b2 = __shfl_xor_sync(kAll, a2, o);
    a2 = fmax(fmax(a2, b2), fmin(a1, b1));
    a1 = fmax(a1, b1);
  }
}
// The group's value; -inf where it has nothing left.
template <typename F>
MOE_DEV F value_of(F a1, F a2, bool top2) {
  return top2 && a2 != -INFINITY ? a1 + a2 : a1;
}
template <typename F>
MOE_DEV F group_value(F a1, F a2, int lpg, bool top2) {
  group_best(a1, a2, lpg);
  return value_of(a1, a2, top2);
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

// Monotone map double -> unsigned (-0 as +0): the order of c by integer
// comparisons, fp64 ones have a latency of 64 cycles here.
MOE_DEV unsigned long long order_key64(double v) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}

// c of one expert in fp64 (about 1500 cycles).  Not inlined, and the loops around it not unrolled:
// straight-line code that one warp runs once is paid for in instruction fetches
// (the unrolled form held its SM for 30 us).
__device__ __noinline__ double exact_c(bool sigmoid, float l, float b, double m, double z) {
  const double e = exp(sigmoid ? -(double)l : (double)l - m);
  return (sigmoid ? 1.0 / (1.0 + e) : e / z) + (double)b;
}

MOE_DEV float logit(const RouteParams& P, uint32_t t, int e) {
  return clean(elem_load(P.logits, P.dtype, (size_t)t * P.stride + e));
}
MOE_DEV float bias_of(const RouteParams& P, int e) { return P.bias ? clean(P.bias[e]) : 0.f; }

// The softmax's largest logit and sum in fp64.
__device__ __noinline__ void exact_sum(const RouteParams& P, uint32_t t, const Owned& o, double& m, double& z) {
  float top = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < o.n; ++i) top = fmaxf(top, logit(P, t, o.e0 + i));
  m = warp_max(top);
  z = 0.0;
#pragma unroll 4
  for (int i = 0; i < o.n; ++i) {
    const float l = logit(P, t, o.e0 + i);
    if (l != -INFINITY) z += exp((double)l - m);
  }
  z = warp_sum(z);
}

// The whole choice in fp64: lane j gets the j-th expert and its logit.
template <int EPL>
__device__ __noinline__ void choose_exact(const RouteParams& P, uint32_t t, const Owned& o, int& id, float& lj) {
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
    key[i] = order_key64(c);
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
__device__ __noinline__ void settle(const RouteParams& P, uint32_t t, const Owned& o, int n, int& id, float& lj) {
  const int lane = threadIdx.x & 31;
  double m = 0.0, z = 1.0, c = -INFINITY;
  if (!P.sigmoid) exact_sum(P, t, o, m, z);
  if (id >= 0) c = exact_c(P.sigmoid, lj, bias_of(P, id), m, z);
  const unsigned long long key = order_key64(c);
  const uint32_t lk = float_order_key(lj);
  int rank = 0;
#pragma unroll 2
  for (int j = 0; j < n; ++j) {
    const unsigned long long k2 = __shfl_sync(kAll, key, j);
    const uint32_t l2 = __shfl_sync(kAll, lk, j);
    const int e2 = __shfl_sync(kAll, id, j);
    rank += k2 > key || (k2 == key && (l2 > lk || (l2 == lk && e2 < id)));
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

// The K best (and, with a bias, those near the cut) one a round, when there are
// too many candidates for one a lane: every lane offers its best.
template <int EPL, typename Slack>
MOE_DEV void choose_rounds(const RouteParams& P, float (&c)[EPL], const Owned& o, bool biased, Slack slack, int& n,
                           int& id, float& cj, bool& unsure) {
  const int lane = threadIdx.x & 31;
  id = -1;
  cj = -INFINITY;
  float cut = INFINITY;
  float best;
  int at;
  auto local_best = [&]() {
    best = -INFINITY;
    at = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (c[i] > best) {
        best = c[i];
        at = i;
      }
  };
  local_best();
#pragma unroll 1
  for (n = 0; n < (biased ? 32 : P.K); ++n) {
    const float top = key_float(__reduce_max_sync(kAll, float_order_key(best)));
    if (top == -INFINITY || (n >= P.K && cut - top > slack(cut))) break;
    const int src = __ffs(__ballot_sync(kAll, best == top)) - 1;
    const int e = __shfl_sync(kAll, o.e0 + at, src);
    if (n < P.K) cut = top;
    if (lane == n) {
      id = e;
      cj = top;
    }
    if (lane == src) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i == at) c[i] = -INFINITY;
      local_best();
    }
  }
  // no lane left, and the next one is near the cut
  const float next = key_float(__reduce_max_sync(kAll, float_order_key(best)));
  unsure = biased && n == 32 && next != -INFINITY && cut - next <= slack(cut);
}

// Values of the two groups at the cut in fp64: true if the one left out comes
// before the other.  Only experts that may be among their group's best (c in fp32
// from `least` on) are formed again.
template <int EPL>
MOE_DEV bool border_swaps(const RouteParams& P, uint32_t t, const Owned& o, const float (&c)[EPL], float least,
                          int in_grp, int out_grp) {
  double m = 0.0, z = 1.0;
  if (!P.sigmoid) exact_sum(P, t, o, m, z);
  uint32_t todo = 0u;  // of the lane's experts
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (EPL <= 32 && (o.grp == in_grp || o.grp == out_grp) && c[i] != -INFINITY && c[i] >= least) todo |= 1u << i;
  double x1 = -INFINITY, x2 = -INFINITY;
  while (__any_sync(kAll, todo != 0u)) {
    if (todo) {
      const int e = o.e0 + __ffs(todo) - 1;
      const double x = exact_c(P.sigmoid, logit(P, t, e), bias_of(P, e), m, z);
      x2 = fmax(x2, fmin(x1, x));
      x1 = fmax(x1, x);
      todo &= todo - 1u;
    }
    __syncwarp();
  }
  const double val = group_value(x1, x2, o.lpg, P.top2);
  const double vi = __shfl_sync(kAll, val, in_grp * o.lpg), vo = __shfl_sync(kAll, val, out_grp * o.lpg);
  return vo > vi || (vo == vi && out_grp < in_grp);
}

template <int EPL>
__global__ void __launch_bounds__(32 * kWarps, EPL <= 8 ? 6 : 1) k_route(const __grid_constant__ RouteParams P) {
  __shared__ float2 s_cand[kWarps][32];  // a candidate's c and id
  __shared__ float s_logit[kWarps][32];  // and its logit
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2* const cand = s_cand[warp];
  float* const cand_l = s_logit[warp];
  Owned o;
  o.lpg = 1 << P.lpg_log;
  o.grp = lane >> P.lpg_log;
  const int first = (lane & (o.lpg - 1)) * P.per;
  o.n = o.grp < P.G ? max(0, min(P.per, P.gs - first)) : 0;
  o.e0 = o.grp * P.gs + first;
  pdl_wait();
  pdl_launch_dependents();
  const bool biased = P.bias != nullptr;
  const bool scored = biased || (P.G > 1 && P.top2);  // c holds scores
  float b[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) b[i] = biased && i < o.n ? clean(P.bias[o.e0 + i]) : 0.f;

  // a token's logits as they lie in memory: those of the warp's next token are
  // asked for before it works on one
  uint32_t w[EPL];
  auto ask = [&](uint32_t t) {
    if (t >= (uint32_t)P.T) return;
    const size_t row = (size_t)t * P.stride + o.e0;
    if (EPL >= 4 && P.vec) {
#pragma unroll
      for (int i = 0; i + 4 <= EPL; i += 4)
        if (i < o.n) {
          const uint4 v = raw_load4(P.logits, P.dtype, row + i);
          w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i < o.n) w[i] = raw_load(P.logits, P.dtype, row + i);
    }
  };
  ask(blockIdx.x * kWarps + warp);
  for (uint32_t t = blockIdx.x * kWarps + warp; t < (uint32_t)P.T; t += gridDim.x * kWarps) {
    float l[EPL], c[EPL];
    if (EPL >= 4 && P.vec) {
#pragma unroll
      for (int i = 0; i + 4 <= EPL; i += 4)
        raw_values4(make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]), P.dtype, l + i);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) l[i] = raw_value(w[i], P.dtype);
    }
    ask(t + gridDim.x * kWarps);
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = i < o.n ? clean(l[i]) : -INFINITY;
    // c in fp32 (the logit where the choice can go by it), the softmax's sum
    float m = 0.f, z = 1.f, smax = 1.f;
    if (!P.sigmoid && (scored || !P.renorm)) {
      m = l[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
      m = key_float(__reduce_max_sync(kAll, float_order_key(m)));
      z = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        c[i] = l[i] == -INFINITY ? 0.f : __expf(l[i] - m);
        z += c[i];
      }
      z = warp_sum(z);
      smax = 1.f / z;
    }
    if (!scored) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = l[i];
    } else {
      if (P.sigmoid) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = __fdividef(1.f, 1.f + __expf(-l[i]));
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] *= smax;
      }
      // (a bias of -inf masks by itself)
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = l[i] == -INFINITY ? -INFINITY : c[i] + b[i];
    }
    // How far apart two fp32 values of c have to be for their order to be that of
    // fp64, in units of 2^-24.  Sigmoid: the fast exp is off by 4 and 2 |l|
    // relative, which s takes up times 1 - s (|l| s (1 - s) < 1/4), sum and
    // quotient by 4: less than 8 of s <= 1.  Softmax, of the largest s: exp by 4
    // and 2 |x| (exp(-|x|) |x| < 1/2), the sum of such terms by 4 and twice their
    // mean |x| (at most ln E < 7) and its EPL + 5 additions, the reciprocal and
    // the product 3: less than EPL + 32.  Both sides of a comparison count, and
    // the rounding of s + b: |c| each.
    constexpr float kSoft = (2 * EPL + 64) * 0x1p-24f;
    auto slack = [&](float v) { return smax * (P.sigmoid ? 0x1p-20f : kSoft) + fabsf(v) * 0x1p-22f + 0x1p-120f; };
    bool unsure = false;
    if (P.G > 1) {
      float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        a2 = fmaxf(a2, fminf(a1, c[i]));
        a1 = fmaxf(a1, c[i]);
      }
      group_best(a1, a2, o.lpg);
      // (half of a sum of two: it stays within fp32's range, and a group held back
      // by the lowest number comes before one that has nothing left)
      const float half = P.top2 ? 0.5f : 1.f, val = value_of(half * a1, half * a2, P.top2);
      int rank = group_rank(val, P.G, o);
      const bool live = o.grp < P.G && val != -INFINITY, in = rank < P.top_groups;
      if (!scored) {
        // By the largest logit, which orders the groups as their scores do but
        // where these are equal in fp64 and the logits are not: both 1 or 0, or
        // the logits closer than a score's rounding.  Equal values go to the lower
        // group, so where the cut may lie between two such the choice is made in
        // fp64.  Elsewhere scores differ by 2^-24 e^-16 and more (softmax, and the
        // sigmoid of negative logits: by 2^-24 of the score).
        auto at_rank = [&](int k) {
          return __shfl_sync(kAll, val, __ffs(__ballot_sync(kAll, o.grp < P.G && rank == k)) - 1);
        };
        const float lo = at_rank(P.top_groups - 1), hi = at_rank(P.top_groups);
        if (hi != -INFINITY) {
          // the lane's group against the nearest one across the cut
          const float x = in ? val : lo, y = in ? hi : val;
          const bool equal = P.sigmoid ? x <= -690.f || y >= 15.f : val - lo >= 690.f;
          unsure = __any_sync(kAll, live && x > y && (x - y <= 0x1p-24f || equal));
        }
      } else {
        // A group's value is off by less than a band of its own: that of the
        // scores, and the roundings of each c and of their sum, which go by the
        // magnitudes of the two c (the sum may cancel).  Groups kept and left out
        // whose bands meet are told apart in fp64, one of each by themselves.
        const bool two = P.top2 && a2 != -INFINITY;
        const float w = two ? a2 : a1, mag = half * fabsf(a1) + (two ? half * fabsf(a2) : 0.f);
        const float band = smax * (P.sigmoid ? 0x1p-21f : 0.5f * kSoft) + mag * 0x1p-22f + 0x1p-120f;
        const float lo = -reduce_max(live && in ? band - val : -INFINITY);
        const float hi = reduce_max(live && !in ? val + band : -INFINITY);
        if (lo <= hi) {
          const bool one = (lane & (o.lpg - 1)) == 0;  // of the group's lanes
          const uint32_t kept = __ballot_sync(kAll, one && live && in && val - band <= hi);
          const uint32_t left = __ballot_sync(kAll, one && live && !in && val + band >= lo);
          const int gi = (__ffs(kept) - 1) >> P.lpg_log, go = (__ffs(left) - 1) >> P.lpg_log;
          if (EPL > 32 || __popc(kept) != 1 || __popc(left) != 1)
            unsure = true;
          else if (border_swaps<EPL>(P, t, o, c, w - 2.f * slack(w), gi, go))
            rank = o.grp == gi ? P.top_groups : o.grp == go ? P.top_groups - 1 : rank;
        }
      }
      // no bias: the choice inside the groups goes by the logits
      const bool kept = rank < P.top_groups;
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = !kept ? -INFINITY : biased ? c[i] : l[i];
    }
    // The choice.  The K-th largest of the lanes' largest c bounds the K-th
    // largest c from below: what reaches it (with a bias: to within the slack)
    // are the candidates, K or somewhat more, and with one a lane each counts
    // those before it.
    int id = -1, n = 0;
    float cj = -INFINITY, lj = -INFINITY;
    if (!unsure) {
      float top = c[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) top = fmaxf(top, c[i]);
      uint32_t key = float_order_key(top), bar_key = 0u;
      for (int have = 0; have < P.K;) {
        bar_key = __reduce_max_sync(kAll, key);
        const bool mine = key == bar_key;
        have += __popc(__ballot_sync(kAll, mine));
        key = mine ? 0u : key;  // (below every float's key)
      }
      float bar = key_float(bar_key);
      if (biased) bar -= slack(bar);
      bar = fmaxf(bar, -kFltMax);  // -inf: not a candidate
      int mine = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) mine += c[i] >= bar;
      int at = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kAll, at, d);
        if (lane >= d) at += v;
      }
      n = __shfl_sync(kAll, at, 31);
      at -= mine;
      if (n <= 32) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (c[i] >= bar) {
            cand[at] = make_float2(c[i], __int_as_float(o.e0 + i));
            cand_l[at++] = l[i];
          }
      }
      __syncwarp();
      if (n <= 32) {
        if (lane < n) {
          const float2 v = cand[lane];
          cj = v.x;
          id = __float_as_int(v.y);
          lj = cand_l[lane];
        }
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          const float2 v = cand[j];
          rank += v.x > cj || (v.x == cj && __float_as_int(v.y) < id);
        }
        __syncwarp();
        if (lane < n) {
          cand[rank] = make_float2(cj, __int_as_float(id));
          cand_l[rank] = lj;
        }
        __syncwarp();
        if (lane < n) {
          const float2 v = cand[lane];
          cj = v.x;
          id = __float_as_int(v.y);
          lj = cand_l[lane];
        }
        __syncwarp();
      } else {
        choose_rounds<EPL>(P, c, o, biased, slack, n, id, cj, unsure);
        lj = id >= 0 ? logit(P, t, id) : -INFINITY;
      }
    }
    if (biased && !unsure) {
      // neighbours closer than the slack: the candidates change places by fp64
      const float next = __shfl_down_sync(kAll, cj, 1);
      if (__any_sync(kAll, lane + 1 < n && cj - next <= slack(cj))) settle(P, t, o, n, id, lj);
    }
    if (unsure) choose_exact<EPL>(P, t, o, id, lj);
    if (lane >= P.K) {
      id = -1;
      lj = -INFINITY;
    }

    // Weights from the chosen logits.  Renormalised, the softmax needs no other
    // logit, and the sigmoid, e^l / (1 + e^l), is formed times e^-top where every
    // chosen logit is below 0: a ratio of two small scores then does not underflow.
    float v = 0.f;
    if (P.renorm) {
      const float top = warp_max(lj);
      if (id >= 0) {
        if (P.sigmoid && !(top < 0.f)) {
          v = 1.f / (1.f + expf(-lj));
        } else {
          v = expf(lj - top);
          if (P.sigmoid) v /= 1.f + expf(lj);
        }
      }
      const float total = warp_sum(v);
      if (id >= 0) v = __fdividef(v, total);
    } else if (id >= 0) {
      v = P.sigmoid ? 1.f / (1.f + expf(-lj)) : expf(lj - m) / z;
    }
    if (lane < P.K) {
      P.ids[(size_t)t * P.K + lane] = id;
      P.w[(size_t)t * P.K + lane] = v * P.scale;
    }
  }
}

}  // namespace

cudaError_t launch_route(RouteParams p, cudaStream_t stream) {
  p.lpg_log = 5;
  for (int g = 1; g < p.G; g <<= 1) --p.lpg_log;
  p.per = (p.gs + (1 << p.lpg_log) - 1) >> p.lpg_log;
  // four experts a load: rows, groups and lanes start on a load's boundary
  if (p.per > 2) {
    const int per4 = (p.per + 3) & ~3;
    const uintptr_t bytes = p.dtype == kF32 ? 16 : 8;
    p.vec = p.gs % 4 == 0 && p.stride % 4 == 0 && reinterpret_cast<uintptr_t>(p.logits) % bytes == 0;
    if (p.vec) p.per = per4;
  }
  // a warp goes through several tokens where there are more than run at once
  const int blocks = 1 + (p.T - 1) / kWarps, most = 6 * p.sms;
  const dim3 grid(blocks < most ? blocks : most);
  const int threads = 32 * kWarps;
  if (p.per <= 2) return launch_behind(k_route<2>, grid, threads, 0, stream, p);
  if (p.per <= 4) return launch_behind(k_route<4>, grid, threads, 0, stream, p);
  if (p.per <= 8) return launch_behind(k_route<8>, grid, threads, 0, stream, p);
  if (p.per <= 16) return launch_behind(k_route<16>, grid, threads, 0, stream, p);
  if (p.per <= 32) return launch_behind(k_route<32>, grid, threads, 0, stream, p);
  return launch_behind(k_route<64>, grid, threads, 0, stream, p);
}

}  // namespace moe

// Adapters (see moe_adapters.cuh): the order of the tokens, the launches.
#include "moe_adapters.cuh"

namespace moe {

cudaError_t launch_adapters_f16(const AdapterParams& p, int blocks, cudaStream_t stream);

namespace {

constexpr int kOrderTokens = 32;  // tokens a block of k_order ranks, eight threads a token

// Places of the window's tokens in the order (adapter, token): a token's place
// is the number of tokens before it, and its place in its adapter's run that less
// the number of tokens of lower adapters: two counts (a third, of the run,
// took 2.6 us more of the whole call at 8192 tokens; the tile finds its end
// itself).  Eight threads a token, each against an eighth of the window.
// marks[place]: whether a tile starts there (a run of one adapter is cut every
// P.tile tokens).
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
  int place = 0, start = 0;
#pragma unroll 4
  for (int j0 = 4 * part; j0 < n; j0 += 32) {
    const int4 v = *reinterpret_cast<const int4*>(s_a + j0);
    const int o[4] = {v.x, v.y, v.z, v.w};
    const int below = a + (j0 + 4 <= i);  // tokens before this one count with the same adapter too
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      place += o[e] < below;
      start += o[e] < a;
    }
  }
  // those of the token's own four
  if (part == (i >> 2 & 7))
    for (int j = i & ~3; j < i; ++j) place += s_a[j] == a;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    place += __shfl_xor_sync(0xffffffffu, place, o);
    start += __shfl_xor_sync(0xffffffffu, start, o);
  }
  if (part == 0 && i < n) {
    P.order[t0 + place] = t0 + i;
    P.adapter_at[t0 + place] = a;
    P.marks[t0 + place] = (place - start) % P.tile == 0;
  }
}

constexpr int kMaxSms = 192;  // the workspace does not depend on the device

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Parts of K: enough blocks for the GPU from `tiles` tiles, each warp at least
// one 32-column block.
int splits_for(int sms, int tiles, int K) {
  const int most = (K + 32 * kWarps - 1) / (32 * kWarps);
  const int want = 2 * sms / (tiles > 0 ? tiles : 1);
  const int s = want < 8 ? want : 8;
  return s < 1 ? 1 : s < most ? s : most;
}

// Parts of K at most: those of the fewest tiles that T tokens can make.
int most_splits(int T, int K) { return 2 * splits_for(kMaxSms, (T + 63) / 64, K); }

}  // namespace

// v for every part of K, then (many tokens) the order and the marks.
size_t adapters_workspace(int T, int K, int N, int R) {
  (void)N;
  const size_t v = align256((size_t)most_splits(T, K) * T * R * 4);
  return T <= kScanT ? v : v + 2 * align256((size_t)T * 4) + align256((size_t)T);
}

cudaError_t launch_adapters(AdapterParams p, cudaStream_t stream) {
  const uintptr_t four = p.y_dtype == kF32 ? 16 : 8;
  p.vec = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.y) % four == 0 &&
          reinterpret_cast<uintptr_t>(p.out) % four == 0 && (p.T == 1 || (p.y_stride % 4 == 0 && p.out_stride % 4 == 0));
  // tokens a tile: 64, or 8 where an adapter has no more than that on average
  // (an adapter with more is then read once every 8)
  p.tile = p.T <= 8 || p.T / 8 <= p.n ? 8 : 64;
  const int least = (p.T + p.tile - 1) / p.tile, likely = least > p.n ? least : p.n < p.T ? p.n : p.T;
  p.splits = splits_for(p.sms, likely, p.K);
  if (p.tile == 64) p.splits *= 2;  // two parts a block
  // columns a block of k_expand goes through: finding the tile and staging its v
  // are paid once a block, so as many as leave two blocks for every SM
  const int step = p.tile == 64 && p.N >= 512 && p.vec ? 2 * kThreads : kThreads;
  const int chunks = (p.N + step - 1) / step;
  const int each = (int)(((long long)likely * chunks + 2 * p.sms - 1) / (2 * p.sms));
  p.cols = (each > chunks ? chunks : each) * step;
  int blocks = p.T;
  if (p.T > kScanT) {
    const int wn = (p.T + kWindow - 1) / kWindow, len = p.T < kWindow ? p.T : kWindow;
    uint8_t* w = reinterpret_cast<uint8_t*>(p.v) + align256((size_t)most_splits(p.T, p.K) * p.T * p.R * 4);
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
  return p.f16 ? launch_adapters_f16(p, blocks, stream) : launch_products<false>(p, blocks, stream);
}

}  // namespace moe

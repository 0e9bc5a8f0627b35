// Attention over a paged cache for units of up to 128 rows: trees of drafted tokens
// and ends of prompts (see moe_attend.cuh for the division of the work).
//
// With 128 rows a token's key and value enter 4 D 128 products for 4 D bytes: more
// than the warp-level instruction can do at the rate of the stream, a third of what
// tcgen05 can.  So the rows are the 128 lanes of tensor memory.  A step is 128
// tokens, its two halves two streams with scores, output, running maximum and sum
// of their own, so that one stream's weights are formed while the other's products
// run; they meet at the end of the unit.  Tensor memory (D <= 128): two buffers of
// 64 columns of scores a stream, which the weights (two numbers of the cache's type
// each, 32 columns each) overwrite as operand of the second product, and the
// output, 64 or 128 columns a stream.
//
//   warps 0, 12   issue the products for the scores of a stream each,
//   warps 13, 14  those of its weighted values (one warp for all took three times as
//                 long as the stream of the cache, one a stream half as long again)
//   warps 1, 15   tensor copies of keys, of values (and queries) (one warp for both
//                 took longer than the stream, too)
//   warps 2, 3    in the tiles that hold tokens which some rows do not see, take values
//                 that are not finite out (a product with a weight of 0 has an effect
//                 then); the rows that do see them get them at the end, as those of
//                 the other tiles, which leave sums that are not finite.  Queries that
//                 tensor copies cannot fetch
//   warps 4-11    a thread a row: scores to weights, four warps a stream
//
// Keys and values of each stream have rings of their own: every barrier then has one
// waiter that meets all of its phases in turn.  (A wait by parity tells a phase from
// the next only: with one ring for all, a waiter could be two phases ahead.)
//
// Measured: a step of 64 KB an SM 1.4 us, 7 TB/s (D = 128); a call of one step 13 us
// (the way from the lengths to the page, the tile, the first scores, and cold
// instructions everywhere); 16 trees of 16 tokens, 139 MB, 39 us.
//
// Every wait is bounded.  After one that ran out, in whichever thread, nobody waits,
// issues or arrives any more, but all still meet at the block's barriers, and results
// become NaN.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_attend.cuh"
#include "moe_elem.cuh"
#include "moe_internal.h"
#include "moe_mma.cuh"
#include "moe_tc.cuh"
#include "moe_tma.cuh"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kThreads = 512, kTok = 64;  // tokens of a stream's half step
constexpr int kOddUnits = 16;  // marks of values taken out: more than the units under way

__host__ __device__ constexpr int depth_for(int dp) { return dp == 64 ? 4 : 2; }  // tiles of a ring
__host__ __device__ constexpr int wide_smem(int dp) { return 4 * depth_for(dp) * kTok * dp * 2 + 2 * 128 * dp * 2 + 1024; }

__device__ __forceinline__ void umma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 lanes x 16 or 32 columns; a read waits for itself: nothing can use it before
__device__ __forceinline__ void tmem_read16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}"
      ", [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_read32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%"
      "26,%27,%28,%29,%30,%31}"
      ", [%32];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_write16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16}"
      ";" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_write32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
      "%27,%28,%29,%30,%31,%32}"
      ";" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A shared-memory descriptor with its address moved by `bytes`.
MOE_DEV uint64_t desc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// One lane of a warp that is here as a whole.  The products and copies are issued
// under this, with operands that all lanes form alike: from a branch on the lane's
// number an instruction took 110 to 190 cycles.
MOE_DEV bool elected() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0u;
}

// A bounded wait.  `gone` is the block's: some wait has run out.
MOE_DEV void await(uint64_t* bar, uint32_t parity, bool& dead, volatile int* gone) {
  if (dead || mbar_try_wait(bar, parity)) return;
  const unsigned long long t0 = global_ns();
  for (uint32_t i = 1; i < kSpinLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if ((i & 31) == 0 && (*gone || global_ns() - t0 > kWaitLimitNs)) break;
    if (i > 64) __nanosleep(32);
  }
  dead = true;
  *gone = 1;
}

// A place in a ring and its pass.
template <int DEPTH>
struct Ring {
  int slot, end;
  uint32_t turn;
  MOE_DEV Ring(int ring, uint32_t first) : slot(ring * DEPTH), end((ring + 1) * DEPTH), turn(first) {}
  MOE_DEV void next() {
    if (++slot == end) {
      slot -= DEPTH;
      turn ^= 1u;
    }
  }
};

// Bits of the 64 tokens from `first` on that row t, the j-th of its sequence, sees.
MOE_DEV uint64_t seen_tokens(const AttendParams& P, const AttendSeq& s, int first, int t, int j) {
  const int left = s.len - first, o = first - (s.len - s.n);  // o: the first one's place among the sequence's own
  uint64_t seen = left >= kTok ? ~0ull : left > 0 ? (1ull << left) - 1ull : 0ull;
  if (t < 0 || o + kTok <= 0) return seen;
  if (!P.mask) {
    const int k = j - o + 1;
    return k >= kTok ? seen : k > 0 ? seen & ((1ull << k) - 1ull) : 0ull;
  }
  const int32_t* const row = P.mask + (long long)t * P.mask_stride;
  auto word = [&](int i) { return i < P.mask_words ? (uint64_t)(uint32_t)row[i] : 0ull; };
  if (o < 0) return seen & ((word(0) | word(1) << 32) << -o | ((1ull << -o) - 1ull));
  const int w = o >> 5, sh = o & 31;
  const uint64_t lo = word(w) | word(w + 1) << 32;
  return seen & (sh ? lo >> sh | word(w + 2) << (64 - sh) : lo);
}

template <bool F16, int DP>
__global__ void __launch_bounds__(kThreads, 1) k_attend_wide(const __grid_constant__ AttendParams P) {
  constexpr int kDepth = depth_for(DP), NS = 4 * kDepth, kSlot = kTok * DP * 2, kQ = 128 * DP * 2, kHalves = DP / 64;
  constexpr int kDt = F16 ? kF16 : kBf16;
  // (as in k_attend: the maximum stays within 2^8, fp16 weights are held 2^7 up)
  constexpr float kLazy = 8.f, kUp = F16 ? 7.f : 0.f;
  constexpr uint32_t kOut = 256;  // columns of tensor memory before the outputs
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* const qs = smem + NS * kSlot;
  __shared__ uint64_t full[NS], empty[NS], s_full[2][2], s_free[2][2], p_full[2][2], o_free, q_full[2], q_empty[2], raw[2 * kDepth];
  __shared__ int s_gone;
  __shared__ uint32_t s_tmem;
  __shared__ float2 s_stat[2][2][128];
  __shared__ uint32_t s_boxes[2][16], s_odd[kOddUnits];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int x = 0; x < 2; ++x) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[x][b], 1);
        mbar_init(&s_free[x][b], 1);
        mbar_init(&p_full[x][b], 128);
      }
      mbar_init(&q_full[x], P.q_box ? 1 : 64);
      mbar_init(&q_empty[x], 2);
    }
    mbar_init(&o_free, 256);
    for (int i = 0; i < 2 * kDepth; ++i) mbar_init(raw + i, 1);
    s_gone = 0;
    mbar_fence_init();
    for (int i = 0; i < kOddUnits; ++i) s_odd[i] = 0u;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 1 && lane == 0) {
    prefetch_tensormap(&P.tm_k);
    prefetch_tensormap(&P.tm_v);
  }
  pdl_wait();
  pdl_launch_dependents();
  fence_proxy_async_global();  // what the kernel before wrote, for the tensor copies
  AttendStep a = attend_begin<kThreads>(P);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s_tmem;
  bool dead = false;
  auto first_of = [](const AttendStep& s, int x) { return s.chunk * 2 * kTok + x * kTok; };
  auto there = [&](const AttendStep& s, int x) { return x == 0 || first_of(s, 1) < s.s.len; };
  auto last_of_unit = [](const AttendStep& s) { return s.left == 1 || s.chunk + 1 == s.s.chunks; };
  // a tile that holds tokens which some rows do not see
  auto mixed = [&](const AttendStep& s, int x) { return first_of(s, x) + kTok > attend_common(P, s.s); };

  // (by whole warps, which stay of one mind)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    await(bar, parity, dead, &s_gone);
    dead = __any_sync(kAll, dead);
  };
  // (rings 0, 1: keys of the streams; 2, 3: values)
  if (warp == 0 || warp == 12) {
    // ------------------------------------------------------------ products: scores
    const int x = warp == 0 ? 0 : 1;  // the warp's stream
    const uint32_t s_desc = tc::instr_desc(128, kTok, 0, F16);
    const uint64_t k_desc0 = tc::smem_desc(smem_u32(smem), 16, 1024), q_desc0 = tc::smem_desc(smem_u32(qs), 16, 1024);
    Ring<kDepth> ring(x, 0u);
    int unit = 0, count = 0;  // count: the stream's chunks so far
    bool begin = true;
    for (; a.left > 0; a.next(P)) {
      if (begin) wait(&q_full[unit & 1], unit >> 1 & 1);
      begin = last_of_unit(a);
      if (there(a, x)) {
        const int buf = count & 1;
        if (count > 1) wait(&s_free[x][buf], (count >> 1) - 1 & 1);
        wait(full + ring.slot, ring.turn);
        tc::tc_fence_after();
        const uint64_t k_desc = desc_at(k_desc0, ring.slot * kSlot), q_desc = desc_at(q_desc0, (unit & 1) * kQ);
        const uint32_t to = tmem + x * 128 + buf * 64;
        if (!dead && elected()) {
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks)
            tc::umma(to, desc_at(q_desc, (ks >> 2) * 128 * 128 + (ks & 3) * 32),
                     desc_at(k_desc, (ks >> 2) * kTok * 128 + (ks & 3) * 32), s_desc, ks > 0);
          tc::umma_commit(empty + ring.slot);
          tc::umma_commit(&s_full[x][buf]);
        }
        __syncwarp();
        ring.next();
        ++count;
      }
      if (begin) {
        if (!dead && elected()) tc::umma_commit(&q_empty[unit & 1]);
        __syncwarp();
        ++unit;
      }
    }
  } else if (warp == 13 || warp == 14) {
    // ------------------------------------------------------------ products: weighted values
    const int x = warp - 13;
    // (values: columns are what lies together)
    const uint32_t o_desc = tc::instr_desc(128, DP, 0, F16) | 1u << 16;
    const uint64_t v_desc0 = tc::smem_desc(smem_u32(smem), kTok * 128, 1024);
    Ring<kDepth> ring(2 + x, 0u);
    int unit = 0, count = 0;
    bool fresh = true;  // the unit's first product is still to come
    for (; a.left > 0; a.next(P)) {
      if (there(a, x)) {
        const int buf = count & 1;
        wait(full + ring.slot, ring.turn);
        wait(&p_full[x][buf], count >> 1 & 1);
        // (the unit's first weights are there: its stream's threads have left the unit before,
        // and met the others there, who had left the one before that: no phase but the last
        // can be open)
        if (fresh && unit > 0) wait(&o_free, (unit - 1) & 1);
        tc::tc_fence_after();
        const uint64_t v_desc = desc_at(v_desc0, ring.slot * kSlot);
        const uint32_t to = tmem + kOut + x * DP, p_at = tmem + x * 128 + buf * 64, add = !fresh;
        if (!dead && elected()) {
#pragma unroll
          for (int term = 1; term >= 0; --term)
#pragma unroll
            for (int ks = 0; ks < kTok / 16; ++ks)
              umma_ts(to, p_at + (ks >> 1) * 32 + term * 16 + (ks & 1) * 8, desc_at(v_desc, ks * 16 * 128), o_desc,
                      term == 1 && ks == 0 ? add : 1u);
          tc::umma_commit(empty + ring.slot);
          tc::umma_commit(&s_free[x][buf]);
        }
        __syncwarp();
        ring.next();
        ++count;
        fresh = false;
      }
      if (last_of_unit(a)) {
        fresh = true;
        ++unit;
      }
    }
  } else if (warp == 1 || warp == 15) {
    // ------------------------------------------------------------ copies
    const bool keys = warp == 1;
    const CUtensorMap* const map = keys ? &P.tm_k : &P.tm_v;
    const int boxes = kTok / P.box;  // of a tile; lane b < boxes knows box b's page
    const uint64_t once = policy_evict_first(), again = policy_evict_last();
    Ring<kDepth> rings[2] = {Ring<kDepth>(keys ? 0 : 2, 1u), Ring<kDepth>(keys ? 1 : 3, 1u)};  // (empty at first)
    int unit = 0, mixed_at = 0;
    struct Where {
      int page[2], in[2];  // the box's page (behind the cache: zeros) and its first slot there
    };
    auto look = [&](const AttendStep& s) {
      Where w;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int t = first_of(s, x) + lane * P.box, at = attend_page(P, t);
        w.in[x] = t - at * P.page_size;
        w.page[x] = -1;
        if (lane < boxes && s.left > 0 && t < s.s.len) w.page[x] = P.table[s.b * P.table_stride + at];
      }
      return w;
    };
    Where now = look(a);
    bool begin = true;
    for (int i = 0; a.left > 0; ++i) {
      if (!keys && begin && P.q_box) {
        // the unit's queries: q_box tokens of the group's heads are its rows in their order
        if (unit >= 2) wait(&q_empty[unit & 1], (unit >> 1) - 1 & 1);
        if (!dead && elected()) {
          mbar_arrive_expect_tx(&q_full[unit & 1], kHalves * 128 * P.G * P.q_box);
#pragma unroll
          for (int half = 0; half < kHalves; ++half)
            tensor_load_3d(qs + (unit & 1) * kQ + half * 128 * 128, &P.tm_q, 64 * half, a.head * P.G,
                           a.s.t0 + a.tile * P.q_box, &q_full[unit & 1], again);
        }
        __syncwarp();
        ++unit;
      }
      begin = last_of_unit(a);
      AttendStep next = a;
      Where soon;
      const uint64_t policy = a.s.tiles > 1 ? again : once;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x == 1) {
          // the next step's pages, behind this one's first copy
          next.next(P);
          soon = look(next);
        }
        if (!there(a, x)) continue;
        const int known = (uint32_t)now.page[x] < (uint32_t)P.pages ? now.page[x] : P.pages;
        if (keys) {
          const uint32_t real = __ballot_sync(kAll, known < P.pages);
          if (lane == 0) s_boxes[x][i & 15] = real;
          __syncwarp();
        }
        wait(empty + rings[x].slot, rings[x].turn);
        // (values that have to be looked through first: on a barrier of their own)
        uint64_t* bar = full + rings[x].slot;
        if (!keys && mixed(a, x)) {
          bar = raw + mixed_at;
          mixed_at = mixed_at + 1 == 2 * kDepth ? 0 : mixed_at + 1;
        }
        uint8_t* const to = smem + rings[x].slot * kSlot;
        if (!dead && elected()) mbar_arrive_expect_tx(bar, kSlot);
        __syncwarp();
#pragma unroll 1
        for (int b = 0; b < boxes; ++b) {
          const int page = __shfl_sync(kAll, known, b), in = __shfl_sync(kAll, now.in[x], b);
          const int c1 = P.slot_first ? in : a.head, c2 = P.slot_first ? a.head : in;
          if (!dead && elected()) {
#pragma unroll
            for (int half = 0; half < kHalves; ++half)
              tensor_load_4d(to + half * kTok * 128 + b * P.box * 128, map, 64 * half, c1, c2, page, bar, policy);
          }
          __syncwarp();
        }
        rings[x].next();
      }
      a = next;
      now = soon;
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ values that are not finite; queries
    const int th = tid - 64;
    Ring<kDepth> rings[2] = {Ring<kDepth>(2, 0u), Ring<kDepth>(3, 0u)};
    int unit = 0, mixed_at = 0;
    uint32_t mixed_turn = 0;
    auto queries = [&](const AttendStep& s) {
      if (unit >= 2) wait(&q_empty[unit & 1], (unit >> 1) - 1 & 1);
      uint8_t* const to = qs + (unit & 1) * kQ;
      const int rows = s.s.n * P.G, r0 = s.tile * P.rows;
      // eight pieces of 16 bytes are asked for at a time
#pragma unroll 1
      for (int x0 = th; x0 < 128 * DP / 8; x0 += 8 * 64) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int x = x0 + 64 * u, r = x / (DP / 8), c = x % (DP / 8);
          v[u] = make_uint4(0u, 0u, 0u, 0u);
          if (r < P.rows && r0 + r < rows && 8 * c < P.D) {
            const int j = (r0 + r) / P.G, h = s.head * P.G + (r0 + r) - j * P.G;
            v[u] = attend_query(P, s.s.t0 + j, h, c);
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int x = x0 + 64 * u, r = x / (DP / 8), c = x % (DP / 8);
          *reinterpret_cast<uint4*>(to + (c >> 3) * 128 * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v[u];
        }
      }
      fence_proxy_async();
      if (!dead) mbar_arrive(&q_full[unit & 1]);
    };
    bool begin = true;
    for (; a.left > 0; a.next(P)) {
      if (begin && !P.q_box) queries(a);
      begin = last_of_unit(a);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!there(a, x)) continue;
        if (mixed(a, x)) {
          wait(raw + mixed_at, mixed_turn);
          if (++mixed_at == 2 * kDepth) {
            mixed_at = 0;
            mixed_turn ^= 1u;
          }
          const int from = max(attend_common(P, a.s) - first_of(a, x), 0);
          uint8_t* const tile = smem + rings[x].slot * kSlot;
          bool odd = false;
          for (int y = th; y < kTok * DP / 8; y += 64) {
            const int r = y / (DP / 8), c = y % (DP / 8);
            if (r < from) continue;
            uint4* const at = reinterpret_cast<uint4*>(tile + (c >> 3) * kTok * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            uint4 v = *at;
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            bool any = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (odd16<F16>(w[e] & 0xFFFFu)) any = true, w[e] &= 0xFFFF0000u;
              if (odd16<F16>(w[e] >> 16)) any = true, w[e] &= 0xFFFFu;
            }
            if (any) *at = make_uint4(w[0], w[1], w[2], w[3]);
            odd |= any;
          }
          if (odd) s_odd[unit % kOddUnits] = (uint32_t)unit + 1u;  // the unit's mark: its number
          fence_proxy_async();
          named_bar_sync(2, 64);
          if (th == 0 && !dead) mbar_arrive(full + rings[x].slot);
        }
        rings[x].next();
      }
      if (begin) ++unit;
    }
  } else {
    // ------------------------------------------------------------ weights
    const int x = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    auto kept = [](float v) { return fminf(v, 3.4e38f); };  // (finite: 0 times infinity)
    const float scale = fabsf(P.scale);
    const uint32_t flip = P.scale < 0.f ? 0x80000000u : 0u;  // the scale's sign goes to the scores
    // (not 0 either: masked scores of -inf)
    const float mul = P.softcap > 0.f ? 1.f : fmaxf(kept(scale * kLog2e), 1.2e-38f);
    const float c1 = P.softcap > 0.f ? kept(scale / P.softcap) : 0.f, c2 = kept(P.softcap * kLog2e);
    int count = 0, unit = 0, i = 0;
    while (a.left > 0) {
      const int r = a.tile * P.rows + row, rows = a.s.n * P.G, j = r / P.G;
      const int t = row < P.rows && r < rows ? a.s.t0 + j : -1;
      const int chunk0 = a.chunk;
      float m = -INFINITY, l = 0.f;
      bool some = false, end = false, other = false;  // this stream, the second one have had a chunk
      for (; !end; ++i) {
        end = last_of_unit(a);
        other |= there(a, 1);
        if (there(a, x)) {
          const int buf = count & 1;
          const uint32_t at = tmem + lanes + x * 128 + buf * 64;
          wait(&s_full[x][buf], count >> 1 & 1);
          tc::tc_fence_after();
          const uint32_t boxes = s_boxes[x][i & 15], all = (1u << kTok / P.box) - 1u;
          const bool part = mixed(a, x) || boxes != all, changed = part || P.softcap > 0.f || flip;
          uint64_t seen = ~0ull;
          if (part) {
            seen = seen_tokens(P, a.s, first_of(a, x), t, j);
            for (int b = 0; b < kTok / P.box; ++b)
              if (!(boxes >> b & 1u)) seen &= ~((~0ull >> (64 - P.box)) << (b * P.box));
            __syncwarp();  // (each lane by its own way here; what follows takes whole warps)
          }
          // twice over the scores, 32 columns at a time: short loops, since what each
          // warp runs through once a step comes from beyond the nearest instruction cache
          float mx = -INFINITY;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t w[32];
            tmem_read32(at + 32 * h, w);
            if (changed) {
              if (flip) {
#pragma unroll
                for (int e = 0; e < 32; ++e) w[e] ^= flip;
              }
              if (P.softcap > 0.f) {
#pragma unroll
                for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(c2 * attend_tanh(__uint_as_float(w[e]) * c1));
              }
              if (part) {
                const uint32_t bits = (uint32_t)(seen >> (32 * h));
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(bits >> e & 1u)) w[e] = 0xFF800000u;  // -inf
              }
              __syncwarp();
              tmem_write32(at + 32 * h, w);
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(w[e]));
            mx = fmaxf(mx, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
          }
          if (changed) tmem_wait_st();
          mx *= mul;
          if (!some) {
            m = mx;
          } else if (__any_sync(kAll, mx > m + kLazy)) {
            // (each row by its own: what the others hold, behind the unit's rows too, must not
            // change its roundings)
            const bool own = mx > m + kLazy;
            const float f = own ? exp2_fast(m - mx) : 1.f;
            if (own) m = mx;
            l *= f;
            // (the buffer's phase before is closed: its present scores were formed behind it)
            wait(&s_free[x][count - 1 & 1], count - 1 >> 1 & 1);
            tc::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < DP; c += 16) {
              uint32_t o[16];
              tmem_read16(tmem + lanes + kOut + x * DP + c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_write16(tmem + lanes + kOut + x * DP + c, o);
            }
          }
          const float base = attend_base(m) - kUp;
          float sum[4] = {};
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t w[32], hi[16], lo[16];
            tmem_read32(at + 32 * h, w);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float p0 = exp2_fast(fmaf(__uint_as_float(w[2 * e]), mul, -base));
              const float p1 = exp2_fast(fmaf(__uint_as_float(w[2 * e + 1]), mul, -base));
              sum[2 * (e & 1)] += p0;
              sum[2 * (e & 1) + 1] += p1;
              hi[e] = pack2(kDt, p0, p1);
              float a0, a1;
              unpack2(kDt, hi[e], a0, a1);
              lo[e] = pack2(kDt, p0 - a0, p1 - a1);
            }
            // (where the scores of these 32 tokens were)
            tmem_write16(at + 32 * h, hi);
            tmem_write16(at + 32 * h + 16, lo);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
          tc::tc_fence_before();
          if (!dead) mbar_arrive(&p_full[x][buf]);
          some = true;
          ++count;
        }
        if (!end) a.next(P);
      }
      // the streams meet: each half of the threads joins half of the columns
      if (some) wait(&s_free[x][count - 1 & 1], count - 1 >> 1 & 1);
      s_stat[unit & 1][x][row] = make_float2(m - kUp, dead ? __int_as_float(0x7FFFFFFF) : l);
      named_bar_sync(1, 256);
      tc::tc_fence_after();
      const float2 st0 = s_stat[unit & 1][0][row], st1 = s_stat[unit & 1][1][row];
      const float top = fmaxf(st0.x, st1.x), base = attend_base(top);
      const float f0 = exp2_fast(st0.x - base), f1 = exp2_fast(st1.x - base), sum = fmaf(st0.y, f0, st1.y * f1);
      const bool from_start = chunk0 == 0, whole = from_start && a.chunk + 1 == a.s.chunks;
      const bool odd = s_odd[unit % kOddUnits] == (uint32_t)unit + 1u;
      const long long slot = 2 * blockIdx.x + (from_start ? 1 : 0);
      const int h = a.head * P.G + r - j * P.G;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
      for (int c = x * (DP / 2); c < (x + 1) * (DP / 2); c += 16) {
        uint32_t o0[16], o1[16];
        tmem_read16(tmem + lanes + kOut + c, o0);
        if (other) tmem_read16(tmem + lanes + kOut + DP + c, o1);
        float v[16], finite = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          v[e] = __uint_as_float(o0[e]) * f0;
          if (other) v[e] = fmaf(__uint_as_float(o1[e]), f1, v[e]);
          finite = fmaf(v[e], 0.f, finite);
        }
        const int end_at = min(a.s.len, (a.chunk + 1) * 2 * kTok);
        if (__any_sync(kAll, t >= 0 && finite != 0.f)) {  // (NaN then)
          // the warp looks through its columns, two lanes a token
          const int first = chunk0 * 2 * kTok + (lane >> 1), at = c + 8 * (lane & 1);
          uint32_t bits = 0u;
          if (at < P.D) bits = attend_odd<F16>(P, a.b, a.head, first, 16, min(end_at, attend_common(P, a.s)), at);
          __syncwarp();
          bits = __reduce_or_sync(kAll, bits << (16 * (lane & 1)));
#pragma unroll
          for (int e = 0; e < 16; ++e) attend_put_odd(v[e], bits >> (2 * e));
        }
        if (t >= 0 && c < P.D) {
          if (odd) {
            // what was taken out of the tiles, for the rows that see it
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              if (c + e >= P.D) break;
              const float4 x = attend_own<F16>(P, a.b, a.head, a.s.len - a.s.n, t, j,
                                               max(attend_common(P, a.s), chunk0 * 2 * kTok), end_at, c + e);
              attend_add_odd(v[e], x.x);
              attend_add_odd(v[e + 1], x.y);
              attend_add_odd(v[e + 2], x.z);
              attend_add_odd(v[e + 3], x.w);
            }
          }
          if (whole) {
            const long long to = t * P.o_stride + h * P.o_head + c;
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = sum == 0.f ? 0.f : v[e] * inv;
            if (P.o_vec && c + 16 <= P.D) {
#pragma unroll
              for (int e = 0; e < 16; e += 4) elem_store4(P.out, P.out_dtype, to + e, v + e);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (c + e < P.D) elem_store(P.out, P.out_dtype, to + e, v[e]);
            }
          } else {
            // four columns of all rows lie together: the lanes' rows are neighbours
            float4* const to = reinterpret_cast<float4*>(P.part) + (slot * (DP / 4) + c / 4) * 128 + row;
#pragma unroll
            for (int e = 0; e < 4; ++e) to[128 * e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          }
        }
        __syncwarp();  // (the next columns are read by whole warps)
      }
      tc::tc_fence_before();
      if (!dead) mbar_arrive(&o_free);
      if (x == 0 && t >= 0) {
        if (!whole)
          P.stat[slot * 128 + row] = make_float2(top, sum);
        else if (P.lse)
          P.lse[(long long)t * P.Hq + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
      }
      ++unit;
      a.next(P);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (s_gone)  // copies and products that are under way end by themselves, in microseconds
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  if (warp == 0) {
    tc::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the parts of a unit, as k_attend_join does.  An item is 8 rows of 16 columns:
// lane 8 q + r has row r, columns 4 q .. 4 q + 3.  With few parts a warp an item, else
// all warps of a block.
constexpr int kJoinWarps = 8, kJoinShare = 16, kFew = 6;
__global__ void __launch_bounds__(32 * kJoinWarps) k_attend_join_wide(const __grid_constant__ AttendParams P) {
  __shared__ float4 s_o[kJoinWarps][32];
  __shared__ float s_l[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x;
  pdl_wait();
  const AttendFrom at = P.from[c];
  if (at.none) attend_none<kJoinWarps>(P);
  if (at.parts == 0) return;
  const int c0 = at.first, parts = at.parts, c1 = c0 + parts - 1;
  const int rows = min(at.n * P.G - at.tile * P.rows, P.rows), groups = (P.D + 15) / 16, items = (rows + 7) / 8 * groups;
  const bool together = parts > kFew;
  const int worker = (c - c0 - 1) * kJoinShare + blockIdx.y, workers = (parts - 1) * kJoinShare;
  const int quads = P.width / 4;
  for (int i = together ? worker : worker * kJoinWarps + warp; i < items; i += together ? workers : workers * kJoinWarps) {
    const int r = i / groups * 8 + (lane & 7), q = i % groups * 4 + (lane >> 3);
    auto slot_of = [&](int p) { return (long long)(p == c0 ? 2 * c0 + 1 : 2 * p); };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (together) {
#pragma unroll 4
      for (int p = c0; p <= c1; ++p) m = fmaxf(m, P.stat[slot_of(p) * 128 + r].x);
    }
    // kFew parts at a time; no more: all of them, their maximum is found on the way
    const int step = together ? kJoinWarps : 1;
#pragma unroll 1
    for (int p0 = c0 + (together ? warp : 0); p0 <= c1; p0 += kFew * step) {
      float2 st[kFew];
      float4 a[kFew];
#pragma unroll
      for (int u = 0; u < kFew; ++u) {
        if (p0 + u * step > c1) break;
        const long long slot = slot_of(p0 + u * step);
        st[u] = P.stat[slot * 128 + r];
        a[u] = reinterpret_cast<const float4*>(P.part)[(slot * quads + q) * 128 + r];
      }
      if (!together) {
#pragma unroll
        for (int u = 0; u < kFew; ++u)
          if (p0 + u <= c1) m = fmaxf(m, st[u].x);
      }
      const float base = attend_base(m);
#pragma unroll
      for (int u = 0; u < kFew; ++u) {
        if (p0 + u * step > c1) break;
        const float f = exp2_fast(st[u].x - base);
        l = fmaf(st[u].y, f, l);
        o.x = fmaf(a[u].x, f, o.x);
        o.y = fmaf(a[u].y, f, o.y);
        o.z = fmaf(a[u].z, f, o.z);
        o.w = fmaf(a[u].w, f, o.w);
      }
    }
    if (together) {
      s_o[warp][lane] = o;
      s_l[warp][lane] = l;
      __syncthreads();
      if (warp == 0) {
#pragma unroll 1
        for (int w = 1; w < kJoinWarps; ++w) {
          const float4 a = s_o[w][lane];
          l += s_l[w][lane];
          o.x += a.x, o.y += a.y, o.z += a.z, o.w += a.w;
        }
      }
      __syncthreads();
      if (warp > 0) continue;
    }
    if (r >= rows) continue;
    if (!attend_finite(o)) {
      float4 odd = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int p = c0; p <= c1; ++p)
        attend_part_odd(odd, reinterpret_cast<const float4*>(P.part)[(slot_of(p) * quads + q) * 128 + r]);
      attend_take_odd(o, odd);
    }
    const int in = at.tile * P.rows + r, j = in / P.G, h = at.head * P.G + in - j * P.G, d = 4 * q;
    const long long t = at.t0 + j, out = t * P.o_stride + h * P.o_head + d;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    float y[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    if (l == 0.f) y[0] = y[1] = y[2] = y[3] = 0.f;
    if (d < P.D) {
      if (P.o_vec) {
        elem_store4(P.out, P.out_dtype, out, y);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) elem_store(P.out, P.out_dtype, out + e, y[e]);
      }
    }
    if (q == 0 && P.lse) P.lse[t * P.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <bool F16, int DP>
cudaError_t launch(const AttendParams& p, cudaStream_t stream) {
  static_assert(wide_smem(DP) + 4096 + 2048 <= 232448, "shared memory");
  auto* const kern = k_attend_wide<F16, DP>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), wide_smem(DP));
  if (e != cudaSuccess) return e;
  return launch_behind(kern, dim3(p.blocks), kThreads, wide_smem(DP), stream, p);
}

}  // namespace

cudaError_t launch_attend_wide(AttendParams p, cudaStream_t stream) {
  // q as (column, head, token), a box the rows of a unit
  if (p.q_vec && 2 * p.q_stride < 1ll << 40 && 2 * p.q_head < 1ll << 40) {
    const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.Hq, (cuuint64_t)p.T};
    const cuuint64_t strides[2] = {(cuuint64_t)(2 * p.q_head), (cuuint64_t)(2 * p.q_stride)};
    const cuuint32_t tokens = p.rows / p.G, box[3] = {64, (cuuint32_t)p.G, tokens}, ones[3] = {1, 1, 1};
    if (tensor_map_encoder()(&p.tm_q, p.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                             const_cast<uint16_t*>(p.q), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
      p.q_box = (int)tokens;
  }
  const cudaError_t e = p.f16 ? p.D <= 64 ? launch<true, 64>(p, stream) : launch<true, 128>(p, stream)
                        : p.D <= 64 ? launch<false, 64>(p, stream)
                                    : launch<false, 128>(p, stream);
  if (e != cudaSuccess) return e;
  return launch_behind(k_attend_join_wide, dim3(p.blocks, kJoinShare), 32 * kJoinWarps, 0, stream, p);
}

}  // namespace moe

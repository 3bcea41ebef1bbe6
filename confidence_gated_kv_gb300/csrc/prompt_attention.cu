// Attention of packed prompts: for every sequence its last lq tokens attend
// to its lk keys, with grouped heads and a causal mask aligned to the end.
//
//   out_i = sum_j softmax_j(scale q_i . k_j) v_j     over the j that row i sees
//   lse_i = log sum_j exp(scale q_i . k_j)
//
// A work item is one KV head and two tiles of 128 score rows.  The rows of a
// tile are (token, query head of the group): all G heads of 128 / G
// consecutive tokens, so that K and V are read once for the whole group and
// one token of a decode step still shares one tile.  K and V stream through
// a ring of shared-memory tiles of 128 keys.
//
// Roles of a CTA's 12 warps: a softmax warpgroup per row tile (a thread per
// row), a warp per row tile that issues the products, one for the copies and
// one that finds the next item.  A CTA takes over the items of CTAs that have
// not started (the copies of the next item run behind the last tiles of the
// current one); with few items the keys of an item are split over a cluster
// of CTAs instead, which merge their parts through distributed shared memory.
//
// What bounds it: the chain of a tile, from its scores through the softmax
// (about 1500 cycles, 700 of them the exponentials) and both products (1024)
// to the next scores; two of them interleave and keep the tensor cores busy
// for 70 % of the time.  Measured (bf16, 40 query heads on 8, d = 128): one
// prompt of 16384 tokens 1.92 ms, 1.43 PFLOP/s; eight prompts of 1 to 2047
// tokens 99 us; single tokens of eight sequences on 15 216 keys 25 us: every
// item is split in two, so the longest histories set the time.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <climits>
#include <cmath>

#include "../../include/confkv.h"
#include "confkv_internal.cuh"
#include "fp32_pair.cuh"
#include "tcgen05.cuh"

namespace cg = cooperative_groups;

namespace confkv {
namespace {

using namespace tc;

constexpr int kRows = 128;               // score rows per tile
constexpr int kKeys = 128;               // keys per tile
constexpr int kThreads = 384;            // two softmax warpgroups, one for copies and products

// Weights in the inputs' type: exp2(scores - reference + kLift).  The
// reference moves when a score passes it by more than kLag bits, so a weight
// stays below 2^(kLift + kLag).  bf16 has the exponents of fp32.  fp16 ends at
// 2^-24: unlifted, a weight 17 nats below the row's largest one is zero, and
// with it thousands of keys behind a dominating one.  Lifted by 11 bits it
// keeps all of its own down to 17 nats and is off by at most 2^-36 of the
// largest weight below; 2^15 leaves a factor of two to the end of the type.
// The closer reference costs rescalings (fp16, 16384 tokens of 40 heads:
// 1828 us with a lift of 7 and a lag of 8, 1865 with 11 and 4, 1896 with 13
// and 2).
template <bool BF16>
struct Weights {
  static constexpr float kLift = BF16 ? 0.f : 11.f, kLag = BF16 ? 8.f : 4.f;
  static constexpr float kUnlift = BF16 ? 1.f : 1.f / 2048.f;      // 2^-kLift
};

constexpr int kRegs = 168;               // registers a thread at launch: 65536 / 384, in eights
constexpr int kSMs = 152;
constexpr int kMaxSplit = 8;             // CTAs of a cluster that share an item

template <int D, bool SPLIT>
struct Tile {
  static constexpr int kBytes = kRows * D * 2;         // a Q, K or V tile
  // K and V tiles in flight; a split item needs room for the merge
  static constexpr int kStages = (D == 128 ? 5 : 8) - (SPLIT ? 1 : 0);
  static constexpr int kMerge = SPLIT ? 2 * kRows * 8 : 0;
  static constexpr int kSmem = (2 + kStages) * kBytes + kMerge + 1024;
  static constexpr int kPitch = D + 4;                 // floats per row of a part
  static_assert(!SPLIT || 2 * kRows * kPitch * 4 <= (2 + kStages) * kBytes, "a part fits the tiles' place");
};

struct Args {
  int B, Hq, Hkv, G, tokens;             // tokens: per 128-row tile
  int split;                             // CTAs per item
  int item0;                             // first item of the launch
  int causal;
  int total_q, total_k;
  const int32_t* cu_q;
  const int32_t* cu_k;
  uint16_t* out;
  long long out_token, out_head;
  float* lse;
  float scale, scale2;                   // scale2 = scale * log2(e)
  int wide;                              // rows of out start on 32-byte boundaries
  int absent;                            // CTA whose softmax warps do nothing (self-test), or -1
  long long limit;                       // cycles after which a wait gives up
};

struct Item {                            // what one CTA computes
  int found;                             // 0: no more work
  int q0, lq, k0, lk;                    // packed rows and lengths of the sequence
  int t0, head;                          // first token (within the sequence), KV head
  int first;                             // first key tile (of a split item)
  int n0, n1;                            // key tiles of each row tile, from `first` on
  int dual;                              // one row tile for both warpgroups, which take every other key tile
};

// Key tiles of an item.
__device__ __forceinline__ int key_tiles(const Item& it) { return it.dual ? it.n0 + it.n1 : max(it.n0, it.n1); }

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// Where a search for an item got to: the first sequence of a group and the
// tiles before it.  A CTA's items mostly follow each other.
struct Search {
  int b0 = 0, before = 0;
};

// Sequence and tile of work item `tile`, by one warp, W sequences per lane at
// a time (one where that is enough: the CTA's next item waits for this; with
// four for every batch the eight ragged prompts took 104 us instead of 99).
// Lengths are clamped to the packed tensors, so no array content
// leads out of them.  CTA `rank` of `split` takes its share of the item's key
// tiles.
template <int W>
__device__ __forceinline__ bool find_in_groups(const Args& a, int tile, int head, int rank, int split, Search& at, Item* it) {
  const int lane = threadIdx.x & 31;
  const int per = 2 * a.tokens;
  if (tile < at.before) at = Search{};
  for (; at.b0 < a.B; at.b0 += 32 * W) {
    const int b = at.b0 + lane * W;
    int q[W + 1], k[W + 1], tiles[W], own = 0;
#pragma unroll
    for (int i = 0; i <= W; ++i) {
      q[i] = a.cu_q[min(b + i, a.B)];
      k[i] = a.cu_k[min(b + i, a.B)];
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int q0 = clampi(q[i], 0, a.total_q);
      tiles[i] = b + i < a.B ? (clampi(q[i + 1], q0, a.total_q) - q0 + per - 1) / per : 0;
      own += tiles[i];
    }
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    int start = at.before + sum - own;
    bool mine = false;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (tile >= start && tile < start + tiles[i]) {
        mine = true;
        const int q0 = clampi(q[i], 0, a.total_q), lq = clampi(q[i + 1], q0, a.total_q) - q0;
        const int k0 = clampi(k[i], 0, a.total_k), lk = clampi(k[i + 1], k0, a.total_k) - k0;
        const int t0 = (tiles[i] - 1 - (tile - start)) * per;     // the longest rows first
        it->q0 = q0; it->lq = lq; it->k0 = k0; it->lk = lk;
        it->t0 = t0; it->head = head;
        const int mid = min(t0 + a.tokens, lq), end = min(t0 + per, lq);
        const int seen0 = a.causal ? clampi(lk - lq + mid, 0, lk) : lk;
        const int seen1 = a.causal ? clampi(lk - lq + end, 0, lk) : lk;
        const int n0 = (seen0 + kKeys - 1) / kKeys, n1 = end > mid ? (seen1 + kKeys - 1) / kKeys : 0;
        const int n = max(n0, n1), from = n * rank / split, to = n * (rank + 1) / split;
        it->first = from;
        it->dual = split > 1 && end == mid;
        it->n0 = it->dual ? (to - from + 1) / 2 : clampi(n0 - from, 0, to - from);
        it->n1 = it->dual ? (to - from) / 2 : clampi(n1 - from, 0, to - from);
      }
      start += tiles[i];
    }
    if (__any_sync(0xffffffffu, mine)) return true;
    at.before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

__device__ __forceinline__ bool find_item(const Args& a, int tile, int head, int rank, int split, Search& at, Item* it) {
  return a.B <= 32 ? find_in_groups<1>(a, tile, head, rank, split, at, it)
                   : find_in_groups<4>(a, tile, head, rank, split, at, it);
}

__device__ int32_t g_prompt_status;      // one word per device: a bounded wait gave up

constexpr long long kWaitLimit = 1LL << 33;     // about four seconds
constexpr long long kTestLimit = 1LL << 20;     // of the self-test: half a millisecond

// Bounded wait; false once it, or another wait of the CTA, has given up.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort, long long limit) {
  if (bar_try(bar, parity)) return true;
  const long long start = clock64();
  do {
    if (bar_try(bar, parity)) return true;
    if (*abort) return false;
  } while (clock64() - start < limit);
  *abort = 1;
  atomicOr(&g_prompt_status, kStatusTimeout);
  return false;
}

template <int D, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                            const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Args a) {
  using T = Tile<D, SPLIT>;
  using W = Weights<BF16>;
  constexpr int kBytes = T::kBytes, kStages = T::kStages;
  constexpr int kHalf = kRows * 128;                    // one 64-channel column block of a tile
  constexpr uint32_t kTmem = 512, kOut = 256;           // scores at 0 and 128, outputs from 256
  constexpr int kReaders = 11;                          // warps that read an item besides the one that finds it
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) uint8_t s_taken[16];
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 20];
  __shared__ Item s_item[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
  const uint32_t sq = smem_addr(smem), skv = sq + 2 * kBytes;
  const uint32_t bar0 = smem_addr(s_bar);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
  const uint32_t rest = bar0 + 16u * kStages;
  auto q_full = [&](int w) { return rest + 8u * w; };
  auto q_empty = [&](int w) { return rest + 16u + 8u * w; };
  auto s_full = [&](int w) { return rest + 32u + 8u * w; };
  auto p_full = [&](int w) { return rest + 48u + 8u * w; };
  auto o_full = [&](int w) { return rest + 64u + 8u * w; };
  auto drained = [&](int w) { return rest + 80u + 8u * w; };
  auto v_last = [&](int i) { return rest + 96u + 8u * (i & 1); };
  auto item_full = [&](int k) { return rest + 112u + 8u * (k & 1); };
  auto item_empty = [&](int k) { return rest + 128u + 8u * (k & 1); };
  const uint32_t taken = rest + 144u, copied = rest + 152u;

  if (warp == 8) tmem_alloc(smem_addr(&s_tmem), kTmem);
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < kStages; ++s) {
      bar_init(full(s), 1);
      bar_init(empty(s), 2);
    }
    for (int w = 0; w < 2; ++w) {
      bar_init(q_full(w), 1);
      bar_init(q_empty(w), 1);
      bar_init(s_full(w), 1);
      bar_init(p_full(w), kRows);
      bar_init(o_full(w), 1);
      bar_init(drained(w), 1);
      bar_init(v_last(w), 1);
      bar_init(item_full(w), 1);
      bar_init(item_empty(w), kReaders);
    }
    bar_init(taken, 1);
    bar_init(copied, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  // what the CTA starts with, while the barriers are set up; nothing before
  // this point touches memory that the previous kernel may write
  pdl_wait();
  const int split = SPLIT ? a.split : 1, rank = SPLIT ? blockIdx.x % split : 0;
  Search search;
  if (warp == 10) {
    const int index = a.item0 + blockIdx.x / split;     // an item per CTA, or per cluster
    const bool found = find_item(a, index / a.Hkv, index % a.Hkv, rank, split, search, &s_item[0]);
    if (lane == 0) s_item[0].found = found;
  }
  fence_before();
  if (SPLIT)
    cg::this_cluster().sync();                          // the other CTAs' shared memory is there
  else
    __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;

  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_on(bar, parity, &s_abort, a.limit); };
  auto all = [&](uint32_t bar, uint32_t parity) { return (bool)__all_sync(0xffffffffu, wait(bar, parity)); };
  // Item k of this CTA, by a whole warp; false at the end of the work.
  auto get_item = [&](int k, Item& it) {
    if (k > 0 && !all(item_full(k), (k - 1) >> 1 & 1)) return false;   // item 0 is there from the start
    it = s_item[k & 1];
    __syncwarp();
    if (lane == 0) bar_arrive(item_empty(k));
    return it.found != 0;
  };
  // Every role ends here before it looks at s_abort: whichever wait gave up,
  // all of them then see it, and wait for what they still have in flight.
  auto leave = [&] {
    __syncwarp();
    bar_sync<1>(kThreads);
  };
  float ref = -INFINITY, l = 0.f;                       // softmax threads: the latest item's row
  bool in_item = false;

  if (warp >= 8) {
    regs_dec<80>();
    if (warp == 8 || warp == 11) {
      // ---------------------------------------------------------- products
      // A warp per row tile: a warp that has issued products goes on to its
      // next wait only when they are done, so one warp for both tiles leaves
      // the tensor cores idle between them.  The whole warp runs the role,
      // one lane issues.
      constexpr uint32_t dqk = mma_desc(kRows, kKeys, BF16, false), dpv = mma_desc(kRows, D, BF16, true);
      const int w = warp == 11;
      const uint32_t scores = tmem + w * kKeys, output = tmem + kOut + w * D;
      uint32_t q = 0;
      auto issue_s = [&](int stage) {
        const uint32_t k = desc_lo(skv + stage * kBytes, 16);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t off = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
          mma_ss(scores, q + off, k + off, desc_hi(1024), dqk, i > 0);
        }
        mma_commit(s_full(w));
        mma_commit(empty(stage));
      };
      auto issue_o = [&](int stage, bool accumulate) {
        const uint32_t v = desc_lo(skv + stage * kBytes, kHalf);
#pragma unroll
        for (int i = 0; i < kKeys / 16; ++i)
          mma_ts(output, scores + 8 * i, v + i * (2048 >> 4), desc_hi(1024), dpv, accumulate || i > 0);
        mma_commit(empty(stage));
      };
      bool ok = true;
      int stage = -1;                                   // the latest tile of the ring and its parity
      uint32_t parity = 0;
      auto next_full = [&] {
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1;
        }
        ok = ok && all(full(stage), parity);
      };
      auto skip = [&](int tiles) {                      // tiles that only the other warp uses
        for (int i = 0; i < 2 * tiles && ok; ++i) {
          next_full();
          if (ok && lane == 0) bar_arrive(empty(stage));
        }
      };
      uint32_t tiles = 0, items = 0;                    // done by this warp: parities of its barriers
      Item it;
      for (int k = 0; ok && get_item(k, it); ++k) {
        const int nw = w ? it.n1 : it.n0;
        const bool dual = SPLIT && it.dual;
        const int wq = dual ? 0 : w;                    // the row tile
        q = desc_lo(sq + wq * kBytes, 16);
        int passed = 0;                                 // key tiles
        if (nw > 0) {
          if (dual && w) {
            skip(1);
            passed = 1;
          }
          next_full();
          ok = ok && all(q_full(wq), items & 1);
          if (ok) {
            fence_after();
            if (elect()) {
              issue_s(stage);
              if (nw == 1) mma_commit(q_empty(w));
            }
            __syncwarp();
          }
        }
        for (int j = 0; j < nw && ok; ++j) {
          next_full();                                  // V of this tile
          const int v = stage;
          const bool more = j + 1 < nw;
          ++passed;
          if (more && !dual) next_full();               // K of the next one
          ok = ok && all(p_full(w), (tiles + j) & 1);
          if (!ok) break;
          fence_after();
          if (elect()) {
            issue_o(v, j > 0);
            if (!more) mma_commit(o_full(w));
            if (more && !dual) {
              issue_s(stage);
              if (j + 2 == nw) mma_commit(q_empty(w));
            }
          }
          __syncwarp();
          if (more && dual) {
            skip(1);
            ++passed;
            next_full();
            if (ok && elect()) issue_s(stage);
            __syncwarp();
          }
        }
        skip(key_tiles(it) - passed);
        tiles += nw;
        items += nw > 0;
      }
      leave();
      if (s_abort && elect()) {                         // nothing in flight when the CTA ends
        mma_commit(drained(w));
        bar_wait(drained(w), 0);
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- copies
      const int q_bytes = a.tokens * a.G * D * 2;
      int count = 0, lasts = 0;                         // K and V tiles copied, v_last barriers used
      uint32_t held = 0;                                // bit i: the copy i before the latest is on v_last
      uint32_t queries[2] = {0, 0};
      bool ok = true;
      Item it;
      for (int k = 0; ok && get_item(k, it); ++k) {
        const int n = key_tiles(it);
        const bool partial = (it.first + n) * kKeys > it.lk;     // the last tile ends behind the sequence
        if (lane == 0) {
          auto load_q = [&](int w) {
            if ((w ? it.n1 : it.n0) == 0 || (w && it.dual)) return;
            uint32_t& used = w ? queries[1] : queries[0];
            if (used > 0) ok = ok && wait(q_empty(w), (used - 1) & 1);
            if (!ok) return;
            ++used;
            bar_expect(q_full(w), q_bytes);
            for (int c = 0; c < D / 64; ++c)
              tma_load(sq + w * kBytes + c * kHalf, &map_q, c * 64, it.head * a.G, it.q0 + it.t0 + w * a.tokens,
                       q_full(w));
          };
          load_q(0);
          for (int i = 0; i < 2 * n && ok; ++i) {
            const int s = count % kStages;
            if (count >= kStages) ok = wait(empty(s), (count / kStages - 1) & 1);
            if (!ok) break;
            const bool last = partial && i == 2 * n - 1;
            const uint32_t bar = last ? v_last(lasts++) : full(s);
            bar_expect(bar, kBytes);
            for (int c = 0; c < D / 64; ++c)
              tma_load(skv + s * kBytes + c * kHalf, i & 1 ? &map_v : &map_k, c * 64, it.head,
                       it.k0 + (it.first + (i >> 1)) * kKeys, bar);
            held = held << 1 | last;
            ++count;
            if (i == 0) load_q(1);
          }
          bar_arrive(copied);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      leave();
      if (s_abort && lane == 0) {
        for (int w = 0; w < 2; ++w)
          if (queries[w]) bar_wait(q_full(w), (queries[w] - 1) & 1);
        for (int i = 0; i < min(count, kStages); ++i)
          if (!(held >> i & 1)) bar_wait(full((count - 1 - i) % kStages), ((count - 1 - i) / kStages) & 1);
        for (int i = max(0, lasts - 2); i < lasts; ++i) bar_wait(v_last(i), (i >> 1) & 1);
      }
    } else {
      // ------------------------------------------ items and the last V tile
      Item it = s_item[0];
      auto publish = [&](int k, int index) {            // index: the CTA taken over, -1 for none
        if (k >= 2 && !all(item_empty(k), ((k >> 1) - 1) & 1)) return false;
        index += a.item0;
        const bool found =
            index >= a.item0 && find_item(a, index / a.Hkv, index % a.Hkv, rank, split, search, &s_item[k & 1]);
        __syncwarp();
        if (lane == 0) {
          s_item[k & 1].found = found;
          bar_arrive(item_full(k));
        }
        __syncwarp();
        it = s_item[k & 1];
        return found;
      };
      int lasts = 0, stage = 0;                         // partial tiles cleared, ring position of the item
      bool more = it.found != 0;
      for (int k = 0; more; ++k) {
        const Item now = it;
        const int n = key_tiles(now);
        int index = -1;
        if (!SPLIT) {
          // Once the last copies of this item are issued: early enough for
          // the next ones to follow them, and no item is held by a CTA that
          // is long busy with another one.
          if (!all(copied, k & 1)) break;
          if (lane == 0) {
            take_cta(smem_addr(s_taken), taken);
            bar_wait(taken, k & 1);
          }
          __syncwarp();
          index = all(taken, k & 1) ? taken_cta(smem_addr(s_taken)) : -1;
          __syncwarp();
        }
        more = publish(k + 1, index);
        stage = (stage + 2 * n) % kStages;              // behind this item's last tile
        if (n > 0 && (now.first + n) * kKeys > now.lk) {
          // The last key tile also holds rows behind the sequence: of the
          // next one, whatever they are.  Their weights are zero, but zero
          // times an infinity or NaN is not: those rows of V are cleared
          // before the tile is passed on.
          const int s = (stage + kStages - 1) % kStages;
          const uint32_t bar = v_last(lasts);
          if (!all(bar, (lasts >> 1) & 1)) break;
          ++lasts;
          const int first = now.lk - (now.first + n - 1) * kKeys;
          for (int c = 0; c < D / 64; ++c)
            for (int i = first * 8 + lane; i < kKeys * 8; i += 32)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(skv + s * kBytes + c * kHalf + i * 16),
                           "r"(0)
                           : "memory");
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
          if (lane == 0) bar_arrive(full(s));
        }
      }
      leave();
    }
    // All warps go on with the launch's register count.  The softmax warps
    // give theirs back before they leave: without that barrier, warps that
    // have nothing to do could take registers that a softmax warpgroup has
    // yet to ask for, and both would wait for ever.
    __syncwarp();
    regs_inc<kRegs>();
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<208>();
    const int w = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + w * kKeys + lane_base, to = tmem + kOut + w * D + lane_base;
    uint32_t tiles = 0, items = 0;                      // done by this warpgroup: parities of its barriers
    bool ok = (int)blockIdx.x != a.absent;
    Item it;
    for (int k = 0; ok && get_item(k, it); ++k) {
      const int nw = w ? it.n1 : it.n0;                 // key tiles of this row tile
      const bool dual = SPLIT && it.dual;
      const int t0 = it.t0 + (dual ? 0 : w) * a.tokens; // first token of the row tile
      if (t0 >= it.lq) continue;
      const int t = t0 + row / a.G;
      const bool valid = row < a.tokens * a.G && t < it.lq;
      const int seen = !valid ? 0 : a.causal ? clampi(it.lk - it.lq + t + 1, 0, it.lk) : it.lk;
      ref = -INFINITY;                                  // reference of the exponentials, and their sum
      l = 0.f;
      for (int j = 0; j < nw; ++j) {
        ok = all(s_full(w), (tiles + j) & 1);
        if (!ok) break;
        fence_after();
        // keys of the tile that the row sees; a row that is not used needs no
        // mask (its weights reach nothing), and would cost its warp one
        const int left = valid ? seen - (it.first + (dual ? 2 * j + w : j)) * kKeys : kKeys;
        const int least = __reduce_min_sync(0xffffffffu, left);   // what every row of the warp sees
        uint32_t s[kKeys];
        float m[4] = {ref, ref, ref, ref};
        tmem_ld32(ts, s);
        wait_ld32(s);
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) {           // the maximum of a quarter while the next one loads
          if (c + 32 < kKeys) tmem_ld32(ts + c + 32, s + c + 32);
          if (least < c + 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c + i >= left) s[c + i] = 0xff800000u;
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            m[i / 2 % 4] = fmaxf(fmaxf(__uint_as_float(s[c + i]), __uint_as_float(s[c + i + 1])), m[i / 2 % 4]);
          if (c + 32 < kKeys) wait_ld32(s + c + 32);
        }
        const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
        // The reference moves only when it would be passed by more than
        // 2^kLag, so that the accumulator in tensor memory is rarely
        // rescaled.  The product that reads it is done: the scores of this
        // tile were issued after it.
        const bool move = valid && ((top - ref) * a.scale2 > W::kLag || ref == -INFINITY);
        if (__any_sync(0xffffffffu, move && j > 0 && top > ref)) {
          const float f = move && top > ref ? ex2((ref - top) * a.scale2) : 1.f;
          l *= f;
#pragma unroll
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld16(to + c, o);
            wait_ld16(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(to + c, o);
          }
        }
        if (move) ref = top;
        const float base = ref == -INFINITY ? 0.f : fmaf(-ref, a.scale2, W::kLift);
        const Pair scale_pair(a.scale2, a.scale2), base_pair(base, base);
        Pair sum[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) {           // a quarter of the weights at a time
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e =
                fma2(Pair(__uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1])), scale_pair, base_pair).get();
            const float x = ex2(e.x), y = ex2(e.y);
            sum[i & 1] = sum[i & 1] + Pair(x, y);
            p[i] = pack2<BF16>(x, y);
          }
          tmem_st16(ts + c / 2, p);
        }
        wait_st();
        fence_before();
        bar_arrive(p_full(w));
        const float2 both = (sum[0] + sum[1]).get();
        l += both.x + both.y;
      }
      tiles += nw;
      if (!ok) break;
      // What the last product does not bear on goes before its wait.
      uint16_t* dst = nullptr;
      float inv = 0.f;                                  // rows without a key are zero
      if (!SPLIT && valid) {
        const long long at = it.q0 + t;
        const int head = it.head * a.G + row % a.G;
        dst = a.out + at * a.out_token + head * a.out_head;
        inv = seen > 0 ? 1.f / l : 0.f;
        if (a.lse)
          a.lse[at * a.Hq + head] =
              seen > 0 ? (ref == -INFINITY ? 0.f : ref * a.scale) + logf(l * W::kUnlift) : -INFINITY;
      }
      if (nw > 0) {
        ok = all(o_full(w), items & 1);
        if (!ok) break;
        fence_after();
        ++items;
      }
      if (SPLIT) {
        in_item = true;
        continue;                                       // merged below
      }
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (nw > 0) {
          tmem_ld32(to + c, o);
          wait_ld32(o);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          o[i] = seen > 0 ? pack2<BF16>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv) : 0;
        if (valid) {
          if (a.wide) {
            st_global32(dst + c, o);
            st_global32(dst + c + 16, o + 8);
          } else {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<uint4*>(dst + c + 2 * i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        __syncwarp();
      }
      fence_before();                                   // the next product overwrites the accumulator
      __syncwarp();
    }
    __syncwarp();
    regs_dec<kRegs>();
    leave();
  }

  if (SPLIT) {
    // ---------------------------------------------------------------- merge
    // Every CTA leaves (reference, sum) and output of its rows in its shared
    // memory; each adds up the parts of its share of the rows.
    cg::cluster_group cluster = cg::this_cluster();
    float* part = reinterpret_cast<float*>(smem);       // [2 * kRows][kPitch], over the tiles
    float2* sums = reinterpret_cast<float2*>(smem + (2 + kStages) * kBytes);   // [2 * kRows]
    const Item it = s_item[0];
    __syncthreads();                                    // the products of both row tiles are done
    const bool done = it.found != 0 && !s_abort;
    // A CTA that gave up left no part: the rows become NaN for those that
    // would add it.
    if (threadIdx.x < 2 * kRows && it.found != 0 && s_abort) sums[threadIdx.x] = make_float2(-INFINITY, NAN);
    if (threadIdx.x < 2 * kRows && in_item && done) {
      const int w = warp >> 2, nw = w ? it.n1 : it.n0;
      sums[threadIdx.x] = make_float2(ref, l);
      const uint32_t to = tmem + kOut + w * D + ((uint32_t)(warp & 3) << 21);
      const int rows = min(a.tokens, it.lq - it.t0 - (it.dual ? 0 : w) * a.tokens) * a.G;
      if ((warp & 3) * 32 < rows) {                     // warps with a row that is used
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (nw > 0) {
            tmem_ld32(to + c, o);
            wait_ld32(o);
          }
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(part + threadIdx.x * T::kPitch + c + i) =
                nw > 0 ? make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]) : make_uint4(0, 0, 0, 0);
        }
      }
    }
    cluster.sync();
    if (done) {
      const int per = a.tokens * a.G;                   // rows of a tile that are used
      const int rows = min(2 * a.tokens, it.lq - it.t0) * a.G;
      constexpr int kLanes = D / 4;                     // per row: four channels each
      const int col = (lane % kLanes) * 4, group = threadIdx.x / kLanes;
      for (int i = rank + split * group; i < rows; i += split * (kThreads / kLanes)) {
        const int slot = i < per ? i : kRows + i - per, t = it.t0 + i / a.G;
        const int seen = a.causal ? clampi(it.lk - it.lq + t + 1, 0, it.lk) : it.lk;
        // the row's parts: one of each CTA, or with two warpgroups per row two
        float top = -INFINITY, sum = 0.f, x[4] = {};
        for (int at = slot; at < (it.dual ? 2 * kRows : slot + 1); at += kRows) {
          float4 y[kMaxSplit];
          float2 z[kMaxSplit];
#pragma unroll
          for (int r = 0; r < kMaxSplit; ++r)           // all parts in flight
            if (r < split) {
              y[r] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, r) + at * T::kPitch + col);
              z[r] = *(cluster.map_shared_rank(sums, r) + at);
            }
          const float before = top;
#pragma unroll
          for (int r = 0; r < kMaxSplit; ++r)
            if (r < split) top = fmaxf(top, z[r].x);
          const float old = before == top ? 1.f : ex2((before - top) * a.scale2);
          sum *= old;
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] *= old;
#pragma unroll
          for (int r = 0; r < kMaxSplit; ++r)
            if (r < split) {
              const float f = z[r].x == top ? 1.f : ex2((z[r].x - top) * a.scale2);
              sum += z[r].y * f;
              x[0] += y[r].x * f;
              x[1] += y[r].y * f;
              x[2] += y[r].z * f;
              x[3] += y[r].w * f;
            }
        }
        const float inv = 1.f / sum;
        const long long at = it.q0 + t;
        const int head = it.head * a.G + i % a.G;
        *reinterpret_cast<uint2*>(a.out + at * a.out_token + head * a.out_head + col) =
            seen > 0 ? make_uint2(pack2<BF16>(x[0] * inv, x[1] * inv), pack2<BF16>(x[2] * inv, x[3] * inv))
                     : make_uint2(0, 0);
        if (a.lse && col == 0)
          a.lse[at * a.Hq + head] =
              seen > 0 ? (top == -INFINITY ? 0.f : top * a.scale) + logf(sum * W::kUnlift) : -INFINITY;
      }
    }
    cluster.sync();                                     // no CTA leaves while another reads its part
  }
  fence_before();
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    fence_after();
    tmem_free(tmem, kTmem);
  }
}

// ---------------------------------------------------------------- host side

using EncodeFn = decltype(&cuTensorMapEncodeTiled);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// (channel, head, token) map of a packed tensor with boxes of 64 channels.
bool encode(CUtensorMap* m, const void* p, bool bf16, int d, long long heads, long long tokens, long long ts,
            long long hs, int box_heads, int box_tokens) {
  if (heads == 1) hs = d;                               // strides of single rows are never used
  if (tokens == 1) ts = hs * heads;
  const cuuint64_t dim[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t stride[2] = {(cuuint64_t)hs * 2, (cuuint64_t)ts * 2};
  const cuuint32_t box[3] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_tokens}, one[3] = {1, 1, 1};
  return encode_fn()(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                     const_cast<void*>(p), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16, bool SPLIT>
int launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, long long items,
           cudaStream_t st) {
  static int done[kMaxDevices] = {};
  auto kernel = prompt_attention_kernel<D, BF16, SPLIT>;
  constexpr int smem = Tile<D, SPLIT>::kSmem;
  if (ensure_smem(kernel, smem, done) != cudaSuccess) return CONFKV_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * a.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = a.split;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, a) == cudaSuccess ? CONFKV_OK : CONFKV_ECUDA;
}

template <int D, bool BF16>
int launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, long long items,
           cudaStream_t st) {
  return a.split > 1 ? launch<D, BF16, true>(mq, mk, mv, a, items, st)
                     : launch<D, BF16, false>(mq, mk, mv, a, items, st);
}

// How the items are launched, from what the host knows: the largest number of
// items and the average number of key tiles of a sequence.  Time is taken as
// rounds of the SMs times (key tiles of a CTA + the tiles that its start and
// its merge take: 3, or 4 with a merge, at about 1.7 us each; 2 more for a
// second launch).  Histories of unlike lengths are not seen: their items get
// the split of the mean, and the longest of them sets the time.  A
// last round with few items can go into a launch of its own whose keys are
// split (160 items of 117 tiles: 323 us with all of them split in two, 251 us
// as 152 whole ones and 8 split in eight).
struct Plan {
  long long whole, rest;                 // items of the first launch, and of one more
  int split, rest_split;
};

double rounds_cost(long long items, double tiles, int* split) {
  double least = 1e30;
  for (int s = 1; s <= kMaxSplit; s *= 2) {
    const double t = std::ceil((double)items * s / kSMs) * (std::ceil(tiles / s) + (s == 1 ? 3.0 : 4.0));
    if (t < least) {
      least = t;
      *split = s;
    }
  }
  return least;
}

Plan plan_items(long long items, double tiles) {
  Plan p{items, 0, 1, 1};
  if (items >= 4LL * kSMs) return p;     // enough rounds to even out
  const double one = rounds_cost(items, tiles, &p.split);
  const long long whole = items / kSMs * kSMs;
  if (whole > 0 && whole < items) {
    int split = 1;
    const double two = whole / kSMs * (tiles + 3.0) + rounds_cost(items - whole, tiles, &split) + 2.0;
    if (two < one) p = Plan{whole, items - whole, 1, split};
  }
  return p;
}

bool rows_ok(const void* p, const int64_t* stride, int d, long long tokens, long long heads) {
  if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  if (tokens > 1 && (stride[0] < d || stride[0] % 8 || stride[0] >= (1LL << 38))) return false;
  if (heads > 1 && (stride[1] < d || stride[1] % 8 || stride[1] >= (1LL << 38))) return false;
  return true;
}

// No two rows share an element.
bool rows_apart(const int64_t* stride, int d, long long tokens, long long heads) {
  return tokens < 2 || heads < 2 || stride[0] >= (heads - 1) * stride[1] + d ||
         stride[1] >= (tokens - 1) * stride[0] + d;
}

}  // namespace
}  // namespace confkv

using namespace confkv;

// test: the call of the self-test.
static int prompt_attention(const confkv_prompt_args* p, bool test, void* stream) {
  if (!p) return CONFKV_EINVAL;
  if (p->B < 1 || p->Hq < 1 || p->Hkv < 1 || p->total_q < 0 || p->total_k < 0) return CONFKV_EINVAL;
  constexpr int32_t most = INT32_MAX - 4096;             // a tile's end behind the last row fits 32 bits
  if (p->total_q > most || p->total_k > most || p->B > most) return CONFKV_EINVAL;
  if (p->Hq % p->Hkv || p->Hq / p->Hkv > kRows || p->reserved != 0) return CONFKV_EINVAL;
  if (p->dtype != CONFKV_Q_FP16 && p->dtype != CONFKV_Q_BF16) return CONFKV_EINVAL;
  if (p->d != 64 && p->d != 128) return CONFKV_ENOTIMPL;
  if (!std::isfinite(p->scale) || !(p->scale > 0.f)) return CONFKV_EINVAL;
  if (!p->cu_q || !p->cu_k || reinterpret_cast<uintptr_t>(p->cu_q) % 4 || reinterpret_cast<uintptr_t>(p->cu_k) % 4)
    return CONFKV_EINVAL;
  if (p->total_q == 0) return CONFKV_OK;
  if (!p->q || !p->out || (p->total_k > 0 && (!p->k || !p->v))) return CONFKV_EINVAL;
  if (!rows_ok(p->q, p->q_stride, p->d, p->total_q, p->Hq) ||
      !rows_ok(p->out, p->out_stride, p->d, p->total_q, p->Hq) ||
      !rows_apart(p->out_stride, p->d, p->total_q, p->Hq) ||
      !rows_ok(p->k, p->k_stride, p->d, p->total_k, p->Hkv) ||
      !rows_ok(p->v, p->v_stride, p->d, p->total_k, p->Hkv))
    return CONFKV_EINVAL;
  if (p->lse && reinterpret_cast<uintptr_t>(p->lse) % 4) return CONFKV_EINVAL;
  Args a{};
  a.B = p->B; a.Hq = p->Hq; a.Hkv = p->Hkv; a.G = p->Hq / p->Hkv;
  a.tokens = kRows / a.G;
  a.causal = p->causal != 0;
  a.total_q = p->total_q; a.total_k = p->total_k;
  a.cu_q = p->cu_q; a.cu_k = p->cu_k;
  a.out = static_cast<uint16_t*>(p->out);
  a.out_token = p->out_stride[0]; a.out_head = p->out_stride[1];
  a.lse = p->lse;
  a.scale = p->scale;
  a.scale2 = p->scale * 1.4426950408889634f;
  a.limit = test ? kTestLimit : kWaitLimit;
  // no more tiles than these, whatever the lengths
  const int per = 2 * a.tokens;
  const long long tiles = p->B == 1 ? (p->total_q + per - 1LL) / per : (long long)p->total_q / per + p->B;
  if (tiles * p->Hkv >= (1LL << 31) / kMaxSplit) return CONFKV_EINVAL;
  a.wide = reinterpret_cast<uintptr_t>(p->out) % 32 == 0 && (p->total_q < 2 || p->out_stride[0] % 16 == 0) &&
           (p->Hq < 2 || p->out_stride[1] % 16 == 0);
  const bool bf16 = p->dtype == CONFKV_Q_BF16;
  if (!encode_fn()) return CONFKV_ECUDA;
  CUtensorMap mq, mk, mv;
  // without keys no copy of K or V is issued: the maps are placeholders
  const bool keys = p->total_k > 0;
  if (!encode(&mq, p->q, bf16, p->d, p->Hq, p->total_q, p->q_stride[0], p->q_stride[1], a.G, a.tokens) ||
      !encode(&mk, keys ? p->k : p->q, bf16, p->d, keys ? p->Hkv : 1, keys ? p->total_k : 1, p->k_stride[0],
              p->k_stride[1], 1, kKeys) ||
      !encode(&mv, keys ? p->v : p->q, bf16, p->d, keys ? p->Hkv : 1, keys ? p->total_k : 1, p->v_stride[0],
              p->v_stride[1], 1, kKeys))
    return CONFKV_EINVAL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Plan plan = plan_items(tiles * p->Hkv, (double)p->total_k / p->B / kKeys);
  auto fn = p->d == 128 ? (bf16 ? launch<128, true> : launch<128, false>)
                        : (bf16 ? launch<64, true> : launch<64, false>);
  // The last CTA that shares the first item: it has a key tile if any has.
  a.absent = test ? plan.split - 1 : -1;
  a.split = plan.split;
  const int first = fn(mq, mk, mv, a, plan.whole, st);
  if (first != CONFKV_OK || plan.rest == 0) return first;
  a.item0 = (int)plan.whole;
  a.absent = -1;
  a.split = plan.rest_split;
  return fn(mq, mk, mv, a, plan.rest, st);
}

extern "C" int confkv_prompt_attention(const confkv_prompt_args* args, void* stream) {
  return prompt_attention(args, false, stream);
}

extern "C" int confkv_selftest_prompt_timeout(const confkv_prompt_args* args, void* stream) {
  return prompt_attention(args, true, stream);
}

extern "C" int confkv_prompt_status(int32_t* bits, void* stream) {
  if (!bits) return CONFKV_EINVAL;
  void* word = nullptr;
  if (cudaGetSymbolAddress(&word, g_prompt_status) != cudaSuccess) return CONFKV_ECUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int32_t host = 0;
  cudaError_t e = cudaMemcpyAsync(&host, word, 4, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && host) e = cudaMemsetAsync(word, 0, 4, st);
  if (e != cudaSuccess) return CONFKV_ECUDA;
  *bits = host;
  return host ? CONFKV_EDEVICE : CONFKV_OK;
}

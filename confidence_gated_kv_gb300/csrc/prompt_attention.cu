// Attention of packed prompts: for every sequence its last lq tokens attend
// to its lk keys, with grouped heads and a causal mask aligned to the end.
//
//   out_i = sum_j softmax_j(scale q_i . k_j) v_j     over the j that row i sees
//   lse_i = log sum_j exp(scale q_i . k_j)
//
// One CTA takes one KV head and two tiles of 128 score rows.  The rows of a
// tile are (token, query head of the group): all G heads of 128 / G
// consecutive tokens, so that K and V are read once for the whole group and
// one token of a decode step still shares one tile.  K and V stream through
// a ring of shared-memory tiles of 128 keys.
#include <cuda_runtime.h>
#include <cmath>
#include <cstring>
#include <mutex>

#include "../../include/confkv.h"
#include "confkv_internal.cuh"
#include "fp32_pair.cuh"
#include "tcgen05.cuh"

namespace confkv {
namespace {

using namespace tc;

constexpr int kRows = 128;               // score rows per tile
constexpr int kKeys = 128;               // keys per tile
constexpr int kThreads = 384;            // two softmax warpgroups, one for copies and products
constexpr int kPolls = 1 << 24;          // polls per wait (a few seconds at most)

template <int D>
struct Tile {
  static constexpr int kBytes = kRows * D * 2;         // a Q, K or V tile
  static constexpr int kStages = D == 128 ? 5 : 8;     // K and V tiles in flight
  static constexpr int kSmem = (2 + kStages) * kBytes + 1024;
};

struct Args {
  int B, Hq, Hkv, G, tokens;             // tokens: per 128-row tile
  int causal;
  int total_q, total_k;
  const int32_t* cu_q;
  const int32_t* cu_k;
  uint16_t* out;
  long long out_token, out_head;
  float* lse;
  float scale, scale2;                   // scale2 = scale * log2(e)
  int32_t* status;
};

struct Item {                            // what one CTA computes
  int q0, lq, k0, lk;                    // packed rows and lengths of the sequence
  int t0, head;                          // first token (within the sequence), KV head
  int n0, n1;                            // key tiles of each row tile
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// Sequence and tile of work item `tile`, by one warp.  Lengths are clamped to
// the packed tensors, so no array content leads out of them.
__device__ bool find_item(const Args& a, int tile, int head, Item* it) {
  const int lane = threadIdx.x & 31;
  const int per = 2 * a.tokens;
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    int q0 = 0, lq = 0;
    if (b < a.B) {
      q0 = clampi(a.cu_q[b], 0, a.total_q);
      lq = clampi(a.cu_q[b + 1], q0, a.total_q) - q0;
    }
    const int nt = (lq + per - 1) / per;
    int sum = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const bool mine = tile >= before + sum - nt && tile < before + sum;
    const unsigned hit = __ballot_sync(0xffffffffu, mine);
    if (hit) {
      if (mine) {
        const int k0 = clampi(a.cu_k[b], 0, a.total_k);
        const int lk = clampi(a.cu_k[b + 1], k0, a.total_k) - k0;
        const int t0 = (nt - 1 - (tile - (before + sum - nt))) * per;   // the longest rows first
        it->q0 = q0; it->lq = lq; it->k0 = k0; it->lk = lk;
        it->t0 = t0; it->head = head;
        const int mid = min(t0 + a.tokens, lq), end = min(t0 + per, lq);
        const int seen0 = a.causal ? clampi(lk - lq + mid, 0, lk) : lk;
        const int seen1 = a.causal ? clampi(lk - lq + end, 0, lk) : lk;
        it->n0 = (seen0 + kKeys - 1) / kKeys;
        it->n1 = end > mid ? (seen1 + kKeys - 1) / kKeys : 0;
      }
      return true;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

// Bounded wait; false once it, or another wait of the CTA, has given up.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
  for (int i = 0; i < kPolls; ++i) {
    if (bar_try(bar, parity)) return true;
    if (*abort) return false;
  }
  *abort = 1;
  atomicOr(status, kStatusTimeout);
  return false;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                            const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Args a) {
  constexpr int kBytes = Tile<D>::kBytes, kStages = Tile<D>::kStages;
  constexpr int kHalf = kRows * 128;                    // one 64-channel column block of a tile
  constexpr uint32_t kTmem = 512, kOut = 256;           // scores at 0 and 128, outputs from 256
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * Tile<D>::kStages + 13];
  __shared__ Item s_item;
  __shared__ uint32_t s_tmem;
  __shared__ int s_found;
  __shared__ volatile int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
  const uint32_t sq = smem_addr(smem), skv = sq + 2 * kBytes;
  const uint32_t bar0 = smem_addr(s_bar);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
  const uint32_t rest = bar0 + 16u * kStages;
  auto q_full = [&](int w) { return rest + 8u * w; };
  auto s_full = [&](int w) { return rest + 16u + 8u * w; };
  auto p_full = [&](int w, int half) { return rest + 32u + 16u * w + 8u * half; };
  auto o_full = [&](int w) { return rest + 64u + 8u * w; };
  const uint32_t v_last = rest + 80u;
  auto drained = [&](int w) { return rest + 88u + 8u * w; };

  if (warp == 8) tmem_alloc(smem_addr(&s_tmem), kTmem);
  if (warp == 9) {
    const bool found = find_item(a, blockIdx.x / a.Hkv, blockIdx.x % a.Hkv, &s_item);
    if (lane == 0) s_found = found;
  }
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < kStages; ++s) {
      bar_init(full(s), 1);
      bar_init(empty(s), 2);
    }
    for (int w = 0; w < 2; ++w) {
      bar_init(q_full(w), 1);
      bar_init(s_full(w), 1);
      bar_init(p_full(w, 0), kRows);
      bar_init(p_full(w, 1), kRows);
      bar_init(o_full(w), 1);
      bar_init(drained(w), 1);
    }
    bar_init(v_last, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  const bool found = s_found != 0;

  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_on(bar, parity, &s_abort, a.status); };

  if (warp >= 8) {
    regs_dec<80>();
    const Item it = s_item;
    const int n = found ? max(it.n0, it.n1) : 0;
    const bool partial = n * kKeys > it.lk;             // the last key tile ends behind the sequence
    if ((warp == 8 || warp == 11) && n > 0) {
      // ---------------------------------------------------------- products
      // A warp per row tile: a warp that has issued products goes on to its
      // next wait only when they are done, so one warp for both tiles leaves
      // the tensor cores idle between them.  The whole warp runs the role,
      // one lane issues.
      constexpr uint32_t dqk = mma_desc(kRows, kKeys, BF16, false), dpv = mma_desc(kRows, D, BF16, true);
      const int w = warp == 11, nw = w ? it.n1 : it.n0;
      const uint32_t scores = tmem + w * kKeys, output = tmem + kOut + w * D, q = desc_lo(sq + w * kBytes, 16);
      auto issue_s = [&](int stage) {
        const uint32_t k = desc_lo(skv + stage * kBytes, 16);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t off = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
          mma_ss(scores, q + off, k + off, desc_hi(1024), dqk, i > 0);
        }
        mma_commit(s_full(w));
      };
      auto issue_o = [&](int stage, int half, bool accumulate) {
        const uint32_t v = desc_lo(skv + stage * kBytes + half * (kHalf / 2), kHalf);
        const uint32_t p = scores + half * (kKeys / 4);
#pragma unroll
        for (int i = 0; i < kKeys / 32; ++i)
          mma_ts(output, p + 8 * i, v + i * (2048 >> 4), desc_hi(1024), dpv, accumulate || half > 0 || i > 0);
      };
      auto all = [&](uint32_t bar, uint32_t parity) { return (bool)__all_sync(0xffffffffu, wait(bar, parity)); };
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
      if (nw > 0) {
        next_full();
        ok = ok && all(q_full(w), 0);
        if (ok) {
          fence_after();
          if (elect()) {
            issue_s(0);
            mma_commit(empty(0));
          }
          __syncwarp();
        }
      }
      for (int j = 0; j < nw && ok; ++j) {
        next_full();                                    // V of this tile
        const int v = stage;
        if (j + 1 < nw) next_full();                    // K of the next one
        const int k = stage;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          ok = ok && all(p_full(w, half), j & 1);
          if (!ok) break;
          fence_after();
          if (elect()) {
            issue_o(v, half, j > 0);
            if (half) {
              if (j + 1 < nw) {
                issue_s(k);
                mma_commit(empty(k));
              } else {
                mma_commit(o_full(w));
              }
              mma_commit(empty(v));
            }
          }
          __syncwarp();
        }
      }
      for (int i = 2 * nw; i < 2 * n && ok; ++i) {      // tiles that only the other row tile sees
        next_full();
        if (ok && lane == 0) bar_arrive(empty(stage));
      }
      if (!ok && elect()) {                             // nothing in flight when the CTA ends
        mma_commit(drained(w));
        for (int i = 0; i < kPolls && !bar_try(drained(w), 0); ++i) {}
      }
    } else if (warp == 9 && lane == 0 && n > 0) {
      // ---------------------------------------------------------- copies
      const int q_bytes = a.tokens * a.G * D * 2;
      auto load_q = [&](int w) {
        if ((w ? it.n1 : it.n0) == 0) return;
        bar_expect(q_full(w), q_bytes);
        for (int c = 0; c < D / 64; ++c)
          tma_load(sq + w * kBytes + c * kHalf, &map_q, c * 64, it.head * a.G, it.q0 + it.t0 + w * a.tokens,
                   q_full(w));
      };
      int issued = 0;
      bool ok = true;
      load_q(0);
      for (int i = 0; i < 2 * n; ++i) {
        const int s = i % kStages;
        if (i >= kStages && !wait(empty(s), (i / kStages - 1) & 1)) { ok = false; break; }
        const uint32_t bar = partial && i == 2 * n - 1 ? v_last : full(s);
        bar_expect(bar, kBytes);
        for (int c = 0; c < D / 64; ++c)
          tma_load(skv + s * kBytes + c * kHalf, i & 1 ? &map_v : &map_k, c * 64, it.head, it.k0 + (i >> 1) * kKeys,
                   bar);
        ++issued;
        if (i == 0) load_q(1);
      }
      if (!ok) {
        for (int w = 0; w < 2; ++w)
          if (w ? it.n1 : it.n0)
            for (int i = 0; i < kPolls && !bar_try(q_full(w), 0); ++i) {}
        for (int j = max(0, issued - kStages); j < issued; ++j) {
          const bool last = partial && j == 2 * n - 1;
          for (int i = 0; i < kPolls && !bar_try(last ? v_last : full(j % kStages),
                                                       last ? 0 : (j / kStages) & 1); ++i) {}
        }
      }
    } else if (warp == 10 && n > 0 && partial) {
      // The last key tile also holds rows behind the sequence: of the next
      // one, whatever they are.  Their probabilities are zero, but zero times
      // an infinity or NaN is not: those rows of V are cleared before the
      // tile is passed on.
      const int s = (2 * n - 1) % kStages;
      if (__all_sync(0xffffffffu, wait(v_last, 0))) {
        const int first = it.lk - (n - 1) * kKeys;
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
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<208>();
    const Item it = s_item;
    const int w = warp >> 2, row = threadIdx.x & 127;
    const int nw = w ? it.n1 : it.n0;                   // key tiles of this row tile
    if (found && it.t0 + w * a.tokens < it.lq) {
      const int t = it.t0 + w * a.tokens + row / a.G;
      const bool valid = row < a.tokens * a.G && t < it.lq;
      const int seen = !valid ? 0 : a.causal ? clampi(it.lk - it.lq + t + 1, 0, it.lk) : it.lk;
      const uint32_t lane_base = (uint32_t)(warp & 3) << 21;
      const uint32_t ts = tmem + w * kKeys + lane_base, to = tmem + kOut + w * D + lane_base;
      float ref = -INFINITY, l = 0.f;                   // reference of the exponentials, their sum
      bool ok = true;
      for (int j = 0; j < nw; ++j) {
        ok = __all_sync(0xffffffffu, wait(s_full(w), j & 1));
        if (!ok) break;
        fence_after();
        const int left = seen - j * kKeys;              // keys of the tile that the row sees
        const bool masked = __any_sync(0xffffffffu, left < kKeys);
        uint32_t s[kKeys];
        float m[4] = {ref, ref, ref, ref};
        tmem_ld32(ts, s);
        wait_ld32(s);
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) {           // the maximum of a quarter while the next one loads
          if (c + 32 < kKeys) tmem_ld32(ts + c + 32, s + c + 32);
          if (masked) {
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
        // The reference moves only when it would be passed by more than 2^8:
        // the weights then stay below 2^8, and the accumulator in tensor
        // memory is rarely rescaled.  The product that reads it is done:
        // the scores of this tile were issued after it.
        const bool move = (top - ref) * a.scale2 > 8.f || ref == -INFINITY;
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
        const float base = ref == -INFINITY ? 0.f : -ref * a.scale2;
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
          if (c & 32) {                                 // the product starts with the first half
            wait_st();
            fence_before();
            bar_arrive(p_full(w, c / 64));
          }
        }
        const float2 both = (sum[0] + sum[1]).get();
        l += both.x + both.y;
      }
      if (ok && nw > 0) {
        ok = __all_sync(0xffffffffu, wait(o_full(w), 0));
        fence_after();
      }
      if (ok) {
        // Rows without a key are zero.  The row goes through the warp's own
        // part of the Q tile, so that the stores are whole rows.
        const float inv = seen > 0 ? 1.f / l : 0.f;
        uint8_t* stage = smem + w * kBytes;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (nw > 0) {
            tmem_ld32(to + c, o);
            wait_ld32(o);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (seen > 0) {
              x.x = pack2<BF16>(__uint_as_float(o[8 * i]) * inv, __uint_as_float(o[8 * i + 1]) * inv);
              x.y = pack2<BF16>(__uint_as_float(o[8 * i + 2]) * inv, __uint_as_float(o[8 * i + 3]) * inv);
              x.z = pack2<BF16>(__uint_as_float(o[8 * i + 4]) * inv, __uint_as_float(o[8 * i + 5]) * inv);
              x.w = pack2<BF16>(__uint_as_float(o[8 * i + 6]) * inv, __uint_as_float(o[8 * i + 7]) * inv);
            }
            const int chunk = (c & 63) / 8 + i;
            *reinterpret_cast<uint4*>(stage + (c >> 6) * kHalf + row * 128 + ((chunk ^ (row & 7)) << 4)) = x;
          }
        }
        if (a.lse && valid) {
          const float lse = seen > 0 ? (ref == -INFINITY ? 0.f : ref * a.scale) + logf(l) : -INFINITY;
          a.lse[(long long)(it.q0 + t) * a.Hq + it.head * a.G + row % a.G] = lse;
        }
        __syncwarp();
        constexpr int kChunks = D / 8, kRowsAtOnce = 32 / kChunks;
        const int chunk = lane % kChunks;
        for (int i = 0; i < 32; i += kRowsAtOnce) {
          const int r = (warp & 3) * 32 + i + lane / kChunks;
          const int tr = it.t0 + w * a.tokens + r / a.G;
          if (r < a.tokens * a.G && tr < it.lq) {
            const uint4 x = *reinterpret_cast<const uint4*>(stage + (chunk >> 3) * kHalf + r * 128 +
                                                            (((chunk & 7) ^ (r & 7)) << 4));
            *reinterpret_cast<uint4*>(a.out + (long long)(it.q0 + tr) * a.out_token +
                                      (long long)(it.head * a.G + r % a.G) * a.out_head + chunk * 8) = x;
          }
        }
      }
    }
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

__device__ int32_t g_prompt_status;      // one word per device: a bounded wait gave up

std::mutex g_mu;
int32_t* g_status_addr[kMaxDevices] = {};

int status_word(int32_t** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return CONFKV_ECUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_status_addr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_prompt_status) != cudaSuccess) return CONFKV_ECUDA;
    g_status_addr[dev] = static_cast<int32_t*>(p);
  }
  *out = g_status_addr[dev];
  return CONFKV_OK;
}

template <int D, bool BF16>
int launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, long long items,
           cudaStream_t st) {
  static int done[kMaxDevices] = {};
  auto kernel = prompt_attention_kernel<D, BF16>;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if (ensure_smem(kernel, Tile<D>::kSmem, done) != cudaSuccess) return CONFKV_ECUDA;
  }
  kernel<<<(unsigned)items, kThreads, Tile<D>::kSmem, st>>>(mq, mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? CONFKV_OK : CONFKV_ECUDA;
}

bool rows_ok(const void* p, const int64_t* stride, int d, long long tokens, long long heads) {
  if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  if (tokens > 1 && (stride[0] < d || stride[0] % 8 || stride[0] >= (1LL << 38))) return false;
  if (heads > 1 && (stride[1] < d || stride[1] % 8 || stride[1] >= (1LL << 38))) return false;
  return true;
}

}  // namespace
}  // namespace confkv

using namespace confkv;

extern "C" int confkv_prompt_attention(const confkv_prompt_args* p, void* stream) {
  if (!p) return CONFKV_EINVAL;
  if (p->B < 1 || p->Hq < 1 || p->Hkv < 1 || p->total_q < 0 || p->total_k < 0) return CONFKV_EINVAL;
  if (p->Hq % p->Hkv || p->Hq / p->Hkv > kRows) return CONFKV_EINVAL;
  if (p->dtype != CONFKV_Q_FP16 && p->dtype != CONFKV_Q_BF16) return CONFKV_EINVAL;
  if (p->d != 64 && p->d != 128) return CONFKV_ENOTIMPL;
  if (!std::isfinite(p->scale) || !(p->scale > 0.f)) return CONFKV_EINVAL;
  if (!p->cu_q || !p->cu_k || reinterpret_cast<uintptr_t>(p->cu_q) % 4 || reinterpret_cast<uintptr_t>(p->cu_k) % 4)
    return CONFKV_EINVAL;
  if (p->total_q == 0) return CONFKV_OK;
  if (!p->q || !p->out || (p->total_k > 0 && (!p->k || !p->v))) return CONFKV_EINVAL;
  if (!rows_ok(p->q, p->q_stride, p->d, p->total_q, p->Hq) ||
      !rows_ok(p->out, p->out_stride, p->d, p->total_q, p->Hq) ||
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
  // no more tiles than these, whatever the lengths
  const long long tiles = (long long)p->total_q / (2 * a.tokens) + p->B;
  if (tiles * p->Hkv >= (1LL << 31)) return CONFKV_EINVAL;
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
  const int r = status_word(&a.status);
  if (r != CONFKV_OK) return r;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p->d == 128)
    return bf16 ? launch<128, true>(mq, mk, mv, a, tiles * p->Hkv, st)
                : launch<128, false>(mq, mk, mv, a, tiles * p->Hkv, st);
  return bf16 ? launch<64, true>(mq, mk, mv, a, tiles * p->Hkv, st)
              : launch<64, false>(mq, mk, mv, a, tiles * p->Hkv, st);
}

extern "C" int confkv_prompt_status(int32_t* bits, void* stream) {
  if (!bits) return CONFKV_EINVAL;
  int32_t* word = nullptr;
  const int r = status_word(&word);
  if (r != CONFKV_OK) return r;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int32_t host = 0;
  cudaError_t e = cudaMemcpyAsync(&host, word, 4, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && host) e = cudaMemsetAsync(word, 0, 4, st);
  if (e != cudaSuccess) return CONFKV_ECUDA;
  *bits = host;
  return host ? CONFKV_EDEVICE : CONFKV_OK;
}

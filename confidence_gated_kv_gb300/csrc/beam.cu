// Selection of beams: the n best of beams x vocabulary continuations per group,
//   s_k + x_kv - log sum_w exp(x_kw).
//
// Within a beam the order is that of its logits, so the first kernel needs no
// sum: a CTA takes 4096 logits of one beam into registers, reduces them to
// (maximum, sum of exponentials) and writes its n largest in order.  The
// second kernel, a CTA per group, joins the sums, turns the candidates' logits
// into scores and ranks what can be among the n best.
//
// Both find their n largest by a bound: of 32 disjoint parts (many places: of
// as many as threads), the n-th largest part maximum.  At least n values reach it, and of random ones only
// a few more; these are ranked by counting.  Where more than kList reach it
// (plateaus of equal values) the places are filled one at a time.
//
// Scores are sums of four fp32 numbers or pairs of them, kept as pairs
// (48 bits): fp64 arithmetic runs at 1/64 of the fp32 rate here, and its
// comparisons alone would take the second kernel 10 us.
//
// What bounds it: one read of the logits, and the latency of the second
// kernel (five dependent reads and reductions).  In a graph, 8 x 4 beams of
// 152064 in fp32, 8 places: 12 us, 4 x 16 in bf16, 32 places: 24, four beams of
// 50257: 8.  Both parts in one launch, a cluster per group, took 9 for these.
// A bound of 64 parts for all numbers of places took 23 for the second and 330
// for 64 places where one of eight beams is far ahead, which take 30.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <climits>
#include <cmath>
#include <type_traits>

#include "../../include/confkv.h"
#include "confkv_internal.cuh"
#include "fp32_pair.cuh"
#include "tcgen05.cuh"

namespace confkv {
namespace {

using tc::ex2;

constexpr int kThreads = 256, kPer = 16, kChunk = kThreads * kPer;   // logits per CTA
constexpr int kJoin = 512;               // threads of the second kernel
constexpr int kMaxN = CONFKV_BEAM_MAX;
constexpr int kList = 512;               // values ranked by counting
constexpr int kMaxChunks = 1024;

struct Candidate {
  float logit;
  int token;
};

struct BeamArgs {
  int groups, beams, V, n, chunks;
  int end_token;
  const void* logits;
  long long group_stride, beam_stride;
  const float* scores;
  const uint8_t* finished;
  float2* sums;                                  // [row][chunk]: maximum, sum of exponentials
  Candidate* best;                               // [row][chunk][n], in order, then -inf
  float* scores_out;
  int32_t *parents, *tokens;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Low bits of the fp32 form that are zero in every value of the type (ordered: all
// zero or all one).
template <typename T>
constexpr int low_zeros() {
  return std::is_same_v<T, float> ? 0 : std::is_same_v<T, __half> ? 13 : 16;
}

// A float's bits in the order of its values (no NaN; -0 as 0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// (value, index) order: larger first, then the lower index.
template <typename V, typename I>
__device__ __forceinline__ bool before(V a, I i, V b, I j) { return a > b || (a == b && i < j); }

// The n-th largest of the parts' maxima, by one warp, from what WARPS warps
// left: `s_most[warp][lane]`.  Up to 16 places: parts are threads of equal index
// modulo 32 (a chunk that is cut short still fills them all), ranked by
// counting.  More: every thread is one; the bits of the bound are found from the
// top (a count each), down to the last 14, or to the LAST ones, which are alike in
// all values, but closer where more than twice as many parts reach it: at sums of
// -3000 the 14 bits are a step of 4 (32 beams of 50257, 64 places: 202 us without
// that, 21 with it).
template <int WARPS, int LAST>
__device__ __forceinline__ float bound_of(const float (*s_most)[32], int n) {
  const int lane = threadIdx.x & 31;
  if (n <= 16) {
    float v = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v = fmaxf(v, s_most[w][lane]);
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) rank += before(__shfl_sync(0xffffffffu, v, i), i, v, lane);
    return __shfl_sync(0xffffffffu, v, __ffs(__ballot_sync(0xffffffffu, rank == n - 1)) - 1);
  }
  uint32_t x[WARPS], most = 0, least = ~0u;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    x[w] = ordered(s_most[w][lane]);
    most = max(most, x[w]);
    least = min(least, x[w]);
  }
  // it lies between the largest and the least of the lanes' largest (of all),
  // whose leading bits it shares
  least = __reduce_min_sync(0xffffffffu, n <= 32 ? most : least);
  most = __reduce_max_sync(0xffffffffu, most);
  const int same = __clz(least ^ most);                  // 32: all alike
  uint32_t bound = same == 0 ? 0u : most & ~0u << (32 - same);
  auto reaching = [&](uint32_t y) {
    int reach = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) reach += x[w] >= y;
    return __reduce_add_sync(0xffffffffu, reach);
  };
  int at = 31 - same;
  for (; at >= (LAST > 14 ? LAST : 14); --at)
    if (reaching(bound | 1u << at) >= n) bound |= 1u << at;
  if (LAST < 14 && at >= LAST && reaching(bound) > 2 * n)
    for (; at >= LAST; --at)
      if (reaching(bound | 1u << at) >= n) bound |= 1u << at;
  return unordered(max(bound, ordered(-INFINITY)));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_chunk_kernel(const __grid_constant__ BeamArgs a) {
  constexpr int kVec = 16 / sizeof(T), kVecs = kPer / kVec;
  __shared__ float s_most[kThreads / 32][32];
  __shared__ float2 s_sum[kThreads / 32];                // of a warp: maximum, sum of exponentials
  __shared__ float s_bound;
  __shared__ int s_count;
  __shared__ float s_value[kList];
  __shared__ int s_index[kList];
  const int thread = threadIdx.x, warp = thread >> 5, lane = thread & 31;
  const unsigned row = blockIdx.x;
  const int chunk = blockIdx.y;
  pdl_wait();
  if (a.finished && a.finished[row]) return;
  const T* x = static_cast<const T*>(a.logits) + row / (unsigned)a.beams * a.group_stride +
               row % (unsigned)a.beams * a.beam_stride;
  // vectors start at the row's first 16-byte boundary; the first chunk also
  // takes what lies before it
  const int head = min(a.V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T));
  float v[kPer + 2];
  const int base = head + chunk * kChunk + thread * kVec;
  auto index = [&](int i) {
    return i < kPer ? base + i / kVec * kThreads * kVec + i % kVec : thread;
  };
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int e = index(j * kVec);
    if (e + kVec <= a.V) {
      const uint4 w = *reinterpret_cast<const uint4*>(x + e);
      const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[j * kVec + i] = to_float(t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[j * kVec + i] = e + i < a.V ? to_float(x[e + i]) : -INFINITY;
    }
  }
  v[kPer] = chunk == 0 && thread < head ? to_float(x[thread]) : -INFINITY;
  v[kPer + 1] = -INFINITY;
  if (thread == 0) s_count = 0;

  float mine = -INFINITY;                                // a NaN is no maximum
#pragma unroll
  for (int i = 0; i <= kPer; ++i) mine = fmaxf(mine, v[i]);
  s_most[warp][lane] = mine;
  // the warp's sum, in fp32 in a fixed order; x - M is exact to half a step of
  // the result.  Without a value above -inf it is zero, or NaN.
  const float M = unordered(__reduce_max_sync(0xffffffffu, ordered(mine))), off = M == -INFINITY ? 0.f : -M;
  Pair sums[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)};
#pragma unroll
  for (int i = 0; i <= kPer; i += 2) {
    const float2 e = ((Pair(v[i], v[i + 1]) + Pair(off, off)) * Pair(1.4426950408889634f, 1.4426950408889634f)).get();
    sums[i / 2 & 1] = sums[i / 2 & 1] + Pair(ex2(e.x), ex2(e.y));
  }
  const float2 both = (sums[0] + sums[1]).get();
  float sum = both.x + both.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = make_float2(M, sum);
  __syncthreads();
  const long long list = (long long)row * a.chunks + chunk;
  if (warp == 0) {
    const float t = bound_of<kThreads / 32, low_zeros<T>()>(s_most, a.n);
    if (lane == 0) s_bound = t;
  } else if (thread == 32) {
    float top = -INFINITY, all = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, s_sum[w].x);
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) all += s_sum[w].y * (s_sum[w].x == top ? 1.f : ex2((s_sum[w].x - top) * 1.4426950408889634f));
    a.sums[list] = make_float2(top, all);
  }
  __syncthreads();
  const float bound = s_bound;
  if (mine >= bound && mine > -INFINITY) {
#pragma unroll
    for (int i = 0; i <= kPer; ++i)
      if (v[i] >= bound && v[i] > -INFINITY) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kList) {
          s_value[at] = v[i];
          s_index[at] = index(i);
        }
      }
  }
  __syncthreads();
  const int count = s_count;
  Candidate* best = a.best + list * a.n;
  if (count <= kList) {
    for (int i = thread; i < count; i += kThreads) {
      const float y = s_value[i];
      const int at = s_index[i];
      int rank = 0;
      for (int j = 0; j < count; ++j) rank += before(s_value[j], s_index[j], y, at);
      if (rank < a.n) best[rank] = Candidate{y, at};
    }
    for (int i = count + thread; i < a.n; i += kThreads) best[i] = Candidate{-INFINITY, 0};
    return;
  }
  // one place at a time: the best that comes after the last one
  float last = INFINITY;
  int last_at = -1;
  for (int k = 0; k < a.n; ++k) {
    float y = -INFINITY;
    int at = INT_MAX;
#pragma unroll
    for (int i = 0; i <= kPer; ++i)
      if (before(last, last_at, v[i], index(i)) && v[i] > -INFINITY && before(v[i], index(i), y, at)) {
        y = v[i];
        at = index(i);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float z = __shfl_xor_sync(0xffffffffu, y, o);
      const int j = __shfl_xor_sync(0xffffffffu, at, o);
      if (before(z, j, y, at)) {
        y = z;
        at = j;
      }
    }
    __syncthreads();                                     // the last round's values are read
    if (lane == 0) {
      s_value[warp] = y;
      s_index[warp] = at;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
      if (before(s_value[w], s_index[w], y, at)) {
        y = s_value[w];
        at = s_index[w];
      }
    if (thread == 0) best[k] = y > -INFINITY ? Candidate{y, at} : Candidate{-INFINITY, 0};
    last = y;
    last_at = at;
  }
}

// a + b as a rounded sum and its error.
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}

// score + (logit - most) - log sum: a normalised pair as one number to compare.
// The beam's largest logit comes off first: as one number with the logarithm it
// could be so large (all logits the type's lowest value) that nothing of that
// is left.
constexpr unsigned long long kNone = 0x007fffff00000000ull;      // of -inf
__device__ __forceinline__ unsigned long long key_of(float score, float logit, float most, float2 log_sum) {
  const float2 a = two_sum(logit, -most), b = two_sum(a.x, score), c = two_sum(b.x, -log_sum.x);
  const float2 r = two_sum(c.x, __fadd_rn(c.y, __fadd_rn(b.y, __fsub_rn(a.y, log_sum.y))));
  if (!(fabsf(r.x) < INFINITY)) return kNone;            // the sum leaves fp32
  return (unsigned long long)ordered(r.x) << 32 | ordered(r.y);
}

__global__ void __launch_bounds__(kJoin, 1) beam_join_kernel(const __grid_constant__ BeamArgs a) {
  __shared__ float2 s_log[kMaxN];                        // of the sum of exponentials
  __shared__ float s_score[kMaxN], s_max[kMaxN], s_total[kMaxN];
  __shared__ float s_most[kJoin / 32][32];
  __shared__ unsigned long long s_key[kList];
  __shared__ long long s_index[kList];
  __shared__ uint8_t s_kind[kMaxN];                      // of a beam: 0 offers nothing, 1 tokens, 2 finished
  __shared__ float s_bound;
  __shared__ int s_count;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = blockIdx.x;
  const long long row0 = (long long)group * a.beams;
  pdl_wait();
  if (threadIdx.x == 0) s_count = 0;
  const int lists = a.beams * a.chunks;
  const Candidate* best = a.best + row0 * a.chunks * a.n;
  // The bound is taken of the first `deep` entries of each list: the heads, or
  // for many places twice as many entries of each beam as there are places (few
  // lists, or a beam that is far ahead of the others, would give a low one by
  // their heads alone).  A thread's first ones are on their way while the sums
  // are joined.
  const int deep = a.n > 16 ? min(a.n, (2 * a.n + a.chunks - 1) / a.chunks) : 1, heads = lists * deep;
  const int entry0 = (int)threadIdx.x / lists, list0 = (int)threadIdx.x - entry0 * lists;
  const Candidate first = threadIdx.x < heads ? best[(long long)list0 * a.n + entry0] : Candidate{-INFINITY, 0};
  const Candidate second = threadIdx.x + kJoin < lists ? best[(long long)(threadIdx.x + kJoin) * a.n] : Candidate{-INFINITY, 0};
  for (int k = warp; k < a.beams; k += kJoin / 32) {
    const bool ended = a.finished && a.finished[row0 + k];
    float M = 0.f, sum = 1.f;
    if (!ended) {
      const float2* sums = a.sums + (row0 + k) * a.chunks;
      const float2 none = make_float2(-INFINITY, 0.f);
      const float2 z0 = lane < a.chunks ? sums[lane] : none, z1 = lane + 32 < a.chunks ? sums[lane + 32] : none;
      M = fmaxf(z0.x, z1.x);
      for (int c = lane + 64; c < a.chunks; c += 32) M = fmaxf(M, sums[c].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      // a chunk without a value above -inf adds its sum: zero, or NaN
      auto scaled = [&](float2 z) {
        return z.x == M || z.x == -INFINITY ? z.y : z.y * ex2((z.x - M) * 1.4426950408889634f);
      };
      sum = scaled(z0) + scaled(z1);
      for (int c = lane + 64; c < a.chunks; c += 32) sum += scaled(sums[c]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane == 0) {
      s_max[k] = M;
      s_total[k] = sum;
      s_kind[k] = ended ? 2 : 1;
    }
  }
  __syncthreads();
  // The logarithms in fp64, all by one or two warps at once: half a step of
  // fp32 at 12 would be 5e-7.
  if (threadIdx.x < a.beams) {
    const int k = threadIdx.x;
    const float score = a.scores[row0 + k];
    const double log_sum = log((double)s_total[k]);
    const float hi = (float)log_sum;
    if (!isfinite(score) || !isfinite(s_max[k]) || !isfinite(hi)) s_kind[k] = 0;
    s_score[k] = score;
    s_log[k] = make_float2(hi, (float)(log_sum - (double)hi));
  }
  __syncthreads();
  // entry e of list i (a chunk of a beam), whose candidate is c
  auto key = [&](int i, int e, const Candidate& c, long long* at) {
    const int k = i / a.chunks, kind = s_kind[k];
    *at = LLONG_MAX;
    if (kind == 0) return kNone;
    if (kind == 2) {
      if (i % a.chunks || e) return kNone;
      *at = (long long)k * a.V + a.end_token;
      return (unsigned long long)ordered(s_score[k]) << 32 | ordered(0.f);
    }
    if (!(c.logit > -INFINITY)) return kNone;
    *at = (long long)k * a.V + c.token;
    return key_of(s_score[k], c.logit, s_max[k], s_log[k]);
  };
  auto load = [&](int i, int e) {
    return e == 0 && i < kJoin ? first : e == 0 && i < 2 * kJoin ? second : best[(long long)i * a.n + e];
  };
  float most = -INFINITY;
  for (int f = threadIdx.x; f < heads; f += kJoin) {
    const bool own = f < kJoin;
    const int e = own ? entry0 : f / lists, i = own ? list0 : f - e * lists;
    long long at;
    most = fmaxf(most, unordered((uint32_t)(key(i, e, own ? first : load(i, e), &at) >> 32)));
  }
  s_most[warp][lane] = most;
  __syncthreads();
  if (warp == 0) {
    const float t = bound_of<kJoin / 32, 0>(s_most, a.n);
    if (lane == 0) s_bound = t;
  }
  __syncthreads();
  const uint32_t bound = ordered(s_bound);                   // in rounded sums
  if (deep > 1 || (ordered(most) >= bound && most > -INFINITY))
    for (int i = threadIdx.x; i < lists; i += kJoin) {
      bool more = true;
      for (int e0 = 0; e0 < a.n && more; e0 += 4) {      // four entries of the list on their way
        Candidate c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = e0 + e < a.n ? load(i, e0 + e) : Candidate{-INFINITY, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          long long at;
          const unsigned long long y = more && e0 + e < a.n ? key(i, e0 + e, c[e], &at) : kNone;
          more = (uint32_t)(y >> 32) >= bound && y > kNone;
          if (more) {
            const int to = atomicAdd(&s_count, 1);
            if (to < kList) {
              s_key[to] = y;
              s_index[to] = at;
            }
          }
        }
      }
    }
  __syncthreads();
  const int count = s_count;
  float* scores = a.scores_out + (long long)group * a.n;
  int32_t *parents = a.parents + (long long)group * a.n, *tokens = a.tokens + (long long)group * a.n;
  auto put = [&](int place, unsigned long long y, long long at) {
    const bool some = y > kNone;
    scores[place] = some ? unordered((uint32_t)(y >> 32)) : -INFINITY;
    parents[place] = some ? (int32_t)(at / a.V) : 0;
    tokens[place] = some ? (int32_t)(at % a.V) : 0;
  };
  if (count <= kList) {
    for (int i = threadIdx.x; i < count; i += kJoin) {
      const unsigned long long y = s_key[i];
      const long long at = s_index[i];
      int rank = 0;
      for (int j = 0; j < count; ++j) rank += before(s_key[j], s_index[j], y, at);
      if (rank < a.n) put(rank, y, at);
    }
    for (int i = count + threadIdx.x; i < a.n; i += kJoin) put(i, kNone, 0);
    return;
  }
  unsigned long long last = ~0ull;
  long long last_at = -1;
  for (int k = 0; k < a.n; ++k) {
    unsigned long long y = kNone;
    long long at = LLONG_MAX;
    for (int i = threadIdx.x; i < lists; i += kJoin)
      for (int e = 0; e < a.n; ++e) {
        long long j;
        const unsigned long long z = key(i, e, load(i, e), &j);
        if (z <= kNone || before(y, at, z, j)) break;    // the rest of the list is no better
        if (before(last, last_at, z, j) && before(z, j, y, at)) {
          y = z;
          at = j;
        }
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long z = __shfl_xor_sync(0xffffffffu, y, o);
      const long long j = __shfl_xor_sync(0xffffffffu, at, o);
      if (before(z, j, y, at)) {
        y = z;
        at = j;
      }
    }
    __syncthreads();
    if (lane == 0) {
      s_key[warp] = y;
      s_index[warp] = at;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoin / 32; ++w)
      if (before(s_key[w], s_index[w], y, at)) {
        y = s_key[w];
        at = s_index[w];
      }
    if (threadIdx.x == 0) put(k, y, at);
    last = y;
    last_at = at;
  }
}

template <typename T>
int launch(const BeamArgs& a, cudaStream_t st) {
  if (launch_pdl(beam_chunk_kernel<T>, dim3((unsigned)(a.groups * a.beams), (unsigned)a.chunks), dim3(kThreads), 0, st, a) !=
          cudaSuccess ||
      launch_pdl(beam_join_kernel, dim3((unsigned)a.groups), dim3(kJoin), 0, st, a) != cudaSuccess)
    return CONFKV_ECUDA;
  return CONFKV_OK;
}

int chunks_of(int V) { return (V + kChunk - 1) / kChunk; }

bool sizes_ok(int groups, int beams, int V, int n) {
  if (groups < 0 || beams < 1 || beams > kMaxN || V < 1 || V > kChunk * kMaxChunks || n < 1 || n > kMaxN) return false;
  if (n > (long long)beams * V) return false;
  return (long long)groups * beams < (1LL << 31) / kMaxChunks;
}

size_t sums_bytes(long long lists) { return ((size_t)lists * sizeof(float2) + 15) / 16 * 16; }

}  // namespace
}  // namespace confkv

using namespace confkv;

extern "C" int confkv_beam_workspace_bytes(int32_t groups, int32_t beams, int32_t V, int32_t n, size_t* bytes) {
  if (!bytes || !sizes_ok(groups, beams, V, n)) return CONFKV_EINVAL;
  const long long lists = (long long)groups * beams * chunks_of(V);
  *bytes = sums_bytes(lists) + (size_t)lists * n * sizeof(Candidate);
  return CONFKV_OK;
}

extern "C" int confkv_beam_select(const confkv_beam_args* p, void* stream) {
  if (!p) return CONFKV_EINVAL;
  size_t need = 0;
  if (confkv_beam_workspace_bytes(p->groups, p->beams, p->V, p->n, &need) != CONFKV_OK) return CONFKV_EINVAL;
  if (p->dtype != CONFKV_FP16 && p->dtype != CONFKV_BF16 && p->dtype != CONFKV_FP32) return CONFKV_EINVAL;
  if (p->end_token < 0 || p->end_token >= p->V) return CONFKV_EINVAL;
  if (p->groups == 0) return CONFKV_OK;
  const uintptr_t size = p->dtype == CONFKV_FP32 ? 4 : 2;
  auto misaligned = [](const void* x, uintptr_t to) { return !x || reinterpret_cast<uintptr_t>(x) % to; };
  if (misaligned(p->logits, size) || misaligned(p->scores, 4) || misaligned(p->scores_out, 4) ||
      misaligned(p->parents, 4) || misaligned(p->tokens, 4) || misaligned(p->workspace, 16))
    return CONFKV_EINVAL;
  for (int i = 0; i < 2; ++i)
    if (p->logits_stride[i] < 0 || p->logits_stride[i] >= (1LL << 38)) return CONFKV_EINVAL;
  if (p->workspace_bytes < need) return CONFKV_ECAPACITY;
  BeamArgs a{};
  a.groups = p->groups; a.beams = p->beams; a.V = p->V; a.n = p->n;
  a.chunks = chunks_of(p->V);
  a.end_token = p->end_token;
  a.logits = p->logits;
  a.group_stride = p->logits_stride[0];
  a.beam_stride = p->logits_stride[1];
  a.scores = p->scores;
  a.finished = p->finished;
  const long long lists = (long long)p->groups * p->beams * a.chunks;
  a.sums = static_cast<float2*>(p->workspace);
  a.best = reinterpret_cast<Candidate*>(static_cast<char*>(p->workspace) + sums_bytes(lists));
  a.scores_out = p->scores_out;
  a.parents = p->parents;
  a.tokens = p->tokens;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return p->dtype == CONFKV_FP32   ? launch<float>(a, st)
         : p->dtype == CONFKV_BF16 ? launch<__nv_bfloat16>(a, st)
                                   : launch<__half>(a, st);
}

// What the two kernels of the drafted-token attention share: the call, who
// sees whom among the drafts, and the type conversions.
//
//   out_r = sum_j softmax_j(scale q_r . k_j) v_j
//
// over the resident entries of (layer, sequence) and, of the drafted tokens,
// those on the row's own path to the root.  For an INT8 entry k = sK c with
// one scale per channel: the scale goes into the query, the codes are exact in
// fp16.  v = sV c likewise: the weighted codes are added up and scaled once.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cfloat>

#include "confkv_internal.cuh"
#include "tcgen05.cuh"

namespace confkv {
namespace tree {

using namespace tc;

constexpr int kMaxDrafts = 128;          // per sequence
constexpr int kMaxSplit = 8;             // CTAs of a cluster that share the keys of some rows

// Weights are exp2(score - reference + kLift), in fp16.  The kernel of few rows
// holds them in two parts, off by 2^-22, which costs it 2 to 5 %.  The kernel of
// many rows rounds them to one part, off by 2^-11 of each: half a step of an fp16
// output, an eighth of that of a bf16 one, and less in a sum of many, whose
// errors differ in sign.  A second part there was built and measured, fp16 inputs:
// 0 to 61 drafts on 37 to 4097 entries, whose relative error against 64 bits is
// 2.6e-4 with one part and 2.1e-4 where only the output is rounded, took 45 us
// instead of 39, 64 drafts on four sequences of 8192 124 instead of 103, 16 on
// eight of 2049 38 instead of 32, most of it to split and to store the weights.
// With bf16 outputs the error is the output's rounding, 1.7e-3, either way.
//
// The reference moves when a score passes it by more than kLag bits, so a
// weight stays below 2^15.  Fp16 ends at 2^-24: a weight is off by at most
// 2^-25 - kLift of the reference's, 2^-29.  The reference moves the less often
// the further it may lag, and a move rescales the accumulator: with a lift of 11
// and a lag of 4, and one key in 200 three times as long, every other tile of 64
// keys did.
constexpr float kLift = 4.f, kLag = 11.f, kUnlift = 1.f / 16.f;

struct Call {
  int layer, T;                          // drafts per sequence
  int split;                             // CTAs of a cluster that share the keys
  int tiles;                             // row tiles per (sequence, KV head)
  float scale2;                          // scale * log2(e)
  const uint16_t *q, *k, *v;             // fp16 or bf16
  uint16_t* out;
  float* lse;
  const int32_t *parents, *lens;         // may be null: a chain, all in use
  long long q_b, q_t, q_h, k_b, k_t, k_h, v_b, v_t, v_h, o_b, o_t, o_h, p_b, p_t;
  long long limit;                       // cycles after which a wait gives up
  int absent;                            // CTA whose softmax warps do nothing (self-test), or -1
  char* dealt;                           // workspace of dealt keys (tree_tiles.cu), or null
  int ctas;                              // among which they are dealt
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst), "l"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint4 lds(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t& word(uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Two 16-bit inputs as fp16 (a bf16 value beyond it becomes infinite).
template <bool BF16>
__device__ __forceinline__ uint32_t half_pair(uint32_t w) {
  return BF16 ? pack2<false>(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)) : w;
}
template <bool BF16>
__device__ __forceinline__ float2 float_pair(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ float half_value(uint16_t w) {     // one input, rounded to fp16
  const uint32_t h = half_pair<BF16>(w);
  return __half2float(__ushort_as_half((unsigned short)h));
}
template <bool BF16>
__device__ __forceinline__ float input_value(uint16_t w) {
  return BF16 ? __uint_as_float((uint32_t)w << 16) : __half2float(__ushort_as_half(w));
}

// Four stored bytes (code + 128) as two fp16 pairs of codes: 0x6400 | byte is
// 1024 + byte, and 1152 is taken off exactly.
__device__ __forceinline__ void codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(w, 0x64646464u, 0x5140), b = __byte_perm(w, 0x64646464u, 0x5342);
  const __half2 off = __half2half2(__ushort_as_half((unsigned short)0x6480));   // 1152
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// Power of two that brings the largest |x| of a query row to [2^13, 2^14): an
// fp16 row then loses nothing of any input's range that its largest value
// leaves visible.  Zero, infinite and NaN rows keep a finite factor.
__device__ __forceinline__ float row_factor(float largest) {
  const int e = min(max((int)(__float_as_uint(largest) >> 23), 14), 254);
  return __uint_as_float((uint32_t)(267 - e) << 23);
}
__device__ __forceinline__ float row_unfactor(float largest) {       // its reciprocal
  const int e = min(max((int)(__float_as_uint(largest) >> 23), 14), 254);
  return __uint_as_float((uint32_t)(e - 13) << 23);
}
// Log2 units of a row's accumulated products.  Never zero or infinite: hidden
// keys are -inf in the accumulator, and -inf * 0 or 0 * inf would make the row
// NaN.  Products stay below 2^40, so a unit below the smallest normal number
// leaves scores of next to zero either way, and one beyond fp32 has a row of
// zeros or scores beyond fp32.
__device__ __forceinline__ float row_unit(const Call& a, float largest) {
  return fminf(fmaxf(a.scale2 * row_unfactor(largest), FLT_MIN), FLT_MAX);
}
// x0, x1 rounded to fp16, and what the rounding left.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack2<false>(x0, x1);
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  lo = pack2<false>(x0 - h.x, x1 - h.y);
}

__device__ __forceinline__ int drafts_of(const Call& a, int b) {
  return a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
}

// Bit j of path[t]: draft j is t or one of its ancestors, for the first
// `drafts` tokens of sequence b, by THREADS threads that the barrier `sync`
// joins.  A parent that is not an earlier draft stands for the cache.  Each
// round doubles the steps that a path covers.
template <int THREADS, typename Sync>
__device__ __forceinline__ void draft_paths(const Call& a, int b, int drafts, int thread, uint4* path, int* up,
                                            Sync sync) {
  constexpr int kEach = (kMaxDrafts + THREADS - 1) / THREADS;
  for (int t = thread; t < kMaxDrafts; t += THREADS) {
    uint32_t m[4];
    int p = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {                        // all before t in a chain, t itself in a tree
      const int n = t + 1 - 32 * i;
      m[i] = t >= drafts ? 0u : n <= 0 ? 0u : a.parents ? (n <= 32 ? 1u << (n - 1) : 0u) : n >= 32 ? ~0u : (1u << n) - 1u;
    }
    if (a.parents && t < drafts) {
      p = a.parents[b * a.p_b + t * a.p_t];
      if (p < 0 || p >= t) p = -1;
    }
    path[t] = make_uint4(m[0], m[1], m[2], m[3]);
    up[t] = p;
  }
  sync();
  if (!a.parents) return;
  for (int steps = 1; steps < drafts; steps <<= 1) {
    uint4 x[kEach];
    int p[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int t = thread + e * THREADS;
      if (t < kMaxDrafts) {
        x[e] = path[t];
        p[e] = up[t];
        if (p[e] >= 0) {
          const uint4 y = path[p[e]];
          x[e] = make_uint4(x[e].x | y.x, x[e].y | y.y, x[e].z | y.z, x[e].w | y.w);
          p[e] = up[p[e]];
        }
      }
    }
    sync();
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (thread + e * THREADS < kMaxDrafts) {
        path[thread + e * THREADS] = x[e];
        up[thread + e * THREADS] = p[e];
      }
    sync();
  }
}

// Values of v that are infinite or NaN would reach rows that do not see them
// (a weight of zero times infinity), so the products take a zero in their
// place and the tokens that have one are marked; the rows that do see such a
// token get its values added at the end.
template <bool BF16>
__device__ __forceinline__ float unfinite(const Call& a, int b, int h, const uint4& path, const uint32_t* bad, int c) {
  float sum = 0.f;
  const uint32_t m[4] = {path.x & bad[0], path.y & bad[1], path.z & bad[2], path.w & bad[3]};
  for (int i = 0; i < 4; ++i)
    for (uint32_t w = m[i]; w; w &= w - 1) {
      const int t = 32 * i + __ffs((int)w) - 1;
      const float x = half_value<BF16>(a.v[b * a.v_b + t * a.v_t + h * a.v_h + c]);
      if (!isfinite(x)) sum += x;
    }
  return sum;
}

}  // namespace tree

// Two kernels (and a join of the second's).  Rows of 16 per CTA, products by mma.sync straight from the
// stored layout; 128 rows per CTA, products by tcgen05 from converted tiles.
// The plans give the split over a cluster (Call::split) and the time to
// expect, for n8_bound INT8 entries in every (layer, sequence); only the
// launch shape follows them.
double plan_tree_rows(const Shape& s, int T, long long n8_bound, int* split);
int launch_tree_rows(const Shape& s, const Dev& d, const tree::Call& a, bool bf16, cudaStream_t st);
double plan_tree_tiles(const Shape& s, int T, long long n8_bound, int* split);
// The same with the keys dealt out by each sequence's own length, where that is
// possible: bytes of its workspace (0: not), time to expect for the INT8
// entries n8[b] and the number of CTAs.
size_t dealt_tree_bytes(const Shape& s, int T);
constexpr int kDealtMost = 304;          // sequences at most
double plan_dealt_tree(const Shape& s, int T, const long long* n8, int* ctas);
int launch_tree_tiles(const Shape& s, const Dev& d, const tree::Call& a, bool bf16, cudaStream_t st);

}  // namespace confkv

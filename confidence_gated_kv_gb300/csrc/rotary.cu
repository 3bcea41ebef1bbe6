// RMS norms of queries and keys per head and the rotary rotation, in one
// pass.  A row is one head of one token:
//
//   y = x * rsqrt(mean(x^2) + eps) * weight          (or y = x without weight)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t) * mscale
//
// for the rot / 2 pairs of the first rot channels, t = position * frequency;
// a pair is channels (2i, 2i + 1) or (i, i + rot / 2).
//
// Angles.  The frequencies come as turns per position in 64-bit fixed point
// (unit 2^-64), so that position * frequency modulo one turn is one 64-bit
// integer product, exact for every 32-bit position.  Its top 32 bits are then
// rounded to fp32, to within 2^-25 half turns (1e-7 rad); an fp32 angle at
// position 10^6 is off by up to 0.03 rad.  sincospi needs no range reduction.
//
// The pass reads and writes every element once and is bound by HBM; a thread
// keeps the sines and cosines of its 16 channels over several heads of a
// token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cmath>

#include "../../include/confkv.h"
#include "confkv_internal.cuh"
#include "fp32_pair.cuh"

namespace confkv {
namespace {

struct RotArgs {
  int n, Hq, Hkv, d, rot, interleaved;
  int in_type, w_type, q_type, k_type;
  float eps, mscale;
  const void *q, *k;
  void *qo, *ko;
  long long q_t, q_h, k_t, k_h, qo_t, qo_h, ko_t, ko_h;
  const void *qw, *kw;
  const int32_t* pos;
  const uint64_t* turns;
  int tokens, heads;         // per block (rows kernel)
};

__device__ __forceinline__ float load1(const void* p, long long i, int type) {
  if (type == CONFKV_FP32) return static_cast<const float*>(p)[i];
  if (type == CONFKV_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store1(void* p, long long i, int type, float x) {
  if (type == CONFKV_FP32)
    static_cast<float*>(p)[i] = x;
  else if (type == CONFKV_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(x);
}

// 8 consecutive elements as they lie in memory, from element offset i (a
// multiple of 8), and as fp32.
template <int TYPE>
struct Raw {
  uint4 w[TYPE == CONFKV_FP32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, long long i) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (TYPE == CONFKV_FP32 ? 4 : 2));
    w[0] = src[0];
    if (TYPE == CONFKV_FP32) w[TYPE == CONFKV_FP32] = src[1];
  }
  __device__ __forceinline__ void floats(float* x) const {
    const uint32_t* u = &w[0].x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (TYPE == CONFKV_FP32) {
        x[j] = __uint_as_float(u[j]);
        x[4 + j] = __uint_as_float((&w[TYPE == CONFKV_FP32].x)[j]);
      } else if (TYPE == CONFKV_BF16) {
        x[2 * j] = __uint_as_float(u[j] << 16);
        x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
      }
    }
  }
};
__device__ __forceinline__ void store8(void* p, long long i, int type, const float* x) {
  if (type == CONFKV_FP32) {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    f[0] = make_float4(x[0], x[1], x[2], x[3]);
    f[1] = make_float4(x[4], x[5], x[6], x[7]);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (type == CONFKV_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void angle(const RotArgs& a, int pos, int i, float* c, float* s) {
  const uint64_t turn = (uint64_t)(int64_t)pos * a.turns[i];      // modulo one turn
  sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, s, c);   // 2^-31: half turns
  *c *= a.mscale;
  *s *= a.mscale;
}

// A block takes `tokens` tokens and `heads` of their heads: it computes the
// sines and cosines of its tokens once into shared memory, then groups of TPR
// threads take a row each, two 8-channel chunks per thread, with the next
// row in flight.  (One thread computing its own angles for four heads, without
// shared memory, was bound by instructions: 49 us for 8192 tokens of 48
// heads of 128 channels against 36 now.)
constexpr int kMaxTokens = 16;
template <int TPR, int IN>
__global__ void __launch_bounds__(256, 4) rotary_rows_kernel(const __grid_constant__ RotArgs a) {
  constexpr int kGroups = 256 / TPR, kDim = 16 * TPR;
  pdl_wait();
  // In the order in which the threads of a row read them, four floats each:
  // weights of q and k, then [token][cosines, sines][rot / 2].
  extern __shared__ __align__(16) float s_float[];
  float* s_turn = s_float + 2 * kDim;
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int heads = a.Hq + a.Hkv;
  const int token0 = blockIdx.x * a.tokens, tokens = min(a.tokens, a.n - token0);
  const int head0 = blockIdx.y * a.heads, count = min(a.heads, heads - head0);
  const int rows = tokens * count, pairs = a.rot / 2;
  // chunks of this thread and whether they are rotated (both or neither:
  // rot is a multiple of 16)
  const int half = a.rot / 16;                 // chunks of one half of the rotated part
  const bool turned = t < half;
  int c0 = 2 * t, c1 = 2 * t + 1;
  if (!a.interleaved && turned) {
    c0 = t;
    c1 = t + half;
  }
  // rows group, group + kGroups, ... as (token, head of the block's)
  struct Row {
    int token, head;
  };
  const int dt = kGroups / count, dh = kGroups % count;
  auto next = [&](Row& r) {
    r.token += dt;
    r.head += dh;
    if (r.head >= count) {
      r.head -= count;
      ++r.token;
    }
  };
  auto fetch = [&](const Row& r, Raw<IN>& r0, Raw<IN>& r1) {
    const long long token = token0 + r.token;
    const int head = head0 + r.head;
    const char* src = static_cast<const char*>(head < a.Hq ? a.q : a.k);
    const long long off = head < a.Hq ? token * a.q_t + head * a.q_h : token * a.k_t + (head - a.Hq) * a.k_h;
    r0.load(src, off + 8 * c0);
    r1.load(src, off + 8 * c1);
  };
  Raw<IN> r0 = {}, r1 = {};
  Row row{group / count, group % count};
  if (row.token < tokens) fetch(row, r0, r1);
  for (int i = threadIdx.x; i < 2 * kDim; i += 256) {
    const void* weight = i < kDim ? a.qw : a.kw;
    const int c = i % kDim;
    if (weight) s_float[i - c + (c >> 2 & 1) * (kDim / 2) + (c >> 3) * 4 + (c & 3)] = load1(weight, c, a.w_type);
  }
  for (int i = threadIdx.x; i < tokens * pairs; i += 256) {
    const int token = i / pairs, p = i % pairs;
    float* turn = s_turn + token * a.rot + (p >> 2 & 1) * (pairs / 2) + (p >> 3) * 4 + (p & 3);
    angle(a, a.pos[token0 + token], p, turn, turn + pairs);
  }
  __syncthreads();
  for (int base = 0; base < rows; base += kGroups) {       // the same count for every thread
    const Row now = row;
    const bool on = now.token < tokens;
    const int token = on ? now.token : 0, head = head0 + now.head;
    const bool is_q = head < a.Hq;
    Pair x[8];                                             // chunk c0, then c1
    {
      float f[16];
      r0.floats(f);
      r1.floats(f + 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = Pair(f[2 * i], f[2 * i + 1]);
    }
    next(row);
    if (row.token < tokens) fetch(row, r0, r1);
    if (a.qw || a.kw) {
      Pair sq = x[0] * x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) sq = fma2(x[i], x[i], sq);
      float ss = sq.get().x + sq.get().y;
#pragma unroll
      for (int o = 1; o < TPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (is_q ? a.qw != nullptr : a.kw != nullptr) {
        const float f = rsqrtf(ss * (1.f / kDim) + a.eps);
        const float4* w = reinterpret_cast<const float4*>(s_float + (is_q ? 0 : kDim));
        const float4 g[4] = {w[c0], w[kDim / 8 + c0], w[c1], w[kDim / 8 + c1]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = x[2 * i] * Pair(f, f) * Pair(g[i].x, g[i].y);
          x[2 * i + 1] = x[2 * i + 1] * Pair(f, f) * Pair(g[i].z, g[i].w);
        }
      }
    }
    if (!on) continue;
    if (turned) {
      const float4* turn = reinterpret_cast<const float4*>(s_turn + token * a.rot) + t;
      const float4 ca = turn[0], cb = turn[half], sa = turn[2 * half], sb = turn[3 * half];
      const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
      const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = x[i].get();
          x[i] = fma2(x[i], Pair(c[i], c[i]), Pair(f.y, f.x) * Pair(-s[i], s[i]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Pair u = x[i], v = x[4 + i], cc(c[2 * i], c[2 * i + 1]);
          x[i] = fma2(u, cc, v * Pair(-s[2 * i], -s[2 * i + 1]));
          x[4 + i] = fma2(v, cc, u * Pair(s[2 * i], s[2 * i + 1]));
        }
      }
    }
    void* dst = is_q ? a.qo : a.ko;
    const int type = is_q ? a.q_type : a.k_type;
    const long long at = token0 + token;
    const long long off = is_q ? at * a.qo_t + head * a.qo_h : at * a.ko_t + (head - a.Hq) * a.ko_h;
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = x[i].get().x;
      y[2 * i + 1] = x[i].get().y;
    }
    store8(dst, off + 8 * c0, type, y);
    store8(dst, off + 8 * c1, type, y + 8);
  }
}

// Any head size, alignment and rotated part: one warp per row, the row in
// shared memory.
constexpr int kMaxDim = 512;
constexpr int kAnyWarps = 4;
__global__ void __launch_bounds__(32 * kAnyWarps) rotary_any_kernel(const __grid_constant__ RotArgs a) {
  __shared__ float s_row[kAnyWarps][kMaxDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, heads = a.Hq + a.Hkv;
  const long long row = (long long)blockIdx.x * kAnyWarps + warp;
  if (row >= (long long)a.n * heads) return;
  const int token = (int)(row / heads), head = (int)(row % heads);
  const bool is_q = head < a.Hq;
  const void* src = is_q ? a.q : a.k;
  const long long off = is_q ? token * a.q_t + head * a.q_h : token * a.k_t + (head - a.Hq) * a.k_h;
  float* x = s_row[warp];
  float ss = 0.f;
  for (int i = lane; i < a.d; i += 32) {
    x[i] = load1(src, off + i, a.in_type);
    ss = fmaf(x[i], x[i], ss);
  }
  const void* weight = is_q ? a.qw : a.kw;
  if (weight) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float f = rsqrtf(ss / a.d + a.eps);
    for (int i = lane; i < a.d; i += 32) x[i] = x[i] * f * load1(weight, i, a.w_type);
  }
  __syncwarp();
  const int half = a.rot / 2;
  if (half) {
    const int pos = a.pos[token];
    for (int i = lane; i < half; i += 32) {
      float c, s;
      angle(a, pos, i, &c, &s);
      const int i0 = a.interleaved ? 2 * i : i, i1 = a.interleaved ? 2 * i + 1 : i + half;
      const float u = x[i0], v = x[i1];
      x[i0] = u * c - v * s;
      x[i1] = v * c + u * s;
    }
    __syncwarp();
  }
  void* dst = is_q ? a.qo : a.ko;
  const int type = is_q ? a.q_type : a.k_type;
  const long long out = is_q ? token * a.qo_t + head * a.qo_h : token * a.ko_t + (head - a.Hq) * a.ko_h;
  for (int i = lane; i < a.d; i += 32) store1(dst, out + i, type, x[i]);
}

int type_bytes(int type) { return type == CONFKV_FP32 ? 4 : type == CONFKV_FP16 || type == CONFKV_BF16 ? 2 : 0; }

// Every row starts on a 16-byte boundary.
bool aligned16(const void* p, const int64_t* stride, int bytes, long long n, long long heads) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (n < 2 || stride[0] * bytes % 16 == 0) &&
         (heads < 2 || stride[1] * bytes % 16 == 0);
}

// No two rows of an output share an element.
bool rows_apart(const int64_t* stride, int d, long long n, long long heads) {
  const long long t = stride[0], h = stride[1];
  if (n > 1 && t < d) return false;
  if (heads > 1 && h < d) return false;
  if (n > 1 && heads > 1) return t >= (heads - 1) * h + d || h >= (n - 1) * t + d;
  return true;
}

// An output that starts where its input does has the same rows.
bool same_place(const void* p, const int64_t* ps, const void* o, const int64_t* os, long long n, long long heads) {
  return p == o && (n < 2 || ps[0] == os[0]) && (heads < 2 || ps[1] == os[1]);
}

template <int TPR>
void launch_rows(RotArgs a, cudaStream_t st) {
  constexpr int groups = 256 / TPR;
  const int heads = a.Hq + a.Hkv;
  // Blocks of about six rows per thread group, whole tokens; with few
  // tokens, fewer rows and then parts of the heads, until the blocks cover the
  // GPU twice or a thread group has one row left.
  const int most = std::min(kMaxTokens, std::max(1, 6 * groups / heads));
  a.tokens = (int)std::max<long long>(1, std::min<long long>(most, a.n / 304));
  const long long blocks = ((long long)a.n + a.tokens - 1) / a.tokens;
  const int parts = (int)std::max<long long>(1, std::min<long long>((heads + groups - 1) / groups, 304 / blocks));
  a.heads = (heads + parts - 1) / parts;
  const dim3 grid((unsigned)blocks, (unsigned)((heads + a.heads - 1) / a.heads));
  const size_t smem = ((size_t)a.tokens * a.rot + 2 * 16 * TPR) * sizeof(float);
  auto kernel = a.in_type == CONFKV_FP32   ? rotary_rows_kernel<TPR, CONFKV_FP32>
                : a.in_type == CONFKV_BF16 ? rotary_rows_kernel<TPR, CONFKV_BF16>
                                           : rotary_rows_kernel<TPR, CONFKV_FP16>;
  launch_pdl(kernel, grid, dim3(256), smem, st, a);
}

}  // namespace
}  // namespace confkv

using namespace confkv;

extern "C" int confkv_rotary_frequencies(int32_t rot, double base, int32_t scaling, double factor,
                                         double original_length, double beta_fast, double beta_slow,
                                         uint64_t* turns, float* mscale) {
  if (!turns || !mscale || rot < 0 || rot % 2 || !(base > 1.0) || !std::isfinite(base)) return CONFKV_EINVAL;
  if (scaling < CONFKV_ROTARY_PLAIN || scaling > CONFKV_ROTARY_YARN) return CONFKV_EINVAL;
  if (scaling != CONFKV_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return CONFKV_EINVAL;
  if (scaling == CONFKV_ROTARY_NTK && rot == 2) return CONFKV_EINVAL;
  if (scaling == CONFKV_ROTARY_YARN &&
      (!(original_length > 0.0) || !std::isfinite(original_length) || !(beta_slow >= 0.0) ||
       !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
    return CONFKV_EINVAL;
  const double tau = 6.283185307179586476925286766559;
  if (scaling == CONFKV_ROTARY_NTK && rot > 2) base *= std::pow(factor, rot / (rot - 2.0));
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == CONFKV_ROTARY_LINEAR) f /= factor;
    if (scaling == CONFKV_ROTARY_YARN) {
      double keep = (original_length * f / tau - beta_slow) / (beta_fast - beta_slow);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f = f * keep + f / factor * (1.0 - keep);
    }
    turns[i] = (uint64_t)std::ldexp(f / tau, 64);          // f <= 1: below 2^62
  }
  *mscale = scaling == CONFKV_ROTARY_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return CONFKV_OK;
}

extern "C" int confkv_qk_rotary(const confkv_rotary_args* p, void* stream) {
  if (!p || p->n < 0 || p->Hq < 1 || p->Hkv < 0 || p->rot < 0 || p->rot % 2 || p->rot > p->d) return CONFKV_EINVAL;
  if (p->d < 1) return CONFKV_EINVAL;
  if (p->d > kMaxDim) return CONFKV_ENOTIMPL;
  const int in = type_bytes(p->in_dtype), wb = type_bytes(p->w_dtype), qb = type_bytes(p->q_out_dtype),
            kb = type_bytes(p->k_out_dtype);
  if (!in || !wb || !qb || !kb) return CONFKV_EINVAL;
  if (!std::isfinite(p->mscale) || ((p->q_weight || p->k_weight) && !(p->eps >= 0.f && std::isfinite(p->eps))))
    return CONFKV_EINVAL;
  if (p->n == 0) return CONFKV_OK;
  const bool keys = p->Hkv > 0;
  if (!p->q || !p->q_out || (keys && (!p->k || !p->k_out))) return CONFKV_EINVAL;
  if (p->rot && (!p->positions || !p->turns)) return CONFKV_EINVAL;
  auto at = [](const void* x, int a) { return reinterpret_cast<uintptr_t>(x) % a == 0; };
  if (!at(p->q, in) || !at(p->q_out, qb) || !at(p->positions, 4) || !at(p->turns, 8) || !at(p->q_weight, wb) ||
      (keys && (!at(p->k, in) || !at(p->k_out, kb) || !at(p->k_weight, wb))))
    return CONFKV_EINVAL;
  if (!rows_apart(p->q_out_stride, p->d, p->n, p->Hq)) return CONFKV_EINVAL;
  if (keys && !rows_apart(p->k_out_stride, p->d, p->n, p->Hkv)) return CONFKV_EINVAL;
  // an output over its input: the same elements in the same places
  if (p->q == p->q_out &&
      (p->in_dtype != p->q_out_dtype || !same_place(p->q, p->q_stride, p->q_out, p->q_out_stride, p->n, p->Hq)))
    return CONFKV_EINVAL;
  if (keys && p->k == p->k_out &&
      (p->in_dtype != p->k_out_dtype || !same_place(p->k, p->k_stride, p->k_out, p->k_out_stride, p->n, p->Hkv)))
    return CONFKV_EINVAL;
  RotArgs a{};
  a.n = p->n; a.Hq = p->Hq; a.Hkv = p->Hkv; a.d = p->d; a.rot = p->rot; a.interleaved = p->interleaved != 0;
  a.in_type = p->in_dtype; a.w_type = p->w_dtype; a.q_type = p->q_out_dtype; a.k_type = p->k_out_dtype;
  a.eps = p->eps; a.mscale = p->mscale;
  a.q = p->q; a.k = p->k; a.qo = p->q_out; a.ko = p->k_out;
  a.q_t = p->q_stride[0]; a.q_h = p->q_stride[1]; a.k_t = p->k_stride[0]; a.k_h = p->k_stride[1];
  a.qo_t = p->q_out_stride[0]; a.qo_h = p->q_out_stride[1];
  a.ko_t = p->k_out_stride[0]; a.ko_h = p->k_out_stride[1];
  a.qw = p->q_weight; a.kw = keys ? p->k_weight : nullptr;
  a.pos = p->positions; a.turns = p->turns;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const long long heads = (long long)p->Hq + p->Hkv;
  // Vectors of 8 channels: head sizes of 4, 8 or 16 threads, halves of the
  // rotated part in whole vectors, every row on a 16-byte boundary.
  const bool rows = (p->d == 64 || p->d == 128 || p->d == 256) && p->rot % 16 == 0 &&
                    aligned16(p->q, p->q_stride, in, p->n, p->Hq) &&
                    aligned16(p->q_out, p->q_out_stride, qb, p->n, p->Hq) &&
                    (!keys || (aligned16(p->k, p->k_stride, in, p->n, p->Hkv) &&
                               aligned16(p->k_out, p->k_out_stride, kb, p->n, p->Hkv))) &&
                    at(a.qw, 16) && at(a.kw, 16);
  if (rows) {
    const int tpr = p->d / 16;
    if (tpr == 4) launch_rows<4>(a, st);
    else if (tpr == 8) launch_rows<8>(a, st);
    else launch_rows<16>(a, st);
  } else {
    const long long blocks = ((long long)p->n * heads + kAnyWarps - 1) / kAnyWarps;
    if (blocks >= (1LL << 31)) return CONFKV_EINVAL;
    rotary_any_kernel<<<(unsigned)blocks, 32 * kAnyWarps, 0, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? CONFKV_OK : CONFKV_ECUDA;
}

// Attention of drafted tokens over the cache, few rows: up to 16 score rows
// (draft, query head of the group) of a KV head per CTA.
//
// The stored blocks of 16 tokens are laid out as the B operands of
// mma.m16n8k16: a warp reads 512 contiguous bytes at a time, has its operands
// in registers and needs no shared memory on the way.  Each warp of the
// cluster takes every so-many-th block, with the next ones in flight, and keeps
// a running reference, sum and output of all rows; the warps of a CTA, then the
// CTAs of the cluster, add up their parts.
//
// Queries of INT8 keys and all weights are two fp16 parts.  Up to eight rows
// take one product for both, the second part in rows 8 to 15, and the registers
// that saves hold a second block in flight.  The weights' second part took
// eight single tokens of five heads on 2049 entries from 18.6 to 18.9 us (cache
// not in L2); two drafts each, with a product of their own for it, 19.3 to 19.9.
//
// What bounds it: the latency of a warp's loads.  Eight single tokens on 2049
// entries, 40 heads on 8, 38 MB: 15 us on the device, 19 with nothing of it in L2
// (0.3 of the copy rate, eight warps an SM).  Copies through shared memory, a ring
// per warp, took a third longer.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cmath>

#include "../../include/confkv.h"
#include "confkv_internal.cuh"
#include "tree.cuh"

namespace cg = cooperative_groups;

namespace confkv {
namespace {

using namespace tree;

constexpr int kRows = 16, kWarps = 4;     // rows of a product; warps of a CTA

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// PAIR: rows 0 .. 7 of the score, whose second parts are rows 8 .. 15 of the
// operand; else rows 0 .. 15 and a second operand.
template <int D, bool BF16, bool PAIR>
struct Rows {
  static constexpr int kOf = PAIR ? 1 : 2;               // rows of a lane: g, and g + 8
  uint32_t q[kOf][D / 16][4];
  float unit[kOf];                                       // log2 units of a score's accumulator
  float ref[kOf], l[kOf];                                // reference and this lane's part of the sum
  float o[D / 8][4];

  // Rows r0 + g (and r0 + g + 8) with the channel scales `scale` (null: none,
  // and then the fp16 values are exact and the second parts zero).
  __device__ __forceinline__ void queries(const Call& a, const Shape& s, int b, int h, int r0, int used,
                                          const float* scale, int g, int t) {
#pragma unroll
    for (int i = 0; i < kOf; ++i) {
      const int r = r0 + g + 8 * i;
      const bool valid = r < used;
      const uint16_t* src = a.q + b * a.q_b + (valid ? r / s.G : 0) * a.q_t + (h * s.G + (valid ? r % s.G : 0)) * a.q_h;
      float2 x[D / 16][2];
      float most = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 16 * kk + 8 * e + 2 * t;
          x[kk][e] = valid ? float_pair<BF16>(*reinterpret_cast<const uint32_t*>(src + c)) : make_float2(0.f, 0.f);
          if (scale) {
            const float2 f = *reinterpret_cast<const float2*>(scale + c);
            x[kk][e].x *= f.x;
            x[kk][e].y *= f.y;
          }
          most = fmaxf(most, fmaxf(fabsf(x[kk][e].x), fabsf(x[kk][e].y)));
        }
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const float f = row_factor(most);
      unit[i] = row_unit(a, most);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t hi, lo;
          split2(x[kk][e].x * f, x[kk][e].y * f, hi, lo);
          q[0][kk][2 * e + i] = hi;
          q[kOf - 1][kk][2 * e + (PAIR ? 1 : i)] = PAIR || kOf == 2 ? lo : hi;
        }
    }
  }

  // Scores of eight keys whose operands are b(kk, b0, b1), in log2 units; hide
  // takes (row, column) of the lane's.  EXACT: fp16 keys, for which the query's
  // first part is exact and its second is left out (zero times an infinite key
  // would be NaN where the score is -inf).
  template <bool EXACT, typename B, typename Hide>
  __device__ __forceinline__ void scores(float (&x)[4], B operands, Hide hidden) {
    float c[2][4] = {};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t b0, b1;
      operands(kk, b0, b1);
      if (PAIR || EXACT) {
        mma(c[kk & 1], q[0][kk], b0, b1);
      } else {
        mma(c[0], q[0][kk], b0, b1);
        mma(c[1], q[kOf - 1][kk], b0, b1);
      }
    }
#pragma unroll
    for (int i = 0; i < kOf; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float y = PAIR && !EXACT ? (c[0][j] + c[1][j]) + (c[0][2 + j] + c[1][2 + j]) : c[0][2 * i + j] + c[1][2 * i + j];
        x[2 * i + j] = hidden(i, j) ? -INFINITY : y * unit[i];
      }
  }

  // Weights of 16 keys from their scores, in two fp16 parts: PAIR as an
  // operand, like the queries, which costs no product; else as two.
  __device__ __forceinline__ void weights(float (&x)[2][4], uint32_t (&p)[4], uint32_t (&p2)[4]) {
    float top[kOf];
    bool move = false;
#pragma unroll
    for (int i = 0; i < kOf; ++i) {
      top[i] = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
      move |= top[i] > ref[i] + kLag;
    }
    if (__any_sync(0xffffffffu, move)) {
      float f[kOf];
#pragma unroll
      for (int i = 0; i < kOf; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        f[i] = top[i] > ref[i] ? ex2(ref[i] - top[i]) : 1.f;       // 0 for the first key
        ref[i] = fmaxf(ref[i], top[i]);
        l[i] *= f[i];
      }
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        o[j][0] *= f[0];
        o[j][1] *= f[0];
        o[j][2] *= f[kOf - 1];
        o[j][3] *= f[kOf - 1];
      }
    }
#pragma unroll
    for (int i = 0; i < kOf; ++i) {
      const float base = ref[i] == -INFINITY ? 0.f : kLift - ref[i];
      float e[2][2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) e[nt][j] = ex2(x[nt][2 * i + j] + base);
      l[i] += (e[0][0] + e[0][1]) + (e[1][0] + e[1][1]);
      if (PAIR) {
        split2(e[0][0], e[0][1], p[0], p[1]);
        split2(e[1][0], e[1][1], p[2], p[3]);
      } else {
        split2(e[0][0], e[0][1], p[i], p2[i]);
        split2(e[1][0], e[1][1], p[2 + i], p2[2 + i]);
      }
    }
  }
};

template <int D, bool BF16, bool PAIR>
__global__ void __launch_bounds__(kWarps * 32)
    tree_rows_kernel(Shape s, Dev d, const __grid_constant__ Call a) {
  constexpr int NC = D / 32, kPitch = D + 4, kMine = PAIR ? 8 : 16;      // rows of a CTA
  constexpr int kAhead = PAIR ? 2 : 1;                   // blocks in flight
  __shared__ __align__(16) float s_part[kWarps][kRows][kPitch];
  __shared__ float2 s_stat[kWarps][kRows];
  __shared__ float2 s_sum[kRows];
  __shared__ uint4 s_path[kMaxDrafts];
  __shared__ int s_up[kMaxDrafts];
  __shared__ uint32_t s_bad[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = a.split, rank = blockIdx.x % split;
  const int tile = blockIdx.x / split % a.tiles, bh = blockIdx.x / split / a.tiles, b = bh / s.Hkv, h = bh % s.Hkv;
  pdl_wait();
  const int drafts = drafts_of(a, b), r0 = tile * kMine, used = drafts * s.G, all = a.T * s.G;
  const int end = min(r0 + kMine, used);                 // rows of this tile that have a draft
  if (threadIdx.x < 4) s_bad[threadIdx.x] = 0;
  draft_paths<kWarps * 32>(a, b, drafts, threadIdx.x, s_path, s_up, [] { __syncthreads(); });

  // rows without a draft see nothing
  if (rank == 0) {
    for (int i = max(r0, used) * (D / 8) + threadIdx.x; i < min(r0 + kMine, all) * (D / 8); i += blockDim.x) {
      const int r = i / (D / 8), c = i % (D / 8) * 8;
      *reinterpret_cast<uint4*>(a.out + b * a.o_b + r / s.G * a.o_t + (h * s.G + r % s.G) * a.o_h + c) =
          make_uint4(0, 0, 0, 0);
      if (a.lse && c == 0) a.lse[((long long)b * a.T + r / s.G) * s.Hq + h * s.G + r % s.G] = -INFINITY;
    }
  }
  if (r0 >= used) return;                                // the whole cluster

  const size_t lb = lb_index(s, a.layer, b), u = unit_index(s, a.layer, b, h);
  const int n8 = d.n8[lb], nb8 = (n8 + 15) / 16, ring = s.WR / 16;
  const int seen = (end - 1) / s.G + 1;                  // drafts up to the last row's own
  const int nbf = ring + (seen + 15) / 16;
  const int workers = split * kWarps, me = rank * kWarps + warp;

  Rows<D, BF16, PAIR> w;
#pragma unroll
  for (int i = 0; i < w.kOf; ++i) {
    w.ref[i] = -INFINITY;
    w.l[i] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < D / 8; ++j) w.o[j][0] = w.o[j][1] = w.o[j][2] = w.o[j][3] = 0.f;

  // ---- INT8 blocks
  if (me < nb8) {
    const uint8_t* kp = d.k8 + u * s.cstride * D + lane * 16;
    const uint8_t* vp = d.v8 + u * s.cstride * D + lane * 16;
    uint4 kn[kAhead][NC], vn[kAhead][NC];
    auto fetch = [&](int i, int at) {
#pragma unroll
      for (int r = 0; r < NC; ++r) {
        kn[at][r] = *reinterpret_cast<const uint4*>(kp + (size_t)i * 16 * D + r * 512);
        vn[at][r] = *reinterpret_cast<const uint4*>(vp + (size_t)i * 16 * D + r * 512);
      }
    };
#pragma unroll
    for (int at = 0; at < kAhead; ++at)
      if (me + at * workers < nb8) fetch(me + at * workers, at);
    w.queries(a, s, b, h, r0, used, d.sK + u * D, g, t);
    for (int i0 = me; i0 < nb8; i0 += kAhead * workers) {
#pragma unroll
      for (int at = 0; at < kAhead; ++at) {
        const int i = i0 + at * workers;
        if (i >= nb8) break;
        float x[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int left = n8 - i * 16 - nt * 8 - 2 * t;   // entries from this lane's first key on
          w.template scores<false>(
              x[nt], [&](int kk, uint32_t& b0, uint32_t& b1) { codes(word(kn[at][nt * (NC / 2) + (kk >> 2)], kk & 3), b0, b1); },
              [&](int, int j) { return j >= left; });
        }
        uint4 vc[NC];
#pragma unroll
        for (int r = 0; r < NC; ++r) vc[r] = vn[at][r];
        if (i + kAhead * workers < nb8) fetch(i + kAhead * workers, at);
        uint32_t p[4], p2[4];
        w.weights(x, p, p2);
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          uint32_t b0, b1;
          codes(word(vc[j >> 2], j & 3), b0, b1);
          mma(w.o[j], p, b0, b1);
          if (!PAIR) mma(w.o[j], p2, b0, b1);
        }
      }
    }
    const float* sv = d.sV + u * D + 2 * t;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      const float2 f = *reinterpret_cast<const float2*>(sv + 8 * j);
      w.o[j][0] *= f.x;
      w.o[j][1] *= f.y;
      w.o[j][2] *= f.x;
      w.o[j][3] *= f.y;
    }
  }

  // ---- fp16 blocks: the window, then the drafts
  int first = (me - nb8) % workers;
  if (first < 0) first += workers;
  if (first < nbf) w.queries(a, s, b, h, r0, used, nullptr, g, t);
  for (int i = first; i < nbf; i += workers) {
    uint4 kc[2 * NC], vc[2 * NC];
    uint32_t see[2];                                     // keys of the block that rows g and g + 8 see
    if (i < ring) {
      const size_t at = (u * ring + i) * 32 * D + lane * 16;
      const int pos = d.pos[lb * s.S + s.cap + i * 16 + (lane & 15)];
#pragma unroll
      for (int r = 0; r < 2 * NC; ++r) {
        kc[r] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(d.k16) + at + r * 512);
        vc[r] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(d.v16) + at + r * 512);
      }
      see[0] = see[1] = __ballot_sync(0xffffffffu, pos >= 0) & 0xffffu;
      // an empty slot may hold anything: its values are cleared
      const uint32_t m0 = (see[0] >> (2 * t) & 1 ? 0xffffu : 0u) | (see[0] >> (2 * t + 1) & 1 ? 0xffff0000u : 0u);
      const uint32_t m1 = (see[0] >> (2 * t + 8) & 1 ? 0xffffu : 0u) | (see[0] >> (2 * t + 9) & 1 ? 0xffff0000u : 0u);
      if (see[0] != 0xffffu)
#pragma unroll
        for (int r = 0; r < 2 * NC; ++r) vc[r] = make_uint4(vc[r].x & m0, vc[r].y & m1, vc[r].z & m0, vc[r].w & m1);
    } else {
      const int base = (i - ring) * 16;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + g + 8 * e;
        const uint4 m = s_path[min(r, used - 1) / s.G];
        see[e] = r < used ? word(m, base >> 5) >> (base & 16) & 0xffffu : 0u;
      }
      // made up like a block of the window, in the place of this warp's part
      const uint32_t to = tc::smem_addr(&s_part[warp][0][0]);
      const int tau = lane & 15, tok = base + tau;
      const uint16_t *kp = a.k + b * a.k_b + tok * a.k_t + h * a.k_h, *vp = a.v + b * a.v_b + tok * a.v_t + h * a.v_h;
      bool bad = false;
      __syncwarp();
#pragma unroll 2
      for (int c = 8 * (lane >> 4); c < D; c += 16) {
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (tok < drafts) {
          x = *reinterpret_cast<const uint4*>(kp + c);
          y = *reinterpret_cast<const uint4*>(vp + c);
        }
        const uint32_t kd = to + k16_offset(D, tau, c), vd = to + 32 * D + v16_offset(D, tau, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {                    // channels c + 2 j, + 1
          asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(kd + 16 * j), "r"(half_pair<BF16>(word(x, j))) : "memory");
          uint32_t z = half_pair<BF16>(word(y, j));
          // a value that is not finite is marked and taken as zero
          if ((z & 0x7c00u) == 0x7c00u) z &= 0xffff0000u, bad = true;
          if ((z & 0x7c000000u) == 0x7c000000u) z &= 0xffffu, bad = true;
          asm volatile("st.shared.b16 [%0], %1;\n" ::"r"(vd + 128 * j), "h"((unsigned short)z) : "memory");
          asm volatile("st.shared.b16 [%0], %1;\n" ::"r"(vd + 128 * j + 64), "h"((unsigned short)(z >> 16)) : "memory");
        }
      }
      if (bad) atomicOr(&s_bad[tok >> 5], 1u << (tok & 31));
      __syncwarp();
#pragma unroll
      for (int r = 0; r < 2 * NC; ++r) {
        kc[r] = lds(to + r * 512 + lane * 16);
        vc[r] = lds(to + 32 * D + r * 512 + lane * 16);
      }
    }
    float x[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
      w.template scores<true>(
          x[nt],
          [&](int kk, uint32_t& b0, uint32_t& b1) {
            const uint4& y = kc[nt * NC + (kk >> 1)];
            b0 = word(y, 2 * (kk & 1));
            b1 = word(y, 2 * (kk & 1) + 1);
          },
          [&](int e, int j) { return !(see[e] >> (8 * nt + 2 * t + j) & 1); });
    uint32_t p[4], p2[4];
    w.weights(x, p, p2);
    // An infinite value times a second part, which may be zero or negative, would
    // be NaN; x * 0 finds those that are not finite.
    const __half2 zero = __float2half2_rn(0.f);
    __half2 not_finite = zero;
#pragma unroll
    for (int r = 0; r < 2 * NC; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t y = word(vc[r], j);
        not_finite = __hfma2(*reinterpret_cast<const __half2*>(&y), zero, not_finite);
      }
    if (!__any_sync(0xffffffffu, !__hbeq2(not_finite, zero))) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const uint4& y = vc[j >> 1];
        mma(w.o[j], p, word(y, 2 * (j & 1)), word(y, 2 * (j & 1) + 1));
        if (!PAIR) mma(w.o[j], p2, word(y, 2 * (j & 1)), word(y, 2 * (j & 1) + 1));
      }
    } else {                                             // the first part alone
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const uint4& y = vc[j >> 1];
        const float second[2] = {w.o[j][2], w.o[j][3]};
        mma(w.o[j], p, word(y, 2 * (j & 1)), word(y, 2 * (j & 1) + 1));
        if (PAIR) w.o[j][2] = second[0], w.o[j][3] = second[1];
      }
    }
  }

  // ---- the parts of the warps
#pragma unroll
  for (int i = 0; i < w.kOf; ++i) {
    w.l[i] += __shfl_xor_sync(0xffffffffu, w.l[i], 1);
    w.l[i] += __shfl_xor_sync(0xffffffffu, w.l[i], 2);
    if (t == 0) s_stat[warp][g + 8 * i] = make_float2(w.ref[i], w.l[i]);
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
      *reinterpret_cast<float2*>(&s_part[warp][g + 8 * i][8 * j + 2 * t]) =
          PAIR ? make_float2(w.o[j][0] + w.o[j][2], w.o[j][1] + w.o[j][3]) : make_float2(w.o[j][2 * i], w.o[j][2 * i + 1]);
  }
  __syncthreads();
  constexpr int kCols = D / 4;
  for (int i = threadIdx.x; i < (end - r0) * kCols; i += blockDim.x) {
    const int r = i / kCols, c = i % kCols * 4;
    float top = -INFINITY, sum = 0.f, y[4] = {};
#pragma unroll
    for (int k = 0; k < kWarps; ++k) top = fmaxf(top, s_stat[k][r].x);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float2 z = s_stat[k][r];
      const float f = z.x == top ? 1.f : ex2(z.x - top);
      const float4 v = *reinterpret_cast<const float4*>(&s_part[k][r][c]);
      sum += z.y * f;
      y[0] += v.x * f;
      y[1] += v.y * f;
      y[2] += v.z * f;
      y[3] += v.w * f;
    }
    *reinterpret_cast<float4*>(&s_part[0][r][c]) = make_float4(y[0], y[1], y[2], y[3]);
    if (c == 0) s_sum[r] = make_float2(top, sum);
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (split > 1)
    cluster.sync();
  else
    __syncthreads();

  // ---- the parts of the CTAs, each its share of the rows
  for (int i = rank + split * (threadIdx.x / kCols); i < end - r0; i += split * (kWarps * 32 / kCols)) {
    const int c = threadIdx.x % kCols * 4, r = r0 + i, tok = r / s.G, head = h * s.G + r % s.G;
    float4 y[kMaxSplit];
    float2 z[kMaxSplit];
    uint32_t bad[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kMaxSplit; ++k)
      if (k < split) {
        const float* part = split > 1 ? cluster.map_shared_rank(&s_part[0][0][0], k) : &s_part[0][0][0];
        const float2* sum = split > 1 ? cluster.map_shared_rank(s_sum, k) : s_sum;
        const uint32_t* mark = split > 1 ? cluster.map_shared_rank(s_bad, k) : s_bad;
        y[k] = *reinterpret_cast<const float4*>(part + i * kPitch + c);
        z[k] = sum[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) bad[j] |= mark[j];
      }
    float top = -INFINITY, sum = 0.f, x[4] = {};
#pragma unroll
    for (int k = 0; k < kMaxSplit; ++k)
      if (k < split) top = fmaxf(top, z[k].x);
#pragma unroll
    for (int k = 0; k < kMaxSplit; ++k)
      if (k < split) {
        const float f = z[k].x == top ? 1.f : ex2(z[k].x - top);
        sum += z[k].y * f;
        x[0] += y[k].x * f;
        x[1] += y[k].y * f;
        x[2] += y[k].z * f;
        x[3] += y[k].w * f;
      }
    const float inv = 1.f / sum;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] *= inv;
    if (bad[0] | bad[1] | bad[2] | bad[3])
      for (int j = 0; j < 4; ++j) x[j] += unfinite<BF16>(a, b, h, s_path[tok], bad, c + j);
    *reinterpret_cast<uint2*>(a.out + b * a.o_b + tok * a.o_t + head * a.o_h + c) =
        make_uint2(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]));
    if (a.lse && c == 0)
      a.lse[((long long)b * a.T + tok) * s.Hq + head] =
          (top == -INFINITY ? 0.f : top * 0.6931471805599453f) + logf(sum * kUnlift);
  }
  if (split > 1) cluster.sync();                         // no CTA leaves while another reads its part
}

template <int D, bool BF16, bool PAIR>
int launch(const Shape& s, const Dev& d, const Call& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)s.B * s.Hkv * a.tiles * a.split));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = a.split;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, tree_rows_kernel<D, BF16, PAIR>, s, d, a) == cudaSuccess ? 0 : -1;
}

}  // namespace

// Time in microseconds by a model: 1, and for each wave of the CTAs that fit (two
// per SM, four of 64 channels) a start and a join and what a warp takes for its
// blocks, the longer the more CTAs share the memory: with 128 channels 0.44 a
// block on an idle GPU, 0.79 with a CTA on every SM and 0.99 with two.  Fitted to
// 75 calls of 9 to 512 rows with equal lengths, to a tenth: 9 rows on 2889
// entries 12 us measured (11), 16 rows of 64 units on 5266 27 (28), 64 of 48 on
// 3956 37 (36).  Up to eight rows 0.45 to 0.70; they always take this kernel, and
// only the split follows.
double plan_tree_rows(const Shape& s, int T, long long n8_bound, int* split) {
  const bool pair = T * s.G <= 8;
  const int mine = pair ? 8 : kRows;
  const long long tiles = ((long long)T * s.G + mine - 1) / mine, units = (long long)s.B * s.Hkv * tiles;
  const long long blocks = (n8_bound + 15) / 16 + s.WR / 16 + (T + 15) / 16, slots = s.D == 128 ? 304 : 608;
  double least = 1e30;
  for (int k = 1; k <= kMaxSplit; k *= 2) {              // clusters of other sizes leave more SMs idle
    if (k > 1 && units * k > slots) break;
    // us for a block of every warp of a CTA, by the CTAs of an SM
    const double of_sm = (double)(units * k) / 152, first = std::min(of_sm, 1.0), second = std::min(std::max(of_sm - 1, 0.0), 1.0);
    const double each = s.D != 128 ? std::max(0.42, 0.21 * std::min(4.0, std::ceil(of_sm)))
                        : pair     ? 0.45 + 0.25 * second
                                   : 0.44 + 0.35 * first + 0.2 * second;
    const double wave = s.D == 128 && !pair ? 7.0 : 6.0;
    const long long waves = (units * k + slots - 1) / slots;
    const double t = 1.0 + wave * (double)waves + each * (double)(waves * ((blocks + kWarps * k - 1) / (kWarps * k))) + (k > 1 ? 0.5 : 0.0);
    if (t < least) {
      least = t;
      *split = k;
    }
  }
  return least;
}

int launch_tree_rows(const Shape& s, const Dev& d, const tree::Call& call, bool bf16, cudaStream_t st) {
  tree::Call a = call;
  const bool pair = a.T * s.G <= 8;
  a.tiles = pair ? 1 : (a.T * s.G + kRows - 1) / kRows;
  auto of = [&](auto fn_bf16, auto fn_f16) { return bf16 ? fn_bf16(s, d, a, st) : fn_f16(s, d, a, st); };
  if (s.D == 128) return pair ? of(launch<128, true, true>, launch<128, false, true>) : of(launch<128, true, false>, launch<128, false, false>);
  return pair ? of(launch<64, true, true>, launch<64, false, true>) : of(launch<64, true, false>, launch<64, false, false>);
}

}  // namespace confkv

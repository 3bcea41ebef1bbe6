// One layer of the cache from and to packed K/V.
//
// Write: the rows of all sequences one after another (no padding), fp16 or
// bf16.  The rule is that of the whole-cache prefill: per (layer, sequence,
// KV head, channel) s = absmax / 127 over the prompt, codes
// clamp(rint(x / s), -127, 127) for all but the newest W tokens, which stay
// fp16 (CONF-KV, gist.science/de/paper/2605.24786, Technischer
// Zusammenfassung, Systemintegration: INT8 per head and per channel).
// A cluster of CTAs takes the K or the V of one (sequence, KV head): its CTAs
// reduce the absmax of their tokens, exchange it through distributed shared
// memory, and then place 16-token blocks, so that one launch does both passes
// and the second one finds the rows in L2.
//
// Read: the resident entries of a layer, dequantised, as packed rows: INT8
// entries in slot order, then the FP16 window by position.
//
// Both move a few bytes per value.  Eight prompts of 4096 tokens, 8 KV heads,
// d = 128: the write takes 73 us for 134 MB read and 71 MB written (30 of
// them the absmax pass, at 4.4 TB/s; then the quantising instructions), the
// read 40 us for 71 MB and 134 MB (5.1 TB/s).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>

#include "../../include/confkv.h"
#include "confkv_internal.cuh"
#include "fp32_pair.cuh"

namespace cg = cooperative_groups;

namespace confkv {
namespace {

constexpr int kChunk = 544;          // shared-memory pitch of a 512-byte piece of an interleaved block
constexpr int kWriteWarps = 8;
constexpr int kMaxCtas = 8;           // CTAs per cluster of the write
constexpr int kReadWarps = 8;

// ------------------------------------------------------------------ reset

__global__ void prefill_reset_kernel(Shape s, Dev d, const __grid_constant__ LengthChunk c) {
  pdl_wait();
  for (int i = threadIdx.x; i < c.count; i += blockDim.x) {
    d.T0[c.first + i] = c.len[i];
    d.conf_done[c.first + i] = 0;
    d.conf_ready[c.first + i] = 0;
  }
  for (int i = threadIdx.x; i < c.count * s.L; i += blockDim.x)
    d.arrive[(size_t)(i / c.count) * s.B + c.first + i % c.count] = 0;
  if (threadIdx.x == 0) {            // packed row of each sequence
    long long row = c.row0;
    for (int i = 0; i < c.count; ++i) {
      d.row0[c.first + i] = row;
      row += c.len[i];
    }
    if (c.first == 0) {
      *d.status = 0;
      *d.step_dev = 0;
      *d.sel_done = 0;
    }
  }
  if (c.first == 0)
    for (size_t i = threadIdx.x; i < sizeof(DevStats) / 4; i += blockDim.x) reinterpret_cast<uint32_t*>(d.stats)[i] = 0;
}

// ------------------------------------------------------------------ write

// Two source values as fp16 (an overflow becomes infinite).
template <bool BF16>
__device__ __forceinline__ __half2 half_pair(uint32_t w) {
  if (BF16) return __floats2half2_rn(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return *reinterpret_cast<const __half2*>(&w);
}

// Larger absolute value of each half of two words; a NaN loses.
template <bool BF16>
__device__ __forceinline__ uint32_t max_abs(uint32_t top, uint32_t w) {
  w &= 0x7fff7fffu;
  if (BF16) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&top),
                                     *reinterpret_cast<const __nv_bfloat162*>(&w));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&top), *reinterpret_cast<const __half2*>(&w));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// 8 values as words whose low byte is clamp(rint(x / s), -127, 127) + 128,
// with the IEEE quotient.  x * (1 / s) is within 2 ulp of it (2^-15 up to
// 127), so the integers agree unless the product lies that close to a half.
// Adding 1.5 2^23 + 128 rounds to an integer (ties to even) and leaves the
// stored byte in the low bits.  No clamp: |x| <= 127 s (1 + 2^-23).
//
// Next to the half-integer h: the sign of e = x - h s, which one fused
// multiply-add gives (and exactly where e is small: h s has at most 32 bits),
// says on which side the quotient lies, and |e| <= s ulp(h) / 2 that it
// rounds to h itself, a tie (to even).  Below 1/2 the spacing is half as
// wide.  No quotient of two floats lies midway between two others.
__device__ __noinline__ uint32_t code_next_to_half(float x, float s, float n, float off) {
  const float h = n + copysignf(0.5f, off);
  const float e = fmaf(-h, s, x);
  float step = __uint_as_float((__float_as_uint(h) & 0x7f800000u) - (24u << 23));
  if (fabsf(h) == 0.5f && (e < 0.f) == (h > 0.f)) step *= 0.5f;
  const float c = fabsf(e) <= s * step ? rintf(h) : e > 0.f ? h + 0.5f : h - 0.5f;
  return (uint32_t)((int)fminf(fmaxf(c, -127.f), 127.f) + kCodeBias);     // a NaN becomes -127
}
template <bool BF16>
__device__ __forceinline__ void quantise8(const uint4& raw, const float (&scale)[8], const float (&inv)[8],
                                          uint32_t (&r)[8]) {
  constexpr float kRound = 12582912.f + 128.f;
  float x[8], q[8];
  bool near = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(half_pair<BF16>((&raw.x)[j]));
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const Pair p = Pair(x[j], x[j + 1]) * Pair(inv[j], inv[j + 1]), whole = p + Pair(kRound, kRound);
    const Pair off = fma2(whole + Pair(-kRound, -kRound), Pair(-1.f, -1.f), p);
    near |= !(fabsf(off.get().x) <= 0.49993f);
    near |= !(fabsf(off.get().y) <= 0.49993f);
    q[j] = p.get().x;
    q[j + 1] = p.get().y;
    r[j] = __float_as_uint(whole.get().x);
    r[j + 1] = __float_as_uint(whole.get().y);
  }
  if (near) {                                          // not rare for a channel whose absmax has few bits
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float n = __uint_as_float(r[j]) - kRound, off = q[j] - n;
      if (!(fabsf(off) <= 0.49993f)) r[j] = code_next_to_half(x[j], scale[j], n, off);
    }
  }
}

template <int D, bool BF16, bool IS_V>
__device__ __forceinline__ void write_unit(const Shape& s, const Dev& d, int layer, int b, int h,
                                           const uint16_t* __restrict__ src, long long ts, uint8_t* smem,
                                           uint32_t* s_abs) {
  constexpr int kPer = D / 8;                          // threads per row
  constexpr int kRowsAtOnce = kWriteWarps * 32 / kPer;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int T0 = d.T0[b], n8 = max(0, T0 - s.W);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ch = threadIdx.x % kPer;                   // 8-channel chunk of this thread
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");   // this CTA's shared memory is there
  const size_t lb = lb_index(s, layer, b), u = unit_index(s, layer, b, h);
  auto row = [&](long long t) { return *reinterpret_cast<const uint4*>(src + t * ts + ch * 8); };

  // ---- absmax over the CTA's share of the tokens (fp16 rounding keeps the
  // order, so bf16 maxima are converted at the end)
  uint32_t top[4] = {0, 0, 0, 0};
  {
    const int per = (T0 + ctas - 1) / ctas, t1 = min(T0, (rank + 1) * per);
    int t = rank * per + threadIdx.x / kPer;
    for (; t + 7 * kRowsAtOnce < t1; t += 8 * kRowsAtOnce) {
      uint4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = row(t + i * kRowsAtOnce);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) top[j] = max_abs<BF16>(top[j], (&x[i].x)[j]);
    }
    for (; t < t1; t += kRowsAtOnce) {
      const uint4 x = row(t);
#pragma unroll
      for (int j = 0; j < 4; ++j) top[j] = max_abs<BF16>(top[j], (&x.x)[j]);
    }
  }
#pragma unroll
  for (int o = kPer; o < 32; o <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) top[j] = max_abs<BF16>(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
  uint32_t* stage = reinterpret_cast<uint32_t*>(smem); // [warp][D / 2]
  if (lane < kPer)
#pragma unroll
    for (int j = 0; j < 4; ++j) stage[warp * (D / 2) + ch * 4 + j] = top[j];
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
  // every CTA sends its maxima to all of the cluster before the one barrier,
  // so that each reads them locally and may leave when it is done
  for (int i = threadIdx.x; i < ctas * (D / 2); i += blockDim.x) {
    const int c = i % (D / 2), to = i / (D / 2);
    uint32_t m = stage[c];
#pragma unroll
    for (int w = 1; w < kWriteWarps; ++w) m = max_abs<BF16>(m, stage[w * (D / 2) + c]);
    *cluster.map_shared_rank(&s_abs[rank * (D / 2) + c], to) = m;
  }
  cluster.sync();
  float scale[8], inv[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t m = 0;
    for (int r = 0; r < ctas; ++r) m = max_abs<BF16>(m, s_abs[r * (D / 2) + ch * 4 + j]);
    const float2 f = __half22float2(half_pair<BF16>(m));
    scale[2 * j] = f.x > 0.f ? __fdiv_rn(f.x, 127.f) : 1.f;
    scale[2 * j + 1] = f.y > 0.f ? __fdiv_rn(f.y, 127.f) : 1.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) inv[i] = __fdiv_rn(1.f, scale[i]);
  if (rank == 0 && threadIdx.x < kPer) {
    float* dst = (IS_V ? d.sV : d.sK) + u * D + ch * 8;
    *reinterpret_cast<float4*>(dst) = make_float4(scale[0], scale[1], scale[2], scale[3]);
    *reinterpret_cast<float4*>(dst + 4) = make_float4(scale[4], scale[5], scale[6], scale[7]);
  }

  // ---- blocks: ceil(n8 / 16) of codes, then the ring
  uint8_t* blk = smem + warp * (D / 16) * kChunk;
  // A lane takes tokens 2t, 2t + 1, 2t + 8 and 2t + 9 of its channels: the
  // four bytes of a V word (v8_offset).
  constexpr int kRowsPerWarp = 32 / kPer, kIter = 16 / kRowsPerWarp, kQuads = kIter / 4;
  auto token = [&](int r) { return 2 * (lane / kPer + kRowsPerWarp * (r >> 2)) + (r & 1) + 4 * (r & 2); };
  const int nb8 = (n8 + 15) / 16, step = ctas * kWriteWarps;
  int i = rank * kWriteWarps + warp;
  for (; i < nb8; i += step) {
#pragma unroll 1
    for (int quad = 0; quad < kQuads; ++quad) {
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = i * 16 + token(quad * 4 + j);
        x[j] = p < n8 ? row(p) : make_uint4(0, 0, 0, 0);
      }
      if (IS_V) {
        uint32_t word[8], r[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          quantise8<BF16>(x[j], scale, inv, r);
#pragma unroll
          for (int c = 0; c < 8; ++c)                  // byte j of each channel's word
            word[c] = j == 0 ? r[c] : __byte_perm(word[c], r[c], j == 1 ? 0x3240 : j == 2 ? 0x3410 : 0x4210);
        }
        uint8_t* o = blk + (ch >> 2) * kChunk + (ch & 3) * 4 + (lane / kPer + kRowsPerWarp * quad) * 16;
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint32_t*>(o + c * 64) = word[c];
      } else {                                         // k8_offset
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t r[8];
          quantise8<BF16>(x[j], scale, inv, r);
          const int tau = token(quad * 4 + j);
          uint8_t* o = blk + ((ch >> 3) + (tau >> 3) * (D / 64)) * kChunk + ((ch >> 1) & 3) * 4 + (ch & 1) * 2 +
                       (tau & 7) * 64;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint16_t*>(o + c * 16) = (uint16_t)__byte_perm(r[2 * c], r[2 * c + 1], 0x0040);
        }
      }
    }
    __syncwarp();
    uint8_t* dst = (IS_V ? d.v8 : d.k8) + (u * (s.cstride / 16) + i) * 16 * D;
#pragma unroll
    for (int r = 0; r < D / 32; ++r)
      *reinterpret_cast<uint4*>(dst + r * 512 + lane * 16) = *reinterpret_cast<const uint4*>(blk + r * kChunk + lane * 16);
    __syncwarp();
  }
  for (i -= nb8; i < s.WR / 16; i += step) {
#pragma unroll
    for (int r = 0; r < kIter; ++r) {                  // the newest position that falls on each slot
      const int tau = token(r);
      const int p = T0 - 1 - ((T0 - 1 - (i * 16 + tau)) % s.WR + s.WR) % s.WR;
      const uint4 x = p >= n8 ? row(p) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 v = half_pair<BF16>((&x.x)[j]);
        const int o0 = IS_V ? v16_offset(D, tau, ch * 8 + 2 * j) : k16_offset(D, tau, ch * 8 + 2 * j);
        const int o1 = IS_V ? v16_offset(D, tau, ch * 8 + 2 * j + 1) : o0 + 2;
        *reinterpret_cast<__half*>(blk + (o0 >> 9) * kChunk + (o0 & 511)) = __low2half(v);
        *reinterpret_cast<__half*>(blk + (o1 >> 9) * kChunk + (o1 & 511)) = __high2half(v);
      }
    }
    __syncwarp();
    uint8_t* dst = reinterpret_cast<uint8_t*>(IS_V ? d.v16 : d.k16) + (u * (s.WR / 16) + i) * 32 * D;
#pragma unroll
    for (int r = 0; r < D / 16; ++r)
      *reinterpret_cast<uint4*>(dst + r * 512 + lane * 16) = *reinterpret_cast<const uint4*>(blk + r * kChunk + lane * 16);
    __syncwarp();
  }
  // ---- positions and EMA of the layer's slots, by the K of KV head 0
  if (h == 0 && !IS_V) {
    for (int i = rank * blockDim.x + threadIdx.x; i < s.S; i += ctas * blockDim.x) {
      int p = -1;
      if (i < n8) {
        p = i;
      } else if (i >= s.cap) {
        const int at = T0 - 1 - ((T0 - 1 - (i - s.cap)) % s.WR + s.WR) % s.WR;
        p = at >= n8 ? at : -1;
      }
      d.pos[lb * s.S + i] = p;
      d.ema[lb * s.S + i] = 0.f;
    }
    if (rank == 0 && threadIdx.x == 0) d.n8[lb] = n8;
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kWriteWarps * 32, 3)
    write_layer_kernel(Shape s, Dev d, int layer, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                       long long k_t, long long k_h, long long v_t, long long v_h) {
  extern __shared__ __align__(16) uint8_t smem[];      // an interleaved block per warp
  __shared__ uint32_t s_abs[kMaxCtas * (D / 2)];       // absmax of each CTA's tokens, channel pairs
  pdl_wait();
  const int unit = blockIdx.x / (int)cg::this_cluster().num_blocks();   // (sequence, KV head, K or V)
  const int h = (unit >> 1) % s.Hkv, b = (unit >> 1) / s.Hkv;
  if (unit & 1)
    write_unit<D, BF16, true>(s, d, layer, b, h, v + d.row0[b] * v_t + h * v_h, v_t, smem, s_abs);
  else
    write_unit<D, BF16, false>(s, d, layer, b, h, k + d.row0[b] * k_t + h * k_h, k_t, smem, s_abs);
}

// ------------------------------------------------------------------ read

// cu[b + 1]: entries of sequences 0 .. b.
__global__ void __launch_bounds__(1024) count_entries_kernel(Shape s, Dev d, int layer, int32_t* __restrict__ cu) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int b = warp; b < s.B; b += 32) {
    const size_t lb = lb_index(s, layer, b);
    int n = 0;
    for (int i = lane; i < s.WR; i += 32) n += d.pos[lb * s.S + s.cap + i] >= 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) cu[b + 1] = n + d.n8[lb];
  }
  __syncthreads();
  if (warp == 0) {
    int before = 0;
    for (int b0 = 0; b0 < s.B; b0 += 32) {
      int x = b0 + lane < s.B ? cu[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < s.B) cu[b0 + lane + 1] = before + x;
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) cu[0] = 0;
  }
}

// 8 stored bytes as codes times scales, in the output type.
__device__ __forceinline__ uint4 dequantise(uint2 w, const float* scale, bool bf16) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t word = i < 2 ? w.x : w.y;
    const float a = __uint_as_float(__byte_perm(word, 0x4b000000u, 0x7540 + 2 * (i & 1))) - 8388736.f;   // 2^23 + 128
    const float b = __uint_as_float(__byte_perm(word, 0x4b000000u, 0x7540 + 2 * (i & 1) + 1)) - 8388736.f;
    const float x = a * scale[2 * i], y = b * scale[2 * i + 1];
    if (bf16) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
      o[i] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
      const __half2 p = __floats2half2_rn(x, y);
      o[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Sequences whose entries every CTA of the read kernel counts by itself.
// Counting in a launch of its own costs about 4 us before the read can start;
// the CTAs' own counts read B * WR positions each, which for more sequences
// is more than their blocks.
constexpr int kCountHere = 16;

template <int D, bool BF16>
__global__ void __launch_bounds__(kReadWarps * 32, 4)
    read_layer_kernel(Shape s, Dev d, int layer, int spans, int per_warp, int counted, int32_t* __restrict__ cu,
                      uint16_t* __restrict__ k, uint16_t* __restrict__ v, long long k_t, long long k_h,
                      long long v_t, long long v_h, int32_t* __restrict__ positions, int rows) {
  constexpr int kPer = D / 8, kRowsAtOnce = 32 / kPer, kPitch = D + 16;
  __shared__ __align__(16) uint8_t s_blk[kReadWarps][32 * kPitch];   // 16 rows of bytes, or of halves
  __shared__ int s_count[kCountHere];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // K or V of one (sequence, KV head)
  const int unit = blockIdx.x / spans >> 1, kv = blockIdx.x / spans & 1, h = unit % s.Hkv, b = unit / s.Hkv;
  const int ch = lane % kPer, g = lane >> 2, t = lane & 3;
  pdl_wait();
  const size_t lb = lb_index(s, layer, b), u = unit_index(s, layer, b, h);
  int row0;
  if (counted) {
    row0 = cu[b];
  } else {
    for (int i = warp; i < s.B; i += kReadWarps) {
      const size_t at = lb_index(s, layer, i);
      int n = 0;
      for (int j = lane; j < s.WR; j += 32) n += d.pos[at * s.S + s.cap + j] >= 0;
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) s_count[i] = n + d.n8[at];
    }
    __syncthreads();
    row0 = 0;
    for (int i = 0; i < b; ++i) row0 += s_count[i];
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      int sum = 0;
      for (int i = 0; i < s.B; ++i) {
        cu[i] = sum;
        sum += s_count[i];
      }
      cu[s.B] = sum;
    }
  }
  const int n8 = d.n8[lb], nb8 = (n8 + 15) / 16, nb = nb8 + s.WR / 16;
  const int32_t* pos = d.pos + lb * s.S;
  const bool first = h == 0 && kv == 0;                // writes the positions
  uint8_t* blk = s_blk[warp];
  uint16_t* out = (kv ? v + h * v_h : k + h * k_h) + ch * 8;
  const long long ot = kv ? v_t : k_t;
  const int i0 = ((blockIdx.x % spans) * kReadWarps + warp) * per_warp, i1 = min(i0 + per_warp, nb);

  // ---- INT8 blocks, the next one in flight
  if (i0 < nb8) {
    float scale[8];
    const float4* sc = reinterpret_cast<const float4*>((kv ? d.sV : d.sK) + u * D + ch * 8);
    const float4 s0 = sc[0], s1 = sc[1];
    scale[0] = s0.x; scale[1] = s0.y; scale[2] = s0.z; scale[3] = s0.w;
    scale[4] = s1.x; scale[5] = s1.y; scale[6] = s1.z; scale[7] = s1.w;
    const uint8_t* src = (kv ? d.v8 : d.k8) + (u * (s.cstride / 16) + i0) * 16 * D + lane * 16;
    uint4 next[D / 32];
#pragma unroll
    for (int r = 0; r < D / 32; ++r) next[r] = *reinterpret_cast<const uint4*>(src + r * 512);
    for (int i = i0; i < min(i1, nb8); ++i) {
      uint4 x[D / 32];
#pragma unroll
      for (int r = 0; r < D / 32; ++r) x[r] = next[r];
      src += 16 * D;
      if (i + 1 < min(i1, nb8)) {
#pragma unroll
        for (int r = 0; r < D / 32; ++r) next[r] = *reinterpret_cast<const uint4*>(src + r * 512);
      }
      if (kv) {                                        // v8_offset: channel 8 (4 r + j) + g, four tokens
#pragma unroll
        for (int r = 0; r < D / 32; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w = (&x[r].x)[j];
            uint8_t* o = blk + (4 * r + j) * 8 + g;
            o[(2 * t) * kPitch] = (uint8_t)w;
            o[(2 * t + 1) * kPitch] = (uint8_t)(w >> 8);
            o[(2 * t + 8) * kPitch] = (uint8_t)(w >> 16);
            o[(2 * t + 9) * kPitch] = (uint8_t)(w >> 24);
          }
      } else {                                         // k8_offset: token 8 nt + g, two channel pairs
#pragma unroll
        for (int r = 0; r < D / 32; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w = (&x[r].x)[j];
            const int nt = r / (D / 64), kk = (r % (D / 64)) * 4 + j;
            uint8_t* o = blk + (8 * nt + g) * kPitch + 16 * kk + 2 * t;
            *reinterpret_cast<uint16_t*>(o) = (uint16_t)w;
            *reinterpret_cast<uint16_t*>(o + 8) = (uint16_t)(w >> 16);
          }
      }
      __syncwarp();
      const int tokens = min(16, n8 - i * 16), row = row0 + i * 16;   // entries of the block and their first row
      if (row + tokens > rows && lane == 0) atomicOr(d.status, kStatusCapacity);
      const int fit = min(tokens, rows - row);
      if (first && lane < fit) positions[row + lane] = pos[i * 16 + lane];
#pragma unroll
      for (int r = 0; r < 16; r += kRowsAtOnce) {
        const int tau = r + lane / kPer;
        const uint4 y = dequantise(*reinterpret_cast<const uint2*>(blk + tau * kPitch + ch * 8), scale, BF16);
        if (tau < fit) *reinterpret_cast<uint4*>(out + (row + tau) * ot) = y;
      }
      __syncwarp();
    }
  }

  // ---- blocks of the window
  for (int i = max(i0, nb8); i < i1; ++i) {
    // output row of slot `lane` (lanes 0-15): behind the ring's older entries; -1: nothing there
    const int32_t* rp = pos + s.cap;
    const int p = lane < 16 ? rp[(i - nb8) * 16 + lane] : -1;
    int row = -1, older[16] = {};
    for (int j = lane; j < s.WR; j += 32) {
      const int x = rp[j];
#pragma unroll
      for (int q = 0; q < 16; ++q) older[q] += x >= 0 && x < rp[(i - nb8) * 16 + q];
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int n = __reduce_add_sync(0xffffffffu, older[q]);
      if (lane == q && p >= 0) row = row0 + n8 + n;
    }
    if (row >= rows) {
      atomicOr(d.status, kStatusCapacity);
      row = -1;
    }
    if (first && row >= 0) positions[row] = p;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(kv ? d.v16 : d.k16) + (u * (s.WR / 16) + (i - nb8)) * 32 * D;
    uint16_t* half = reinterpret_cast<uint16_t*>(blk);
#pragma unroll
    for (int r = 0; r < D / 16; ++r) {
      const uint4 y = *reinterpret_cast<const uint4*>(src + r * 512 + lane * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = (&y.x)[j];
        if (kv) {                                      // v16_offset: channel 8 (2 r + j / 2) + g, two tokens
          const int c = 8 * (2 * r + (j >> 1)) + g, tau = 8 * (j & 1) + 2 * t;
          half[tau * kPitch + c] = (uint16_t)w;
          half[(tau + 1) * kPitch + c] = (uint16_t)(w >> 16);
        } else {                                       // k16_offset: token 8 nt + g, a channel pair
          const int nt = r / (D / 32), kk = 2 * (r % (D / 32)) + (j >> 1);
          *reinterpret_cast<uint32_t*>(half + (8 * nt + g) * kPitch + 16 * kk + 8 * (j & 1) + 2 * t) = w;
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 16; r += kRowsAtOnce) {
      const int tau = r + lane / kPer;
      const int to = __shfl_sync(0xffffffffu, row, tau);
      uint4 y = *reinterpret_cast<const uint4*>(blk + (tau * kPitch + ch * 8) * 2);
      if (BF16) {
        uint32_t* w = &y.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
          const __nv_bfloat162 q = __floats2bfloat162_rn(f.x, f.y);
          w[j] = *reinterpret_cast<const uint32_t*>(&q);
        }
      }
      if (to >= 0) *reinterpret_cast<uint4*>(out + to * ot) = y;
    }
    __syncwarp();
  }
}

}  // namespace

int launch_prefill_reset(const Shape& s, const Dev& d, const int32_t* len, cudaStream_t st) {
  LengthChunk c;
  c.row0 = 0;
  for (c.first = 0; c.first < s.B; c.first += LengthChunk::kMax) {
    c.count = std::min(LengthChunk::kMax, s.B - c.first);
    for (int i = 0; i < c.count; ++i) c.len[i] = len[c.first + i];
    if (launch_pdl(prefill_reset_kernel, dim3(1), dim3(256), 0, st, s, d, c) != cudaSuccess) return -1;
    for (int i = 0; i < c.count; ++i) c.row0 += c.len[i];
  }
  return 0;
}

template <int D, bool BF16>
static int launch_write(const Shape& s, const Dev& d, int layer, const void* k, const void* v, const int64_t* ks,
                        const int64_t* vs, int max_len, cudaStream_t st) {
  static int done[kMaxDevices] = {};
  constexpr int smem = kWriteWarps * (D / 16) * kChunk;
  if (ensure_smem(write_layer_kernel<D, BF16>, smem, done) != cudaSuccess) return -1;
  // CTAs per (sequence, head, K or V): enough to fill the GPU, as long as
  // each still has 64 tokens
  const long long units = 2LL * s.B * s.Hkv;
  int ctas = 1;
  while (ctas < kMaxCtas && units * ctas < 4LL * 152 && max_len / (2 * ctas) >= 64) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * ctas));
  cfg.blockDim = dim3(kWriteWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, write_layer_kernel<D, BF16>, s, d, layer, static_cast<const uint16_t*>(k),
                            static_cast<const uint16_t*>(v), (long long)ks[0], (long long)ks[1], (long long)vs[0],
                            (long long)vs[1]) == cudaSuccess
             ? 0
             : -1;
}

int launch_write_layer(const Shape& s, const Dev& d, int layer, bool bf16, const void* k, const void* v,
                       const int64_t* k_stride, const int64_t* v_stride, int max_len, cudaStream_t st) {
  auto fn = s.D == 128 ? (bf16 ? launch_write<128, true> : launch_write<128, false>)
                       : (bf16 ? launch_write<64, true> : launch_write<64, false>);
  return fn(s, d, layer, k, v, k_stride, v_stride, max_len, st);
}

int launch_read_layer(const Shape& s, const Dev& d, int layer, bool bf16, void* k, void* v, const int64_t* ks,
                      const int64_t* vs, int32_t* positions, int32_t* cu, int rows, long long n8_bound,
                      cudaStream_t st) {
  const bool counted = s.B > kCountHere;
  if (counted) count_entries_kernel<<<1, 1024, 0, st>>>(s, d, layer, cu);
  // one block per warp until the GPU is full, then up to eight
  const long long blocks = (n8_bound + 15) / 16 + s.WR / 16, units = 2LL * s.B * s.Hkv;
  const long long per_warp = std::min(8LL, std::max(1LL, blocks * units / (152LL * 8 * kReadWarps)));
  const int spans = (int)((blocks + kReadWarps * per_warp - 1) / (kReadWarps * per_warp));
  const dim3 grid((unsigned)(spans * units));
  auto kernel = s.D == 128 ? (bf16 ? read_layer_kernel<128, true> : read_layer_kernel<128, false>)
                           : (bf16 ? read_layer_kernel<64, true> : read_layer_kernel<64, false>);
  return launch_pdl(kernel, grid, dim3(kReadWarps * 32), 0, st, s, d, layer, spans, (int)per_warp, (int)counted, cu,
                    static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), (long long)ks[0], (long long)ks[1],
                    (long long)vs[0], (long long)vs[1], positions, rows) == cudaSuccess
             ? 0
             : -1;
}

}  // namespace confkv

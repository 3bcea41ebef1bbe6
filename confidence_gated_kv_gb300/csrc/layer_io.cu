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
// Both move a few bytes per value and are bound by HBM.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>

#include "../../include/confkv.h"
#include "confkv_internal.cuh"

namespace cg = cooperative_groups;

namespace confkv {
namespace {

constexpr int kChunk = 528;          // shared-memory pitch of a 512-byte piece of an interleaved block
constexpr int kWriteWarps = 16;
constexpr int kReadWarps = 8;
constexpr int kReadBlocks = 2;       // 16-token blocks per warp of the read kernel

// ------------------------------------------------------------------ reset

__global__ void prefill_reset_kernel(Shape s, Dev d, LengthChunk c) {
  for (int i = threadIdx.x; i < c.count; i += blockDim.x) {
    d.T0[c.first + i] = c.len[i];
    d.conf_done[c.first + i] = 0;
    d.conf_ready[c.first + i] = 0;
    for (int l = 0; l < s.L; ++l) d.arrive[(size_t)l * s.B + c.first + i] = 0;
  }
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

// 8 source values as fp16 pairs.
__device__ __forceinline__ uint4 load_half8(const uint16_t* p, bool bf16) {
  uint4 u = *reinterpret_cast<const uint4*>(p);
  if (bf16) {
    uint32_t* w = &u.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return u;
}

// clamp(rint(x / s), -127, 127) with the IEEE quotient.  x * (1 / s) is
// within 2 ulp of it (below 2^-15 up to 127), so the integers agree unless
// the product lies that close to a half; only then is the quotient computed.
__device__ __forceinline__ int quantise(float x, float s, float inv) {
  float q = x * inv;
  if (fabsf(fabsf(q - truncf(q)) - 0.5f) < 6.1e-5f) q = __fdiv_rn(x, s);
  return (int)fminf(fmaxf(rintf(q), -127.f), 127.f);
}

template <int D>
__global__ void __launch_bounds__(kWriteWarps * 32, 2)
    write_layer_kernel(Shape s, Dev d, int layer, int bf16, const uint16_t* __restrict__ k,
                       const uint16_t* __restrict__ v, long long k_t, long long k_h, long long v_t, long long v_h) {
  constexpr int kPer = D / 8;                          // threads per row
  constexpr int kRowsAtOnce = kWriteWarps * 32 / kPer;
  extern __shared__ __align__(16) uint8_t smem[];      // an interleaved block per warp
  __shared__ uint32_t s_abs[D / 2];                    // absmax of this CTA's tokens, fp16 pairs
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int unit = blockIdx.x / ctas;                  // (sequence, KV head, K or V)
  const bool is_v = unit & 1;
  const int h = (unit >> 1) % s.Hkv, b = (unit >> 1) / s.Hkv;
  const int T0 = d.T0[b], n8 = max(0, T0 - s.W);
  const uint16_t* src = is_v ? v : k;
  const long long ts = is_v ? v_t : k_t;
  src += d.row0[b] * ts + h * (is_v ? v_h : k_h);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ch = threadIdx.x % kPer;                   // 8-channel chunk of this thread
  const size_t lb = lb_index(s, layer, b), u = unit_index(s, layer, b, h);

  for (int i = threadIdx.x; i < D / 2; i += blockDim.x) s_abs[i] = 0;
  __syncthreads();
  // ---- absmax over the CTA's share of the tokens
  __half2 top[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) top[i] = __float2half2_rn(0.f);
  {
    const int per = (T0 + ctas - 1) / ctas, t1 = min(T0, (rank + 1) * per);
    int t = rank * per + threadIdx.x / kPer;
    for (; t + 3 * kRowsAtOnce < t1; t += 4 * kRowsAtOnce) {
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = load_half8(src + (t + i * kRowsAtOnce) * ts + ch * 8, bf16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2* w = reinterpret_cast<const __half2*>(&x[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) top[j] = __hmax2(top[j], __habs2(w[j]));
      }
    }
    for (; t < t1; t += kRowsAtOnce) {
      const uint4 x = load_half8(src + t * ts + ch * 8, bf16);
      const __half2* w = reinterpret_cast<const __half2*>(&x);
#pragma unroll
      for (int j = 0; j < 4; ++j) top[j] = __hmax2(top[j], __habs2(w[j]));
    }
  }
#pragma unroll
  for (int o = kPer; o < 32; o <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) top[j] = __hmax2(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
  // fp16 absolute values order like their bits, so each half can be merged
  // as an integer: one lane per chunk and warp, one 32-bit word per pair
  __half2* stage = reinterpret_cast<__half2*>(smem);   // [warp][D / 2]
  if (lane < kPer)
#pragma unroll
    for (int j = 0; j < 4; ++j) stage[warp * (D / 2) + ch * 4 + j] = top[j];
  __syncthreads();
  for (int i = threadIdx.x; i < D / 2; i += blockDim.x) {
    __half2 m = stage[i];
    for (int w = 1; w < kWriteWarps; ++w) m = __hmax2(m, stage[w * (D / 2) + i]);
    s_abs[i] = *reinterpret_cast<const uint32_t*>(&m);
  }
  cluster.sync();
  float scale[8], inv[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    __half2 m = __float2half2_rn(0.f);
    for (int r = 0; r < ctas; ++r) {
      const uint32_t w = *cluster.map_shared_rank(&s_abs[ch * 4 + j], r);
      m = __hmax2(m, *reinterpret_cast<const __half2*>(&w));
    }
    const float2 f = __half22float2(m);
    scale[2 * j] = f.x > 0.f ? __fdiv_rn(f.x, 127.f) : 1.f;
    scale[2 * j + 1] = f.y > 0.f ? __fdiv_rn(f.y, 127.f) : 1.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) inv[i] = __fdiv_rn(1.f, scale[i]);
  if (rank == 0 && threadIdx.x < kPer) {
    float* dst = (is_v ? d.sV : d.sK) + u * D + ch * 8;
    *reinterpret_cast<float4*>(dst) = make_float4(scale[0], scale[1], scale[2], scale[3]);
    *reinterpret_cast<float4*>(dst + 4) = make_float4(scale[4], scale[5], scale[6], scale[7]);
  }
  cluster.sync();                                      // no CTA leaves while another reads its maxima

  // ---- blocks: ceil(n8 / 16) of codes, then the ring
  uint8_t* blk = smem + warp * (D / 16) * kChunk;
  constexpr int kRowsPerWarp = 32 / kPer, kIter = 16 / kRowsPerWarp;
  const int nb8 = (n8 + 15) / 16, nb = nb8 + s.WR / 16;
  const int first_ring = n8;
  const int c0 = is_v ? (ch >> 2) * kChunk + (ch & 3) * 4
                      : ((ch >> 1) >> 2) * kChunk + ((ch >> 1) & 3) * 4 + (ch & 1) * 2;
  for (int i = rank * kWriteWarps + warp; i < nb; i += ctas * kWriteWarps) {
    const bool ring = i >= nb8;
    uint4 x[kIter];
    int tau[kIter];
    bool there[kIter];
#pragma unroll
    for (int r = 0; r < kIter; ++r) {
      tau[r] = r * kRowsPerWarp + lane / kPer;
      int p;
      if (ring) {                                      // the newest position that falls on the slot
        const int slot = (i - nb8) * 16 + tau[r];
        p = T0 - 1 - ((T0 - 1 - slot) % s.WR + s.WR) % s.WR;
        there[r] = p >= first_ring;
      } else {
        p = i * 16 + tau[r];
        there[r] = p < n8;
      }
      x[r] = there[r] ? load_half8(src + p * ts + ch * 8, bf16) : make_uint4(0, 0, 0, 0);
    }
    if (!ring) {
#pragma unroll
      for (int r = 0; r < kIter; ++r) {
        const __half2* w = reinterpret_cast<const __half2*>(&x[r]);
        int code[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(w[j]);
          code[2 * j] = there[r] ? quantise(f.x, scale[2 * j], inv[2 * j]) + kCodeBias : kCodeBias;
          code[2 * j + 1] = there[r] ? quantise(f.y, scale[2 * j + 1], inv[2 * j + 1]) + kCodeBias : kCodeBias;
        }
        if (is_v) {                                    // v8_offset
          uint8_t* o = blk + c0 + ((tau[r] & 7) >> 1) * 16 + (((tau[r] >> 3) << 1) | (tau[r] & 1));
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j * 64] = (uint8_t)code[j];
        } else {                                       // k8_offset
          uint8_t* o = blk + c0 + (tau[r] >> 3) * (D / 64) * kChunk + (tau[r] & 7) * 64;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint16_t*>(o + j * 16) = (uint16_t)(code[2 * j] | code[2 * j + 1] << 8);
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < kIter; ++r) {
        const uint16_t* w = reinterpret_cast<const uint16_t*>(&x[r]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int o = is_v ? v16_offset(D, tau[r], ch * 8 + j) : k16_offset(D, tau[r], ch * 8 + j);
          *reinterpret_cast<uint16_t*>(blk + (o >> 9) * kChunk + (o & 511)) = w[j];
        }
      }
    }
    __syncwarp();
    uint8_t* dst = ring ? reinterpret_cast<uint8_t*>(is_v ? d.v16 : d.k16) + (u * (s.WR / 16) + (i - nb8)) * 32 * D
                        : (is_v ? d.v8 : d.k8) + (u * (s.cstride / 16) + i) * 16 * D;
    for (int r = 0; r < (ring ? D / 16 : D / 32); ++r)
      *reinterpret_cast<uint4*>(dst + r * 512 + lane * 16) = *reinterpret_cast<const uint4*>(blk + r * kChunk + lane * 16);
    __syncwarp();
  }
  // ---- positions and EMA of the layer's slots, by the K of KV head 0
  if (h == 0 && !is_v) {
    for (int i = rank * blockDim.x + threadIdx.x; i < s.S; i += ctas * blockDim.x) {
      int p = -1;
      if (i < n8) {
        p = i;
      } else if (i >= s.cap && T0 > 0) {
        const int slot = i - s.cap, back = ((T0 - 1 - slot) % s.WR + s.WR) % s.WR;
        p = T0 - 1 - back >= first_ring ? T0 - 1 - back : -1;
      }
      d.pos[lb * s.S + i] = p;
      d.ema[lb * s.S + i] = 0.f;
    }
    if (rank == 0 && threadIdx.x == 0) d.n8[lb] = n8;
  }
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

template <int D>
__global__ void __launch_bounds__(kReadWarps * 32)
    read_layer_kernel(Shape s, Dev d, int layer, int bf16, int spans, const int32_t* __restrict__ cu,
                      uint16_t* __restrict__ k, uint16_t* __restrict__ v, long long k_t, long long k_h,
                      long long v_t, long long v_h, int32_t* __restrict__ positions, int rows) {
  constexpr int kPer = D / 8, kRowsAtOnce = 32 / kPer, kPitch = D + 16;
  __shared__ __align__(16) uint8_t s_blk[kReadWarps][32 * kPitch];   // 16 rows of bytes, or of halves
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / spans, h = unit % s.Hkv, b = unit / s.Hkv;
  const int ch = lane % kPer;
  pdl_wait();
  const size_t lb = lb_index(s, layer, b), u = unit_index(s, layer, b, h);
  const int n8 = d.n8[lb], nb8 = (n8 + 15) / 16, nb = nb8 + s.WR / 16;
  const int row0 = cu[b];
  const int32_t* pos = d.pos + lb * s.S;
  uint8_t* blk = s_blk[warp];
  const int i0 = ((blockIdx.x % spans) * kReadWarps + warp) * kReadBlocks;
  for (int i = i0; i < min(i0 + kReadBlocks, nb); ++i) {
    const bool ring = i >= nb8;
    // output row of slot `lane` (lanes 0-15); -1: nothing there
    int row = -1, p = -1;
    if (!ring) {
      const int slot = i * 16 + lane;
      if (lane < 16 && slot < n8) {
        row = row0 + slot;
        p = pos[slot];
      }
    } else {
      const int32_t* rp = pos + s.cap;
      p = lane < 16 ? rp[(i - nb8) * 16 + lane] : -1;
      int older = 0;
      for (int j0 = 0; j0 < s.WR; j0 += 32) {
        const int q = j0 + lane < s.WR ? rp[j0 + lane] : -1;
        for (int j = 0; j < 32; ++j) {
          const int x = __shfl_sync(0xffffffffu, q, j);
          older += x >= 0 && x < p;
        }
      }
      if (p >= 0) row = row0 + n8 + older;
    }
    if (row >= rows) {
      atomicOr(d.status, kStatusCapacity);
      row = -1;
    }
    if (h == 0 && row >= 0) positions[row] = p;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float scale[8];
      if (!ring) {
        const uint8_t* src = (kv ? d.v8 : d.k8) + (u * (s.cstride / 16) + i) * 16 * D;
        const float4* sc = reinterpret_cast<const float4*>((kv ? d.sV : d.sK) + u * D + ch * 8);
        const float4 s0 = sc[0], s1 = sc[1];
        scale[0] = s0.x; scale[1] = s0.y; scale[2] = s0.z; scale[3] = s0.w;
        scale[4] = s1.x; scale[5] = s1.y; scale[6] = s1.z; scale[7] = s1.w;
        const int g = lane >> 2, t = lane & 3;
        uint4 x[D / 32];
#pragma unroll
        for (int r = 0; r < D / 32; ++r) x[r] = *reinterpret_cast<const uint4*>(src + r * 512 + lane * 16);
#pragma unroll
        for (int r = 0; r < D / 32; ++r) {
          const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (kv) {                                  // v8_offset: channel 8 (4 r + j) + g, four tokens
              uint8_t* o = blk + (4 * r + j) * 8 + g;
              o[(2 * t) * kPitch] = (uint8_t)w[j];
              o[(2 * t + 1) * kPitch] = (uint8_t)(w[j] >> 8);
              o[(2 * t + 8) * kPitch] = (uint8_t)(w[j] >> 16);
              o[(2 * t + 9) * kPitch] = (uint8_t)(w[j] >> 24);
            } else {                                   // k8_offset: token 8 nt + g, two channel pairs
              const int nt = r / (D / 64), kk = (r % (D / 64)) * 4 + j;
              uint8_t* o = blk + (8 * nt + g) * kPitch + 16 * kk + 2 * t;
              *reinterpret_cast<uint16_t*>(o) = (uint16_t)w[j];
              *reinterpret_cast<uint16_t*>(o + 8) = (uint16_t)(w[j] >> 16);
            }
          }
        }
      } else {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(kv ? d.v16 : d.k16) +
                             (u * (s.WR / 16) + (i - nb8)) * 32 * D;
        for (int e = lane; e < 16 * D; e += 32) {
          const int tau = e / D, c = e % D;
          const int o = kv ? v16_offset(D, tau, c) : k16_offset(D, tau, c);
          reinterpret_cast<uint16_t*>(blk)[tau * kPitch + c] = *reinterpret_cast<const uint16_t*>(src + o);
        }
      }
      __syncwarp();
      uint16_t* out = (kv ? v : k) + h * (kv ? v_h : k_h) + ch * 8;
      const long long ot = kv ? v_t : k_t;
#pragma unroll
      for (int r = 0; r < 16; r += kRowsAtOnce) {
        const int tau = r + lane / kPer;
        const int to = __shfl_sync(0xffffffffu, row, tau);
        if (to < 0) continue;
        uint4 y;
        if (!ring) {
          y = dequantise(*reinterpret_cast<const uint2*>(blk + tau * kPitch + ch * 8), scale, bf16);
        } else {
          y = *reinterpret_cast<const uint4*>(blk + (tau * kPitch + ch * 8) * 2);
          if (bf16) {
            uint32_t* w = &y.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
              const __nv_bfloat162 q = __floats2bfloat162_rn(f.x, f.y);
              w[j] = *reinterpret_cast<const uint32_t*>(&q);
            }
          }
        }
        *reinterpret_cast<uint4*>(out + to * ot) = y;
      }
      __syncwarp();
    }
  }
}

}  // namespace

int launch_prefill_reset(const Shape& s, const Dev& d, const int32_t* len, cudaStream_t st) {
  LengthChunk c;
  c.row0 = 0;
  for (c.first = 0; c.first < s.B; c.first += LengthChunk::kMax) {
    c.count = std::min(LengthChunk::kMax, s.B - c.first);
    for (int i = 0; i < c.count; ++i) c.len[i] = len[c.first + i];
    prefill_reset_kernel<<<1, 256, 0, st>>>(s, d, c);
    for (int i = 0; i < c.count; ++i) c.row0 += c.len[i];
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <int D>
static int launch_write(const Shape& s, const Dev& d, int layer, bool bf16, const void* k, const void* v,
                        const int64_t* ks, const int64_t* vs, int max_len, cudaStream_t st) {
  static int done[kMaxDevices] = {};
  constexpr int smem = kWriteWarps * (D / 16) * kChunk;
  if (ensure_smem(write_layer_kernel<D>, smem, done) != cudaSuccess) return -1;
  // CTAs per (sequence, head, K or V): enough to fill the GPU twice, as long
  // as each still has 64 tokens
  const long long units = 2LL * s.B * s.Hkv;
  int ctas = 1;
  while (ctas < 8 && units * ctas < 4LL * 152 && max_len / (2 * ctas) >= 64) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * ctas));
  cfg.blockDim = dim3(kWriteWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, write_layer_kernel<D>, s, d, layer, (int)bf16, static_cast<const uint16_t*>(k),
                            static_cast<const uint16_t*>(v), (long long)ks[0], (long long)ks[1], (long long)vs[0],
                            (long long)vs[1]) == cudaSuccess ? 0 : -1;
}

int launch_write_layer(const Shape& s, const Dev& d, int layer, bool bf16, const void* k, const void* v,
                       const int64_t* k_stride, const int64_t* v_stride, int max_len, cudaStream_t st) {
  return s.D == 128 ? launch_write<128>(s, d, layer, bf16, k, v, k_stride, v_stride, max_len, st)
                    : launch_write<64>(s, d, layer, bf16, k, v, k_stride, v_stride, max_len, st);
}

int launch_read_layer(const Shape& s, const Dev& d, int layer, bool bf16, void* k, void* v, const int64_t* ks,
                      const int64_t* vs, int32_t* positions, int32_t* cu, int rows, long long n8_bound,
                      cudaStream_t st) {
  count_entries_kernel<<<1, 1024, 0, st>>>(s, d, layer, cu);
  const long long blocks = (n8_bound + 15) / 16 + s.WR / 16;
  const int spans = (int)((blocks + kReadWarps * kReadBlocks - 1) / (kReadWarps * kReadBlocks));
  const dim3 grid((unsigned)((long long)spans * s.B * s.Hkv));
  auto kernel = s.D == 128 ? read_layer_kernel<128> : read_layer_kernel<64>;
  return launch_pdl(kernel, grid, dim3(kReadWarps * 32), 0, st, s, d, layer, (int)bf16, spans, (const int32_t*)cu,
                    static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), (long long)ks[0], (long long)ks[1],
                    (long long)vs[0], (long long)vs[1], positions, rows) == cudaSuccess
             ? 0
             : -1;
}

}  // namespace confkv

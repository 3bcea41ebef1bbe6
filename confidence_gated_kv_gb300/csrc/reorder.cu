// Exchange of cache states between the beams of a group, in place.
//
// A state is the same bytes at the same offsets for every sequence, so a
// thread that owns an offset can take the values of all sequences that are a
// parent into registers before it writes any: no order between threads, no
// copy aside, whatever the parents form (chains, cycles, one for all).  Each
// parent is read once and each sequence that moves written once.
//
// Lengths are exchanged by a second, small launch: the first one reads them.
//
// What bounds it: HBM, reads and writes mixed.  With few parents a thread takes
// several columns at once, so that eight loads are in flight.  Two groups of
// eight beams with 8192 entries, four layers: 207 us for 1.06 GB (0.77 of the
// copy rate).  More than eight beams wait in shared memory, one batch of copies at
// a time: two groups of 16 with 2049 entries 168 to 258 us (0.71 to 0.66, by how
// many move), one of 64 in two layers 422 to 764 (0.30 to 0.23).  Lengths by the last CTA of a group instead of a launch of their
// own took 4 us more on the device and 4 less on the host.
#include <cuda_runtime.h>
#include <algorithm>

#include "../../include/confkv.h"
#include "confkv_internal.cuh"

namespace confkv {
namespace {

constexpr int kMax = CONFKV_BEAM_MAX;
constexpr int kThreads = 256;

// 16-byte columns of a layer's regions, in chunks of one CTA pass.
struct Plan {
  int columns;                           // per chunk: kColumns a thread
  int blocks;                            // 16-token INT8 blocks that the bound allows
  unsigned codes, ring, scales, meta8, metaR;    // chunks of one of 2 Hkv planes, and of one of two arrays
  unsigned per_layer, total;
};
constexpr int kColumns = 4;

struct Moves {
  int count;                             // parents that some other sequence takes over
  int from[kMax];                        // sequence
  unsigned long long to[kMax];           // sequences of the group
};

__device__ __forceinline__ void find_moves(Moves& m, int* parent, const int32_t* parents, int beams, int b0) {
  if (threadIdx.x < kMax) {
    const int p = threadIdx.x < beams ? parents[b0 + threadIdx.x] : -1;
    parent[threadIdx.x] = p >= 0 && p < beams ? p : (int)threadIdx.x;
  }
  if (threadIdx.x == 0) m.count = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    for (int half = 0; half < 2; ++half) {
      const int k = half * 32 + threadIdx.x;
      unsigned long long to = 0;
      for (int i = 0; i < beams; ++i)
        if (parent[i] == k && i != k) to |= 1ull << i;
      const unsigned some = __ballot_sync(0xffffffffu, to != 0);
      const int at = m.count + __popc(some & ((1u << threadIdx.x) - 1u));
      if (to) {
        m.from[at] = b0 + k;
        m.to[at] = to;
      }
      __syncwarp();
      if (threadIdx.x == 0) m.count += __popc(some);
      __syncwarp();
    }
  }
  __syncthreads();
}

// What a chunk covers: column c of sequence b is at base + b stride + 16 c.
struct Region {
  char* base;
  long long stride;
  int columns, per_block;                // per_block: columns of an INT8 block (0: the region is whole)
  int first;                             // first column of the chunk
  const int32_t* n8;                     // of the layer's sequences
};

__device__ __forceinline__ bool there(const Region& r, int from, int col) {
  return col < r.columns && (r.per_block == 0 || col / r.per_block * 16 < r.n8[from]);
}

// Up to P parents, 8 / P columns of a thread at a time.
template <int P>
__device__ __forceinline__ void move_columns(const Region& r, const Moves& m, int b0) {
  constexpr int U = P >= 8 ? 1 : 8 / P < kColumns ? 8 / P : kColumns;
  const int count = m.count;
#pragma unroll
  for (int u0 = 0; u0 < kColumns; u0 += U) {
    uint4 x[U][P];
    bool some[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int col = r.first + (u0 + u) * kThreads + threadIdx.x;
        some[u][j] = j < count && there(r, m.from[j], col);
        if (some[u][j]) x[u][j] = *reinterpret_cast<const uint4*>(r.base + m.from[j] * r.stride + (long long)col * 16);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < P; ++j)
        if (some[u][j]) {
          const int col = r.first + (u0 + u) * kThreads + threadIdx.x;
          for (unsigned long long to = m.to[j]; to; to &= to - 1)
            *reinterpret_cast<uint4*>(r.base + (b0 + __ffsll((long long)to) - 1) * r.stride + (long long)col * 16) = x[u][j];
        }
  }
}

// WIDE: more parents than registers hold; they wait in shared memory.
template <bool WIDE>
__global__ void __launch_bounds__(kThreads) reorder_kernel(Shape s, Dev d, const int32_t* __restrict__ parents,
                                                           int beams, const __grid_constant__ Plan plan) {
  extern __shared__ uint4 s_wait[];                      // [parent][thread]
  __shared__ Moves m;
  __shared__ int s_parent[kMax];
  const int b0 = blockIdx.y * beams;
  pdl_wait();
  find_moves(m, s_parent, parents, beams, b0);
  const int count = m.count;
  if (count == 0) return;
  for (unsigned chunk = blockIdx.x; chunk < plan.total; chunk += gridDim.x) {
    const int l = (int)(chunk / plan.per_layer);
    unsigned i = chunk - l * plan.per_layer;
    const size_t lb = lb_index(s, l, 0), u = unit_index(s, l, 0, 0);
    Region r;
    r.per_block = 0;
    r.n8 = d.n8 + lb;
    if (i < plan.codes * 2 * s.Hkv) {
      const unsigned plane = i / plan.codes;
      i -= plane * plan.codes;
      r.base = reinterpret_cast<char*>(plane & 1 ? d.v8 : d.k8) + (u + (plane >> 1)) * s.cstride * s.D;
      r.stride = (long long)s.Hkv * s.cstride * s.D;
      r.per_block = s.D;
      r.columns = plan.blocks * s.D;
    } else if ((i -= plan.codes * 2 * s.Hkv) < plan.ring * 2) {
      const bool v = i >= plan.ring;
      i -= v ? plan.ring : 0;
      r.base = reinterpret_cast<char*>(v ? d.v16 : d.k16) + u * s.WR * s.D * 2;
      r.stride = (long long)s.Hkv * s.WR * s.D * 2;
      r.columns = (int)(r.stride / 16);
    } else if ((i -= plan.ring * 2) < plan.scales * 2) {
      const bool v = i >= plan.scales;
      i -= v ? plan.scales : 0;
      r.base = reinterpret_cast<char*>(v ? d.sV : d.sK) + u * s.D * 4;
      r.stride = (long long)s.Hkv * s.D * 4;
      r.columns = (int)(r.stride / 16);
    } else {
      i -= plan.scales * 2;
      const bool ema = i >= plan.meta8 + plan.metaR;
      i -= ema ? plan.meta8 + plan.metaR : 0;
      r.base = (ema ? reinterpret_cast<char*>(d.ema) : reinterpret_cast<char*>(d.pos)) + lb * s.S * 4;
      r.stride = (long long)s.S * 4;
      if (i < plan.meta8) {
        r.per_block = 4;
        r.columns = plan.blocks * 4;
      } else {
        i -= plan.meta8;
        r.base += (long long)s.cap * 4;
        r.columns = s.WR / 4;
      }
    }
    r.first = (int)(i * plan.columns);
    if (!WIDE) {
      if (count <= 2)
        move_columns<2>(r, m, b0);
      else if (count <= 4)
        move_columns<4>(r, m, b0);
      else
        move_columns<8>(r, m, b0);
    } else {
      for (int c = 0; c < kColumns; ++c) {
        const int col = r.first + c * (int)blockDim.x + threadIdx.x;
        for (int j = 0; j < count; ++j)
          if (there(r, m.from[j], col))
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(
                             (uint32_t)__cvta_generic_to_shared(s_wait + j * blockDim.x + threadIdx.x)),
                         "l"(r.base + m.from[j] * r.stride + (long long)col * 16)
                         : "memory");
        asm volatile("cp.async.wait_all;\n" ::: "memory");
        for (int j = 0; j < count; ++j)
          if (there(r, m.from[j], col)) {
            const uint4 x = s_wait[j * blockDim.x + threadIdx.x];
            for (unsigned long long to = m.to[j]; to; to &= to - 1)
              *reinterpret_cast<uint4*>(r.base + (b0 + __ffsll((long long)to) - 1) * r.stride + (long long)col * 16) = x;
          }
      }
    }
  }
}

// n8 of every (layer, sequence): a warp per (layer, group).
__global__ void __launch_bounds__(kThreads) reorder_counts_kernel(Shape s, Dev d, const int32_t* __restrict__ parents,
                                                                  int beams) {
  pdl_wait();
  const int groups = s.B / beams, lane = threadIdx.x & 31;
  const long long i = blockIdx.x * (long long)(kThreads / 32) + (threadIdx.x >> 5);
  if (i >= (long long)s.L * groups) return;
  const int b0 = (int)(i % groups) * beams;
  const size_t at = lb_index(s, (int)(i / groups), b0);
  int n[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int k = lane + 32 * e;
    if (k < beams) {
      const int p = parents[b0 + k];
      n[e] = d.n8[at + (p >= 0 && p < beams ? p : k)];
    }
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (lane + 32 * e < beams) d.n8[at + lane + 32 * e] = n[e];
}

}  // namespace

int launch_reorder(const Shape& s, const Dev& d, const int32_t* parents, int beams, long long n8_bound,
                   cudaStream_t st) {
  const bool wide = beams > 8;
  const int threads = wide ? 128 : kThreads;
  Plan p{};
  p.columns = threads * kColumns;
  p.blocks = (int)((n8_bound + 15) / 16);
  // columns of a region fit 31 bits, and so do the chunks of a layer
  const long long widest = std::max((long long)p.blocks * s.D, (long long)s.Hkv * s.WR * s.D / 8);
  if (widest >= (1LL << 31) - p.columns) return -1;
  auto chunks = [&](long long columns) { return (unsigned)((columns + p.columns - 1) / p.columns); };
  p.codes = chunks((long long)p.blocks * s.D);
  p.ring = chunks((long long)s.Hkv * s.WR * s.D / 8);
  p.scales = chunks((long long)s.Hkv * s.D / 4);
  p.meta8 = chunks((long long)p.blocks * 4);
  p.metaR = chunks(s.WR / 4);
  const long long per_layer = 2 * (s.Hkv * (long long)p.codes + p.ring + p.scales + p.meta8 + p.metaR);
  if (per_layer * s.L >= (1LL << 31)) return -1;
  p.per_layer = (unsigned)per_layer;
  p.total = (unsigned)(per_layer * s.L);
  const int groups = s.B / beams;
  if (groups > 65535) return -1;
  const long long want = std::max(1LL, 152LL * 8 / groups);
  const dim3 grid((unsigned)std::min<long long>(p.total, want), (unsigned)groups);
  cudaError_t e;
  if (wide) {
    static int done[kMaxDevices] = {};
    const int smem = beams * threads * 16;
    if (ensure_smem(reorder_kernel<true>, smem, done) != cudaSuccess) return -1;
    e = launch_pdl(reorder_kernel<true>, grid, dim3(threads), smem, st, s, d, parents, beams, p);
  } else {
    e = launch_pdl(reorder_kernel<false>, grid, dim3(threads), 0, st, s, d, parents, beams, p);
  }
  if (e != cudaSuccess) return -1;
  const long long warps = (long long)s.L * groups;
  const unsigned blocks = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
  return launch_pdl(reorder_counts_kernel, dim3(blocks), dim3(kThreads), 0, st, s, d, parents, beams) == cudaSuccess ? 0
                                                                                                                  : -1;
}

}  // namespace confkv

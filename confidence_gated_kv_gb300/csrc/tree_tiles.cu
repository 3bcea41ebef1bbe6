// Attention of drafted tokens over the cache, many rows: 128 score rows
// (draft, query head of the group) of a KV head per CTA, products on tcgen05.
//
// The stored blocks of 16 tokens are interleaved for mma.m16n8k16, so warps
// convert them on their way: bulk copies bring them in, a lane's words become
// fp16 (codes exactly) and go into K-major tiles of 64 keys (K: rows of keys;
// V transposed: rows of channels) without bank conflicts.
//
// Roles of a CTA's 24 warps: two softmax warpgroups (a thread per row) that
// take alternate key tiles of the same rows, each with scores and an output of
// its own in tensor memory; eight warps that convert a block of K or of V of
// each tile; a warp per softmax warpgroup and kind of product that issues it;
// one for the copies, three for the drafts' paths.
// Queries stay in tensor memory: for INT8 keys in two fp16 parts (q sK to
// 2^-22, two products), for fp16 keys exact in one.  Weights go through shared
// memory, so that the scores of a warpgroup's next tile are computed while it
// is at the weights of this one.  The parts of the two warpgroups, and of the
// CTAs of a cluster that share the keys, are joined at the end.
//
// Loops are unrolled only as far as loads need it: a first version of 179 KB
// of code, with the loads of three tiles in registers, spent most of its time
// on instruction fetches (every step of every role took some 600 cycles).
//
// What bounds it: the chain of a softmax warpgroup's tile (scores, softmax,
// product, about 2800 cycles, two of them interleaved: 0.75 us per tile of 64
// keys and CTA) and 17 to 20 us around it, most of them first fetches of
// instructions (queries, the first tile, the change to fp16 keys, the join).
// 64 drafts on four sequences of 8192, 40 heads on 8: 105 us, the tensor pipe
// a third active; the kernel of few rows takes 248.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstddef>

#include "../../include/confkv.h"
#include "confkv_internal.cuh"
#include "fp32_pair.cuh"
#include "tree.cuh"

namespace cg = cooperative_groups;

namespace confkv {
namespace {

using namespace tree;

constexpr int kRows = 128, kKeys = 64;
constexpr int kChange = 7;               // tiles that fp16 keys (and the change to them) take as long as, more than their own
constexpr int kThreads = 768;
constexpr int kConverters = 4;           // warps 8 .. 11 for K and 12 .. 15 for V: a 16-token block of the tile each
// Registers a thread: at launch, and of the roles (two softmax warpgroups, the
// converter warpgroups, the rest), whose sum is the launch's.
constexpr int kRegs = 80, kSoftmaxRegs = 128, kConverterRegs = 64, kIssueRegs = 48;
static_assert(2 * kSoftmaxRegs + 2 * kConverterRegs + 2 * kIssueRegs == 6 * kRegs, "no more than the launch has");

template <int D>
struct Tile {
  static constexpr int kBytes = kKeys * D * 2;           // a converted K or V tile; a slot of stored blocks
  static constexpr int kStages = 3, kSlots = 3;
  static constexpr int kQueryPitch = 2 * D + 16;         // bytes: rows on different banks
  static constexpr int kWeights = kRows * kKeys * 2;     // of a warpgroup's tile
  static constexpr int kSmem = (2 * kStages + kSlots) * kBytes + 2 * kWeights + kRows * kQueryPitch + 1024;
  static constexpr int kPitch = D + 4;                   // floats per row of a part
  static_assert(2 * kRows * kPitch * 4 <= (2 * kStages + kSlots) * kBytes + 2 * kWeights, "the parts fit the tiles' place");
};

__device__ __forceinline__ void sts(uint32_t addr, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(addr), "r"(x) : "memory");
}

// A lane's words of a stored block are those of 8 x 8 matrices (lane 4 g + t:
// row g, columns 2 t and 2 t + 1), whose rows stmatrix writes 16 bytes at a
// time, four matrices at once.  `at`: the tile + the place that this lane
// addresses (row lane & 7 of matrix lane >> 3), low bits ready for the swizzle,
// where 16-byte column c of a 128-byte row r lies at c ^ (r & 7).
__device__ __forceinline__ void store_matrices(uint32_t at, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(x0), "r"(x1), "r"(x2),
               "r"(x3)
               : "memory");
}
// K, place: row, column lane >> 3.  V (transposed), place: row of channel group
// lane >> 4, column 2 block + (lane >> 3 & 1).
__device__ __forceinline__ uint32_t k_place(int lane) { return (lane & 7) * 128 + (((lane >> 3) ^ (lane & 7)) << 4); }
__device__ __forceinline__ uint32_t v_place(int lane, int block) {
  return (lane >> 4) * 1024 + (lane & 7) * 128 + (((2 * block + (lane >> 3 & 1)) ^ (lane & 7)) << 4);
}
// 512 bytes r of a block of fp16 values (k16_offset, v16_offset):
template <int D>
__device__ __forceinline__ void store_k16(uint32_t at, int block, int r, uint4 x) {
  const int nt = r / (D / 32), k2 = r % (D / 32);        // token 8 nt + g, channels 32 k2 + 8 i + 2 t
  store_matrices((at ^ ((k2 & 1) << 6)) + (2 * block + nt) * 1024 + (k2 >> 1) * (kKeys * 128), x.x, x.y, x.z, x.w);
}
__device__ __forceinline__ void store_v16(uint32_t at, int r, uint4 x) {
  store_matrices(at + 2 * r * 1024, x.x, x.y, x.z, x.w);     // channel 8 (2 r + i / 2) + g, tokens 8 (i & 1) + 2 t
}
// and of codes (k8_offset, v8_offset):
template <int D>
__device__ __forceinline__ void store_k8(uint32_t at, int block, int r, uint4 x) {
  const int nt = r / (D / 64), c = r % (D / 64);         // token 8 nt + g, channels 64 c + 16 i + 8 e + 2 t
  const uint32_t to = at + (2 * block + nt) * 1024 + c * (kKeys * 128);
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) codes(word(x, i), y[2 * i], y[2 * i + 1]);
  store_matrices(to, y[0], y[1], y[2], y[3]);
  store_matrices(to ^ 64, y[4], y[5], y[6], y[7]);
}
__device__ __forceinline__ void store_v8(uint32_t at, int r, uint4 x) {
  uint32_t y[8];                                         // channel 8 (4 r + i) + g, tokens 8 e + 2 t
#pragma unroll
  for (int i = 0; i < 4; ++i) codes(word(x, i), y[2 * i], y[2 * i + 1]);
  store_matrices(at + 4 * r * 1024, y[0], y[1], y[2], y[3]);
  store_matrices(at + (4 * r + 2) * 1024, y[4], y[5], y[6], y[7]);
}

// ------------------------------------------------------------- dealt keys
// Each sequence's keys are dealt to as many CTAs per row tile as its own length
// deserves, so that all CTAs take about as long, one for each SM or two; parts
// go through a workspace and a second kernel joins them.
// The lengths and the drafts in use are on the device only, so a warp of every
// CTA works out the same deal.  Against equal parts within clusters, which cost
// 4 us less at equal lengths, at the time this was taken: 37 to 4097 entries
// with 0 to 61 drafts 76 -> 43 us; one sequence of 32768 with 32 drafts, for
// which clusters find 96 SMs, 92 -> 76 us; 64 drafts on four of 8192, two CTAs an
// SM, 128 -> 113 us.
constexpr int kSMs = 152, kCtas = 2 * kSMs;
static_assert(kDealtMost == kCtas, "a row tile of a sequence takes a CTA");
constexpr int kMostParts = 32, kLeastTiles = 4;          // parts of a row tile; key tiles of a part
struct Deal {                            // of a sequence
  int first, parts, tiles, unused;       // CTA, parts of a row tile, row tiles with drafts per KV head
};
struct Place {
  int b, at, parts, tiles;               // of a CTA: at / parts: KV head and row tile, at % parts: its part
};
struct DealtSpace {
  Deal deal[kCtas];                      // by sequence
  uint4 bad[kCtas];                      // by CTA: drafts among its keys with values that are not finite
  float2 sum[kCtas][kRows];              // reference and sum of a row
  float4 part[1];                        // [CTA][kRows][D / 4], not normalised
};
__host__ __device__ __forceinline__ long long key_tiles(const Shape& s, long long n8, int drafts) {
  return (n8 + kKeys - 1) / kKeys + (s.WR / 16 + (drafts + 15) / 16 + 3) / 4 + kChange;
}

__device__ __forceinline__ void deal_keys(const Shape& s, const Dev& d, const Call& a, int lane, int* keys, int* units,
                                          Place& place) {
  int longest = 1;
  for (int b = lane; b < s.B; b += 32) {
    const int drafts = drafts_of(a, b);
    keys[b] = (int)key_tiles(s, d.n8[lb_index(s, a.layer, b)], drafts);
    units[b] = (drafts * s.G + kRows - 1) / kRows * s.Hkv;
    if (units[b]) longest = max(longest, keys[b]);
  }
  __syncwarp();
  longest = __reduce_max_sync(0xffffffffu, longest);
  // the fewest tiles of a part for which there are CTAs enough
  int each = max((longest + kMostParts - 1) / kMostParts, kLeastTiles), enough = max(longest, each);
  while (each < enough) {
    const int half = (each + enough) / 2;
    int ctas = 0;
    for (int b = lane; b < s.B; b += 32) ctas += units[b] * ((keys[b] + half - 1) / half);
    if (__reduce_add_sync(0xffffffffu, ctas) <= a.ctas)
      enough = half;
    else
      each = half + 1;
  }
  DealtSpace* space = reinterpret_cast<DealtSpace*>(a.dealt);
  int first = 0;
  for (int b0 = 0; b0 < s.B; b0 += 32) {
    const int b = b0 + lane, parts = b < s.B ? (keys[b] + each - 1) / each : 0, ctas = b < s.B ? parts * units[b] : 0;
    int upto = ctas;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const int mine = first + upto - ctas, at = (int)blockIdx.x - mine;
    if (at >= 0 && at < ctas) place = Place{b, at, parts, units[b] / s.Hkv};
    if (blockIdx.x == 0 && b < s.B) space->deal[b] = Deal{mine, parts, units[b] / s.Hkv, 0};
    first += __shfl_sync(0xffffffffu, upto, 31);
  }
}

// A row from its parts, by D / 4 lanes: part(k, z, y) gives the (reference,
// sum) and four channels of the k-th.  `bad`: drafts with values that are not
// finite; path(): those that the row sees.
template <bool BF16, typename Part, typename Path>
__device__ __forceinline__ void write_row(const Shape& s, const Call& a, int b, int h, int r, int col, bool used, int parts,
                                          const uint32_t* bad, Part part, Path path) {
  const int tok = r / s.G, head = h * s.G + r % s.G;
  uint16_t* dst = a.out + b * a.o_b + tok * a.o_t + head * a.o_h + col;
  float* lse = a.lse && col == 0 ? a.lse + ((long long)b * a.T + tok) * s.Hq + head : nullptr;
  if (!used) {                                           // no draft: sees nothing
    *reinterpret_cast<uint2*>(dst) = make_uint2(0, 0);
    if (lse) *lse = -INFINITY;
    return;
  }
  float top = -INFINITY, sum = 0.f, x[4] = {};
#pragma unroll 1
  for (int k0 = 0; k0 < parts; k0 += 4) {                // four parts in flight
    float4 y[4];
    float2 z[4];
    float next = top;
#pragma unroll
    for (int k = 0; k < 4; ++k) part(min(k0 + k, parts - 1), z[k], y[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k) next = fmaxf(next, z[k].x);
    const float old = top == next ? 1.f : ex2(top - next);
    top = next;
    sum *= old;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] *= old;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k0 + k < parts) {
        const float f = z[k].x == top ? 1.f : ex2(z[k].x - top);
        sum += z[k].y * f;
        x[0] += y[k].x * f;
        x[1] += y[k].y * f;
        x[2] += y[k].z * f;
        x[3] += y[k].w * f;
      }
    }
  }
  const float inv = 1.f / sum;
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] *= inv;
  if (bad[0] | bad[1] | bad[2] | bad[3])
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      const float y = unfinite<BF16>(a, b, h, path(tok), bad, col + j);
      x[0] += j == 0 ? y : 0.f;
      x[1] += j == 1 ? y : 0.f;
      x[2] += j == 2 ? y : 0.f;
      x[3] += j == 3 ? y : 0.f;
    }
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]));
  if (lse) *lse = (top == -INFINITY ? 0.f : top * 0.6931471805599453f) + logf(sum * kUnlift);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tiles_kernel(Shape s, Dev d, const __grid_constant__ Call a) {
  using T = Tile<D>;
  constexpr int kBytes = T::kBytes, kStages = T::kStages, kSlots = T::kSlots;
  constexpr uint32_t kTmem = 512, kQuery = 128, kOut = 256;     // scores at 0 and 64
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[4 * kStages + 2 * kSlots + 17];
  __shared__ uint4 s_path[kMaxDrafts];
  __shared__ int s_up[kMaxDrafts];
  __shared__ float2 s_sum[2 * kRows], s_both[kRows];     // reference and sum of the rows: of each warpgroup, of the CTA
  __shared__ __align__(16) float s_scale[D];             // of V
  __shared__ __align__(16) float s_query[D];             // scales of K
  __shared__ float s_most[2][kRows];                     // largest |q| of a row: with those scales, without
  __shared__ uint32_t s_bad[4];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ Place s_place;
  __shared__ int s_keys[kCtas], s_units[kCtas];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
  const uint32_t tiles_at = smem_addr(smem), bar0 = smem_addr(s_bar);
  auto k_at = [&](int st) { return tiles_at + st * 2 * kBytes; };
  auto v_at = [&](int st) { return tiles_at + st * 2 * kBytes + kBytes; };
  auto k_full = [&](int st) { return bar0 + 8u * st; };
  auto v_full = [&](int st) { return bar0 + 8u * (kStages + st); };
  auto k_empty = [&](int st) { return bar0 + 8u * (2 * kStages + st); };
  auto v_empty = [&](int st) { return bar0 + 8u * (3 * kStages + st); };
  auto slot_at = [&](int sl) { return tiles_at + (2 * kStages + sl) * kBytes; };
  auto slot_full = [&](int sl) { return bar0 + 32u * kStages + 8u * sl; };
  auto slot_empty = [&](int sl) { return bar0 + 32u * kStages + 8u * (kSlots + sl); };
  const uint32_t rest = bar0 + 32u * kStages + 16u * kSlots;
  auto s_full = [&](int w) { return rest + 8u * w; };
  auto p_full = [&](int w) { return rest + 16u + 8u * w; };
  auto o_full = [&](int w) { return rest + 32u + 8u * w; };
  auto q_full = [&](int phase) { return rest + 48u + 8u * phase; };     // 0: for INT8 keys, 1: for fp16 keys
  auto s_read = [&](int w) { return rest + 80u + 8u * w; };
  auto o_done = [&](int w) { return rest + 96u + 8u * w; };
  auto drained = [&](int i) { return rest + 64u + 8u * (i < 2 ? i : i + 5); };
  const uint32_t paths_full = rest + 112u;
  const uint32_t weights_at = tiles_at + (2 * kStages + kSlots) * kBytes, query_at = weights_at + 2 * T::kWeights;

  if (warp == 16) tmem_alloc(smem_addr(&s_tmem), kTmem);
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < kStages; ++i) {
      bar_init(k_full(i), kConverters);
      bar_init(v_full(i), kConverters);
      bar_init(k_empty(i), 1);
      bar_init(v_empty(i), 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      bar_init(slot_full(i), 1);
      bar_init(slot_empty(i), 2 * kConverters);
    }
    for (int w = 0; w < 2; ++w) {
      bar_init(s_full(w), 1);
      bar_init(p_full(w), kRows / 32);
      bar_init(o_full(w), 1);
      bar_init(q_full(w), 2 * kRows / 32);
      bar_init(drained(w), 1);
      bar_init(drained(2 + w), 1);
      bar_init(s_read(w), kRows / 32);
      bar_init(o_done(w), 1);
    }
    bar_init(paths_full, 3);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (threadIdx.x < 4) s_bad[threadIdx.x] = 0;
  int split = a.split, rank = blockIdx.x % split;
  int tile = blockIdx.x / split % a.tiles, bh = blockIdx.x / split / a.tiles, b = bh / s.Hkv, h = bh % s.Hkv;
  pdl_wait();
  if (a.dealt) {
    asm volatile("griddepcontrol.launch_dependents;\n");
    if (warp == 0) {
      if (lane == 0) s_place.parts = 0;
      __syncwarp();
      deal_keys(s, d, a, lane, s_keys, s_units, s_place);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const Place p = s_place;
    if (p.parts == 0) {                                  // nothing for this CTA
      if (warp == 16) tmem_free(s_tmem, kTmem);
      return;
    }
    split = p.parts;
    b = p.b;
    rank = p.at % split;
    tile = p.at / split % p.tiles;
    h = p.at / split / p.tiles;
  }
  const size_t lb = lb_index(s, a.layer, b), u = unit_index(s, a.layer, b, h);
  const int n8 = d.n8[lb], ring = s.WR / 16;
  const int drafts = drafts_of(a, b), r0 = tile * kRows, used = drafts * s.G, all = a.T * s.G;
  const int rows = min(kRows, used - r0);                // of this tile that have a draft
  // Query rows into shared memory, and the factors that fit them into fp16,
  // by the first 16 warps: a row by D / 8 lanes.
  if (threadIdx.x < 512) {
    constexpr int kPer = D / 8, kAtOnce = 512 / kPer;
    const int first = threadIdx.x / kPer, c = threadIdx.x % kPer;
    const float4* sk = reinterpret_cast<const float4*>(d.sK + u * D + 8 * c);
    const float4 f0 = sk[0], f1 = sk[1];
    const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
    uint4 x[kRows / kAtOnce];
#pragma unroll
    for (int j = 0; j < kRows / kAtOnce; ++j) {
      const int i = first + j * kAtOnce, r = r0 + i;
      x[j] = i < rows ? *reinterpret_cast<const uint4*>(a.q + b * a.q_b + r / s.G * a.q_t + (h * s.G + r % s.G) * a.q_h + 8 * c)
                      : make_uint4(0, 0, 0, 0);
    }
    if (first == 0)
#pragma unroll
      for (int j = 0; j < 8; ++j) s_query[8 * c + j] = f[j];
#pragma unroll 1
    for (int j = 0; j < kRows / kAtOnce; ++j) {
      float most[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 y = float_pair<BF16>(word(x[0], k));
        most[0] = fmaxf(most[0], fmaxf(fabsf(y.x * f[2 * k]), fabsf(y.y * f[2 * k + 1])));
        most[1] = fmaxf(most[1], fmaxf(fabsf(y.x), fabsf(y.y)));
      }
#pragma unroll
      for (int o = 1; o < kPer; o <<= 1) {
        most[0] = fmaxf(most[0], __shfl_xor_sync(0xffffffffu, most[0], o));
        most[1] = fmaxf(most[1], __shfl_xor_sync(0xffffffffu, most[1], o));
      }
      const int i = first + j * kAtOnce;
      *reinterpret_cast<uint4*>(smem + (query_at - tiles_at) + i * T::kQueryPitch + 16 * c) = x[0];
      if (c < 2) s_most[c][i] = most[c];
#pragma unroll
      for (int k = 0; k + 1 < kRows / kAtOnce; ++k) x[k] = x[k + 1];
    }
  }
  // tiles of 64 keys: INT8 entries, then the window followed by the drafts up
  // to the last row's own
  const int nbf = rows > 0 ? ring + ((r0 + rows - 1) / s.G + 16) / 16 : 0;
  const int t8 = rows > 0 ? (n8 + kKeys - 1) / kKeys : 0, total = t8 + (nbf + 3) / 4;
  // the last part of several has the fp16 keys, and fewer tiles for it
  const int longer = total + (split > 1 ? kChange : 0);
  const int from = min(total, (int)((long long)longer * rank / split)), to = min(total, (int)((long long)longer * (rank + 1) / split));
  const int n = to - from, n_codes = min(max(t8 - from, 0), n);     // tiles of this CTA; INT8 ones, which come first
  if (threadIdx.x >= 512 && threadIdx.x < 512 + D) s_scale[threadIdx.x - 512] = d.sV[u * D + threadIdx.x - 512];
  fence_before();
  __syncthreads();
  if (a.split > 1) asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory");      // this CTA's shared memory is there
  fence_after();
  const uint32_t tmem = s_tmem;
  // Bounded waits of a whole warp; false once one, or another wait of the CTA,
  // has given up.  Two at once where both are wanted: a wait that is already
  // met costs some 150 cycles.
  auto ok_both = [&](uint32_t x, uint32_t px, uint32_t y, uint32_t py) {
    bool met = bar_test(x, px) & bar_test(y, py);
    if (__all_sync(0xffffffffu, met)) return true;
    const long long start = clock64();
    while (true) {
      met = bar_try(x, px) & bar_try(y, py);
      if (__all_sync(0xffffffffu, met)) return true;
      if (__any_sync(0xffffffffu, s_abort || clock64() - start > a.limit)) break;
    }
    if (!s_abort) atomicOr(d.status, kStatusTimeout);
    s_abort = 1;
    return false;
  };
  auto ok_all = [&](uint32_t bar, uint32_t parity) {
    bool met = bar_test(bar, parity);
    if (__all_sync(0xffffffffu, met)) return true;
    const long long start = clock64();
    while (true) {
      met = bar_try(bar, parity);
      if (__all_sync(0xffffffffu, met)) return true;
      if (__any_sync(0xffffffffu, s_abort || clock64() - start > a.limit)) break;
    }
    if (!s_abort) atomicOr(d.status, kStatusTimeout);
    s_abort = 1;
    return false;
  };
  // One arrival for a warp: those of 32 lanes at one barrier take their turns.
  auto arrive = [&](uint32_t bar) {
    fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive(bar);
  };
  // Every role ends here before it looks at s_abort: whichever wait gave up,
  // all of them then see it.  The roles that took registers have given them
  // back before; the others go on with the launch's count only after.
  auto leave = [&] {
    __syncwarp();
    bar_sync<1>(kThreads);
  };
  float ref = -INFINITY, l = 0.f;                        // softmax threads: reference (log2 units) and sum
  int mine = 0;                                          // tiles of this warpgroup

  if (warp >= 16) {
    regs_dec<kIssueRegs>();
    const int w = warp & 1;
    if (warp < 20) {
      // ---------------------------------------------------------- products
      // Warps 16 and 17 issue the scores of a softmax warpgroup's tiles, 18 and
      // 19 add up the values.  A warp that has issued products goes on to its
      // next wait only when they are done, so each kind has its own.  One lane
      // issues.
      constexpr uint32_t dqk = mma_desc(kRows, kKeys, false, false), dpv = mma_desc(kRows, D, false, false);
      const uint32_t scores = tmem + w * kKeys, output = tmem + kOut + w * D, query = tmem + kQuery;
      bool ok = true;
      if (warp < 18) {
        for (int i = w, c = 0; i < n && ok; i += 2, ++c) {
          const int st = i % kStages;
          if (c == 0 || (i >= n_codes && i - 2 < n_codes)) ok = ok_all(q_full(i >= n_codes), 0);
          // once the scores of the tile before are read
          const uint32_t read = c > 0 ? s_read(w) : k_full(st), parity = c > 0 ? (c - 1) & 1 : i / kStages & 1;
          ok = ok && ok_both(k_full(st), i / kStages & 1, read, parity);
          if (!ok) break;
          fence_after();
          if (elect()) {
            const uint32_t k = desc_lo(k_at(st), 16);
#pragma unroll 1
            for (int part = 0; part < (i < n_codes ? 2 : 1); ++part)
#pragma unroll
              for (int j = 0; j < D / 16; ++j)
                mma_ts(scores, query + part * (D / 2) + 8 * j, k + (((j >> 2) * (kKeys * 128) + (j & 3) * 32) >> 4),
                       desc_hi(1024), dqk, part + j > 0);
            mma_commit(s_full(w));
            mma_commit(k_empty(st));
          }
          __syncwarp();
        }
      } else {
        for (int i = w, c = 0; i < n && ok; i += 2, ++c) {
          const int st = i % kStages;
          ok = ok_both(v_full(st), i / kStages & 1, p_full(w), c & 1);
          if (!ok) break;
          fence_after();
          if (elect()) {
            const uint32_t v = desc_lo(v_at(st), 16), p = desc_lo(weights_at + w * T::kWeights, 16);
#pragma unroll
            for (int j = 0; j < kKeys / 16; ++j) mma_ss(output, p + 2 * j, v + 2 * j, desc_hi(1024), dpv, c > 0 || j > 0);
            mma_commit(o_done(w));
            mma_commit(i + 2 < n ? v_empty(st) : o_full(w));
          }
          __syncwarp();
        }
      }
      leave();
      if (s_abort && elect()) {                          // nothing in flight when the CTA ends
        mma_commit(drained(warp - 16));
        bar_wait(drained(warp - 16), 0);
      }
    } else {
      // ---------------------------------------------------------- copies
      // A slot for the K and V of an INT8 tile, one each for those of an fp16
      // tile; only stored blocks are copied.
      int count = 0;
      if (warp > 20 && rows > 0) {
        draft_paths<96>(a, b, drafts, threadIdx.x - 672, s_path, s_up, [] { bar_sync<2>(96); });
        __syncwarp();
        if (lane == 0) bar_arrive(paths_full);
      } else if (warp == 20) {
        const uint8_t *k8 = d.k8 + u * s.cstride * D, *v8 = d.v8 + u * s.cstride * D;
        const uint8_t* k16 = reinterpret_cast<const uint8_t*>(d.k16) + u * ring * 32 * D;
        const uint8_t* v16 = reinterpret_cast<const uint8_t*>(d.v16) + u * ring * 32 * D;
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
          const bool half = i >= n_codes;
          const int kb = (from + i - (half ? t8 : 0)) * 4;
          const int blocks = min(4, (half ? ring : (n8 + 15) / 16) - kb);      // none, or less, behind the window
          const uint32_t bytes = max(blocks, 0) * 16 * D * (half ? 2 : 1);
          for (int e = 0; e < (half ? 2 : 1) && ok; ++e) {
            const int sl = count % kSlots;
            if (count >= kSlots) ok = ok_all(slot_empty(sl), (count / kSlots - 1) & 1);
            if (!ok) break;
            if (lane == 0) {
              bar_expect(slot_full(sl), half ? bytes : 2 * bytes);
              if (half) {
                if (bytes) bulk_load(slot_at(sl), (e ? v16 : k16) + (size_t)kb * 32 * D, bytes, slot_full(sl));
              } else {
                bulk_load(slot_at(sl), k8 + (size_t)kb * 16 * D, bytes, slot_full(sl));
                bulk_load(slot_at(sl) + kBytes / 2, v8 + (size_t)kb * 16 * D, bytes, slot_full(sl));
              }
            }
            __syncwarp();
            ++count;
          }
        }
      }
      leave();
      if (s_abort && warp == 20 && lane == 0)            // no copy in flight when the CTA ends
        for (int i = max(0, count - kSlots); i < count; ++i) bar_wait(slot_full(i % kSlots), i / kSlots & 1);
    }
    __syncwarp();
    regs_inc<kRegs>();
  } else if (warp >= 8) {
    regs_dec<kConverterRegs>();
    // ---------------------------------------------------------- conversion
    const int block = warp & 3, t = lane & 3;
    const bool is_v = warp >= 12;
    const uint32_t place = is_v ? v_place(lane, block) : k_place(lane);
    const uint32_t tile0 = tiles_at + (is_v ? kBytes : 0) + place;
    const uint32_t full0 = is_v ? v_full(0) : k_full(0), empty0 = is_v ? v_empty(0) : k_empty(0);
    // Slot by slot: one for an INT8 tile, that of K and that of V for an fp16
    // tile (window blocks, then drafts, then nothing).  A warp waits for the
    // slots that it does not read, too, or its releases could run a use of the
    // slot ahead of the others'.
    auto position = [&](int i) {                         // of a slot of this warp's block of tile i, or -1
      const int kb = (from + i - t8) * 4 + block;
      return is_v && i >= n_codes && i < n && kb < ring ? d.pos[lb * s.S + s.cap + kb * 16 + (lane & 15)] : -1;
    };
    int pos = position(n_codes);
    const int slots = n + (n - n_codes);
#pragma unroll 1
    for (int sl = 0, slot = 0, use = 0; sl < slots; ++sl) {
      const bool half = sl >= n_codes;
      const int i = half ? n_codes + ((sl - n_codes) >> 1) : sl, st = i % kStages;
      const bool wanted = !half || ((sl - n_codes) & 1) == is_v;
      const uint32_t full = slot_full(slot);
      if (!(wanted && i >= kStages ? ok_both(full, use & 1, empty0 + 8 * st, (i / kStages - 1) & 1)
                                   : ok_both(full, use & 1, full, use & 1)))
        break;
      uint32_t at = tile0 + st * 2 * kBytes;
      uint32_t src = slot_at(slot) + lane * 16;
      if (wanted) {
        if (!half) {
          // Slots behind the last entry, and blocks that were not copied, hold
          // some bytes, whose codes are finite.
          src += (is_v ? kBytes / 2 : 0) + block * 16 * D;
          uint4 x[D / 32];
#pragma unroll
          for (int r = 0; r < D / 32; ++r) x[r] = lds(src + r * 512);
          if (is_v) {
#pragma unroll
            for (int r = 0; r < D / 32; ++r) store_v8(at, r, x[r]);
          } else {
#pragma unroll
            for (int r = 0; r < D / 32; ++r) store_k8<D>(at, block, r, x[r]);
          }
        } else {
          const int kb = (from + i - t8) * 4 + block;
          src += block * 32 * D;
          if (kb < ring) {
            // an empty slot of the window may hold anything: its values are cleared
            const uint32_t see = __ballot_sync(0xffffffffu, pos >= 0) & 0xffffu;
            pos = position(i + 1);
            const uint32_t m0 = (see >> (2 * t) & 1 ? 0xffffu : 0u) | (see >> (2 * t + 1) & 1 ? 0xffff0000u : 0u);
            const uint32_t m1 = (see >> (2 * t + 8) & 1 ? 0xffffu : 0u) | (see >> (2 * t + 9) & 1 ? 0xffff0000u : 0u);
#pragma unroll 1
            for (int r = 0; r < D / 16; ++r) {
              const uint4 y = lds(src + r * 512);
              if (is_v)
                store_v16(at, r, make_uint4(y.x & m0, y.y & m1, y.z & m0, y.w & m1));
              else
                store_k16<D>(at, block, r, y);
            }
          } else {
            // drafts, 16 bytes of a token's row at a time, by way of the slot
            const int key = lane & 15, tok = (kb - ring) * 16 + key;
            const uint16_t* rp =
                (is_v ? a.v + b * a.v_b + h * a.v_h : a.k + b * a.k_b + h * a.k_h) + tok * (is_v ? a.v_t : a.k_t);
            const uint32_t row = src - lane * 16 + key * 2 * D;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              const int c = 2 * j + (lane >> 4);         // channels 8 c .. 8 c + 7, at a column that spreads the banks
              if (tok < drafts)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(row + ((c ^ (key & 7)) << 4)), "l"(rp + 8 * c)
                             : "memory");
            }
            asm volatile("cp.async.wait_all;\n" ::: "memory");
            uint32_t bad = 0;
            at -= place;
#pragma unroll 1
            for (int j = 0; j < D / 16; ++j) {
              const int c = 2 * j + (lane >> 4);
              uint4 x = make_uint4(0, 0, 0, 0);
              if (tok < drafts) x = lds(row + ((c ^ (key & 7)) << 4));
#pragma unroll
              for (int k = 0; k < 4; ++k) word(x, k) = half_pair<BF16>(word(x, k));
              if (!is_v) {                               // row: the key; 16-byte column c & 7 of column block c >> 3
                const uint32_t to = at + (c >> 3) * (kKeys * 128) + (block * 16 + key) * 128 + (((c ^ key) & 7) << 4);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(to), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                             : "memory");
                continue;
              }
              // a value that is not finite is marked and taken as zero
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t& z = word(x, k);
                if ((z & 0x7c00u) == 0x7c00u) z &= 0xffff0000u, bad = 1;
                if ((z & 0x7c000000u) == 0x7c000000u) z &= 0xffffu, bad = 1;
              }
              // Even tokens take channels 0 .. 3 of the chunk from their odd
              // neighbours, which take 4 .. 7; a word is the pair's values.
              const bool odd = lane & 1;
              const uint32_t p0 = __shfl_xor_sync(0xffffffffu, odd ? x.x : x.z, 1);
              const uint32_t p1 = __shfl_xor_sync(0xffffffffu, odd ? x.y : x.w, 1);
              const uint32_t e0 = odd ? p0 : x.x, o0 = odd ? x.z : p0, e1 = odd ? p1 : x.y, o1 = odd ? x.w : p1;
              const uint32_t to = at + (8 * c + 4 * odd) * 128 + (key & 6) * 2;
              const int col = (2 * block + (key >> 3)) ^ (4 * odd);
              sts(to + (col << 4), __byte_perm(e0, o0, 0x5410));
              sts(to + 128 + ((col ^ 1) << 4), __byte_perm(e0, o0, 0x7632));
              sts(to + 256 + ((col ^ 2) << 4), __byte_perm(e1, o1, 0x5410));
              sts(to + 384 + ((col ^ 3) << 4), __byte_perm(e1, o1, 0x7632));
            }
            if (bad) atomicOr(&s_bad[tok >> 5], 1u << (tok & 31));
          }
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) {
        if (wanted) bar_arrive(full0 + 8 * st);
        bar_arrive(slot_empty(slot));
      }
      if (++slot == kSlots) slot = 0, ++use;
    }
    leave();
    __syncwarp();
    regs_inc<kRegs>();
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<kSoftmaxRegs>();
    float unit = 0.f;                                    // log2 units of a score
    const int w = warp >> 2, row = threadIdx.x & 127, r = r0 + row;
    const bool valid = row < rows;
    const int tok = valid ? r / s.G : 0;
    const uint32_t weights_row = weights_at + w * T::kWeights + row * 128;
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + w * kKeys + lane_base, to_ = tmem + kOut + w * D + lane_base, tq = tmem + kQuery + lane_base;
    // Query row of this thread into tensor memory, half of the channels by
    // each warpgroup: times the scales of K in two parts, or as it is.
    auto queries = [&](int phase) {
      const float most = s_most[phase][row], f = row_factor(most);
      unit = row_unit(a, most);
#pragma unroll 1
      for (int c = w * (D / 16); c < (w + 1) * (D / 16); ++c) {
        uint32_t hi[4], lo[4];
        uint4 x = lds(query_at + row * T::kQueryPitch + 16 * c);
        const float4 z0 = *reinterpret_cast<const float4*>(&s_query[8 * c]), z1 = *reinterpret_cast<const float4*>(&s_query[8 * c + 4]);
        const float z[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 y = float_pair<BF16>(word(x, j));
          // the scale first: with it the factor cannot overflow
          split2(y.x * (phase ? 1.f : z[2 * j]) * f, y.y * (phase ? 1.f : z[2 * j + 1]) * f, hi[j], lo[j]);
        }
        tmem_st4(tq + 4 * c, hi);
        if (phase == 0) tmem_st4(tq + D / 2 + 4 * c, lo);
      }
      wait_st();
      arrive(q_full(phase));
    };
    bool ok = (int)blockIdx.x != a.absent;
    // The queries of the first tiles; later, those as they are in the place of
    // the scaled ones, once no product needs these: the scores of the last two
    // INT8 tiles are there.
    int phase = n_codes > 0 ? 0 : 1, wanted = n > 0 ? phase : 2;
    auto write_queries = [&] {
      if (phase == 1)
        for (int j = max(0, n_codes - 2); j < n_codes && ok; ++j) ok = ok_all(s_full(j & 1), j >> 1 & 1);
      if (!ok) return;
      fence_after();
      queries(phase);
      wanted = phase++ == 0 && n_codes < n ? 1 : 2;
    };
    int pos[2];                                          // slots of the window that lane `lane` asks about
    auto positions = [&](int i) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int slot = ((from + i - t8) * 4 + 2 * e) * 16 + lane;
        pos[e] = i >= n_codes && i < n && slot < s.WR ? d.pos[lb * s.S + s.cap + slot] : -1;
      }
    };
    positions(w);
    for (int i = w - 2; ok; i += 2) {
      // before the first tile, before the first fp16 tile, or (if that is the
      // other warpgroup's) after the last one
      if (wanted == 0 || (wanted == 1 && (i >= n_codes || i < 0 || i >= n))) write_queries();
      if (i < 0) continue;
      if (i >= n || !ok) break;
      const bool half = i >= n_codes;
      const int left = n8 - (from + i) * kKeys;          // INT8 entries from the tile's first on
      uint32_t see[2] = {0xffffffffu, 0xffffffffu};      // keys of the tile that the row sees
      const bool whole = !half && left >= kKeys;
      if (!whole) {
        if (half && i < n_codes + 2) ok = ok_all(paths_full, 0);
        if (!ok) break;
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          uint32_t m = left >= 32 * e + 32 ? 0xffffffffu : left > 32 * e ? (1u << (left - 32 * e)) - 1u : 0u;
          if (half) {                                    // filled slots of the window, the drafts on its path
            const int kb = (from + i - t8) * 4 + 2 * e;
            m = __ballot_sync(0xffffffffu, (e ? pos[1] : pos[0]) >= 0);
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
              const int base = (kb + j - ring) * 16;
              if (base >= 0 && base < kMaxDrafts) {
                const uint32_t* path = reinterpret_cast<const uint32_t*>(&s_path[tok]);
                m |= (path[base >> 5] >> (base & 16) & 0xffffu) << (16 * j);
              }
            }
          }
          if (e)
            see[1] = m;
          else
            see[0] = m;
        }
      }
      if (i + 2 >= n_codes) positions(i + 2);
      ok = ok_all(s_full(w), mine & 1);
      if (!ok) break;
      fence_after();
      uint32_t x[kKeys];
      tmem_ld32(ts, x);
      tmem_ld32(ts + 32, x + 32);
      wait_ld32(x);
      wait_ld32(x + 32);
      arrive(s_read(w));
      float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (!whole) {
#pragma unroll
        for (int j = 0; j < kKeys; ++j)
          if (!(see[j / 32] >> (j & 31) & 1)) x[j] = 0xff800000u;
      }
#pragma unroll
      for (int j = 0; j < kKeys; j += 2)
        m[j / 2 % 4] = fmaxf(fmaxf(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), m[j / 2 % 4]);
      const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * unit;
      // The accumulator is rescaled when the reference moves, and takes the
      // scales of V when the INT8 entries of this warpgroup are done, both
      // after the product that wrote it.  When one row of the warp has to move,
      // those that lag at all follow, so that the others soon need not.
      const bool scale = half && mine > 0 && i - 2 < n_codes;
      if (scale || __any_sync(0xffffffffu, valid && top > ref + kLag)) {
        const float f = top > ref && ref > -INFINITY ? ex2(ref - top) : 1.f;
        if (mine > 0) {
          ok = ok_all(o_done(w), (mine - 1) & 1);
          if (!ok) break;
          fence_after();
          l *= f;
          auto times = [&](auto factor) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(to_ + c, o);
              wait_ld16(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * factor(c + j));
              tmem_st16(to_ + c, o);
            }
          };
          if (scale)
            times([&](int c) { return f * s_scale[c]; });
          else
            times([&](int) { return f; });
          wait_st();
        }
        ref = fmaxf(ref, top);
      }
      const float base = ref == -INFINITY ? 0.f : kLift - ref;
      const Pair unit_pair(unit, unit), base_pair(base, base);
      Pair sum[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)};
#pragma unroll
      for (int j = 0; j < kKeys / 2; ++j) {
        const float2 e = fma2(Pair(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), unit_pair, base_pair).get();
        const float y = ex2(e.x), z = ex2(e.y);
        sum[j & 1] = sum[j & 1] + Pair(y, z);
        x[j] = pack2<false>(y, z);
      }
      // the row of 128 bytes, 16-byte column c at c ^ (row & 7), once the
      // product of the tile before has read it
      if (mine > 0) ok = ok_all(o_done(w), (mine - 1) & 1);
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(weights_row + ((c ^ (row & 7)) << 4)),
                     "r"(x[4 * c]), "r"(x[4 * c + 1]), "r"(x[4 * c + 2]), "r"(x[4 * c + 3])
                     : "memory");
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      arrive(p_full(w));
      const float2 both = (sum[0] + sum[1]).get();
      l += both.x + both.y;
      ++mine;
    }
    if (ok && mine > 0) ok = ok_all(o_full(w), 0);
    fence_after();
    __syncwarp();
    regs_dec<kRegs>();
    leave();
  }

  // -------------------------------------------------------------------- join
  // (reference, sum) and output of every row, of both warpgroups, in shared
  // memory over the tiles; each CTA adds up the parts of its share of the rows,
  // or leaves its own in the workspace.
  cg::cluster_group cluster = cg::this_cluster();
  float* part = reinterpret_cast<float*>(smem);          // [2 * kRows][kPitch]
  const bool done = !s_abort, leaves = a.dealt && split > 1;
  DealtSpace* space = reinterpret_cast<DealtSpace*>(a.dealt);
  if (warp < 8) {
    // a CTA that gave up left no part: the rows become NaN
    s_sum[threadIdx.x] = done ? make_float2(ref, l) : make_float2(-INFINITY, NAN);
    const int w = warp >> 2;
    const uint32_t at = tmem + kOut + w * D + ((uint32_t)(warp & 3) << 21);
    const bool scale = mine > 0 && w + 2 * (mine - 1) < n_codes;     // its last tile had INT8 entries
    if ((warp & 3) * 32 < rows && done) {
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (mine > 0) {
          tmem_ld32(at + c, o);
          wait_ld32(o);
        }
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
          if (mine > 0)
            y = make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]), __uint_as_float(o[j + 2]),
                            __uint_as_float(o[j + 3]));
          if (scale) {
            const float4 f = *reinterpret_cast<const float4*>(s_scale + c + j);
            y = make_float4(y.x * f.x, y.y * f.y, y.z * f.z, y.w * f.w);
          }
          *reinterpret_cast<float4*>(part + threadIdx.x * T::kPitch + c + j) = y;
        }
      }
    }
  }
  __syncthreads();
  constexpr int kLanes = D / 4;                          // per row: four channels each
  const int col = threadIdx.x % kLanes * 4;
  for (int i = threadIdx.x / kLanes; i < rows; i += kThreads / kLanes) {
    const float2 z0 = s_sum[i], z1 = s_sum[kRows + i];
    float4* p = reinterpret_cast<float4*>(part + i * T::kPitch + col);
    const float4 x = *p, y = *reinterpret_cast<const float4*>(part + (kRows + i) * T::kPitch + col);
    const float top = fmaxf(z0.x, z1.x);
    const float f = z0.x == top ? 1.f : ex2(z0.x - top), g = z1.x == top ? 1.f : ex2(z1.x - top);
    if (leaves) p = reinterpret_cast<float4*>(reinterpret_cast<float*>(space->part) + ((long long)blockIdx.x * kRows + i) * D + col);
    *p = make_float4(x.x * f + y.x * g, x.y * f + y.y * g, x.z * f + y.z * g, x.w * f + y.w * g);
    if (col == 0) (leaves ? space->sum[blockIdx.x] : s_both)[i] = make_float2(top, z0.y * f + z1.y * g);
  }
  if (leaves && threadIdx.x == 0) space->bad[blockIdx.x] = make_uint4(s_bad[0], s_bad[1], s_bad[2], s_bad[3]);
  if (a.split > 1) {
    asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    // drafts with values that are not finite: the cluster has to know
    if (threadIdx.x < 4 * split && s_bad[threadIdx.x & 3] && threadIdx.x >> 2 != rank)
      atomicOr(cluster.map_shared_rank(s_bad, threadIdx.x >> 2) + (threadIdx.x & 3), s_bad[threadIdx.x & 3]);
    cluster.sync();
  } else {
    __syncthreads();
  }
  for (int i = rank + split * (threadIdx.x / kLanes); i < min(kRows, all - r0) && !leaves; i += split * (kThreads / kLanes))
    write_row<BF16>(
        s, a, b, h, r0 + i, col, i < rows, split, s_bad,
        [&](int k, float2& z, float4& y) {
          z = (a.split > 1 ? cluster.map_shared_rank(s_both, k) : s_both)[i];
          y = *reinterpret_cast<const float4*>((a.split > 1 ? cluster.map_shared_rank(part, k) : part) + i * T::kPitch + col);
        },
        [&](int t) { return s_path[t]; });
  if (a.split > 1) cluster.sync();                       // no CTA leaves while another reads its part
  fence_before();
  __syncthreads();
  if (warp == 16) {
    __syncwarp();
    fence_after();
    tmem_free(tmem, kTmem);
  }
}

// Rows of dealt keys from their parts, and rows without drafts of the tiles
// that no CTA took.
constexpr int kJoinThreads = 256, kJoinRows = 16;
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(Shape s, const __grid_constant__ Call a) {
  constexpr int kLanes = D / 4, kChunks = kRows / kJoinRows;
  __shared__ uint32_t s_bad[4];
  const int chunk = blockIdx.x % kChunks, tile = blockIdx.x / kChunks % a.tiles, bh = blockIdx.x / kChunks / a.tiles;
  const int b = bh / s.Hkv, h = bh % s.Hkv, r0 = tile * kRows, all = a.T * s.G;
  if (threadIdx.x < 4) s_bad[threadIdx.x] = 0;
  pdl_wait();
  const DealtSpace* space = reinterpret_cast<const DealtSpace*>(a.dealt);
  const Deal deal = space->deal[b];
  if (tile < deal.tiles && deal.parts == 1) return;      // written by its CTA
  const int parts = tile < deal.tiles ? deal.parts : 0, cta = deal.first + (h * deal.tiles + tile) * parts;
  const int used = drafts_of(a, b) * s.G, col = threadIdx.x % kLanes * 4;
  __syncthreads();
  if (threadIdx.x < 4 * parts) {
    const uint32_t bad = reinterpret_cast<const uint32_t*>(space->bad + cta)[threadIdx.x];
    if (bad) atomicOr(&s_bad[threadIdx.x & 3], bad);
  }
  __syncthreads();
  for (int i = chunk * kJoinRows + threadIdx.x / kLanes; i < min((chunk + 1) * kJoinRows, all - r0); i += kJoinThreads / kLanes)
    write_row<BF16>(
        s, a, b, h, r0 + i, col, r0 + i < used, parts, s_bad,
        [&](int k, float2& z, float4& y) {
          z = space->sum[cta + k][i];
          y = space->part[((cta + k) * kRows + i) * kLanes + col / 4];
        },
        [&](int t) {
          uint32_t m[4] = {0, 0, 0, 0};
          for (int j = t; j >= 0;) {
            m[j >> 5] |= 1u << (j & 31);
            const int p = a.parents ? a.parents[b * a.p_b + j * a.p_t] : j - 1;
            j = p < j ? p : -1;
          }
          return make_uint4(m[0], m[1], m[2], m[3]);
        });
}

template <int D, bool BF16>
int launch(const Shape& s, const Dev& d, const Call& a, cudaStream_t st) {
  static int done[kMaxDevices] = {};
  auto kernel = tree_tiles_kernel<D, BF16>;
  if (ensure_smem(kernel, Tile<D>::kSmem, done) != cudaSuccess) return -1;
  cudaLaunchConfig_t cfg = {};
  const long long units = (long long)s.B * s.Hkv * a.tiles;
  cfg.gridDim = dim3((unsigned)(a.dealt ? a.ctas : units * a.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tile<D>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = a.split;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, s, d, a) != cudaSuccess) return -1;
  if (!a.dealt) return 0;
  return launch_pdl(tree_join_kernel<D, BF16>, dim3((unsigned)(units * (kRows / kJoinRows))), dim3(kJoinThreads), 0, st, s, a) ==
                 cudaSuccess
             ? 0
             : -1;
}

}  // namespace

// Time in microseconds by a model: for the CTAs of an SM, one after the other, the
// start, the switch to fp16 keys and the join (19, 13 with 64 channels; 0.7 of that
// for each after the first, which finds its instructions fetched), and 0.76 a tile.
static double tiles_time(const Shape& s, long long ctas, long long tiles) {
  return (s.D == 128 ? 19.0 : 13.0) * (0.3 + 0.7 * (double)ctas) + 0.76 * (double)(ctas * tiles);
}

// Rounds of the clusters that are resident: those of one kind fill the SMs of a GPC
// only in part, those of 7 and 8 CTAs a good two thirds of the GPU.
double plan_tree_tiles(const Shape& s, int T, long long n8_bound, int* split) {
  static const int resident[kMaxSplit + 1] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
  const long long units = (long long)s.B * s.Hkv * (((long long)T * s.G + kRows - 1) / kRows);
  const long long keys = (n8_bound + kKeys - 1) / kKeys + (s.WR + T + kKeys - 1) / kKeys;
  double least = 1e30;
  for (int k = 1; k <= kMaxSplit; ++k) {
    const double t = tiles_time(s, (units + resident[k] - 1) / resident[k], (keys + k - 1) / k) + (k > 1 ? 1.0 : 0.0);
    if (t < least) {
      least = t;
      *split = k;
    }
  }
  return least;
}

size_t dealt_tree_bytes(const Shape& s, int T) {
  const long long units = (long long)s.B * s.Hkv * (((long long)T * s.G + kRows - 1) / kRows);
  return T == 0 || units > kCtas ? 0 : offsetof(DealtSpace, part) + (size_t)kCtas * kRows * s.D * sizeof(float);
}

double plan_dealt_tree(const Shape& s, int T, const long long* n8, int* most) {
  const long long units = (long long)s.Hkv * (((long long)T * s.G + kRows - 1) / kRows);       // of a sequence
  long long longest = 1;
  for (int b = 0; b < s.B; ++b) longest = std::max(longest, key_tiles(s, n8[b], T));
  double least = 1e30;
  for (int waves = 1; waves <= kCtas / kSMs; ++waves) {
    if (units * s.B > waves * kSMs) continue;
    long long each = std::max((longest + kMostParts - 1) / kMostParts, (long long)kLeastTiles), enough = std::max(longest, each);
    while (each < enough) {
      const long long half = (each + enough) / 2;
      long long ctas = 0;
      for (int b = 0; b < s.B; ++b) ctas += units * ((key_tiles(s, n8[b], T) + half - 1) / half);
      if (ctas <= waves * kSMs)
        enough = half;
      else
        each = half + 1;
    }
    const double t = 4.0 + tiles_time(s, waves, each);
    if (t < least) {
      least = t;
      *most = waves * kSMs;
    }
  }
  return least;
}

int launch_tree_tiles(const Shape& s, const Dev& d, const tree::Call& call, bool bf16, cudaStream_t st) {
  tree::Call a = call;
  a.tiles = (a.T * s.G + kRows - 1) / kRows;
  auto fn = s.D == 128 ? (bf16 ? launch<128, true> : launch<128, false>) : (bf16 ? launch<64, true> : launch<64, false>);
  return fn(s, d, a, st);
}

}  // namespace confkv

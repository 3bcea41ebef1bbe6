// Thin wrappers over the PTX instructions that the prompt attention kernel
// uses: mbarriers, tiled TMA loads, tensor memory and tcgen05.mma.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace confkv {
namespace tc {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// ------------------------------------------------------------- mbarriers
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// One poll of a phase; the thread may sleep in it, for up to kSleepNs unless
// the phase completes.  A poll that returns at once instead takes issue slots
// from the softmax warps of the same quarter of the SM.
constexpr uint32_t kSleepNs = 20000;
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kSleepNs)
      : "memory");
  return ok != 0;
}
// Polls until the phase completes; false after about four seconds.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  if (bar_try(bar, parity)) return true;
  const long long start = clock64();
  do {
    if (bar_try(bar, parity)) return true;
  } while (clock64() - start < (1LL << 33));
  return false;
}

// Barrier ID over `threads` threads of converged warps.
template <int ID>
__device__ __forceinline__ void bar_sync(int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"n"(ID), "r"(threads) : "memory");
}

// ------------------------------------------------------------- TMA
// Box at (x, head, token) of a (channel, head, token) tensor map.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int head, int token,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n" ::"r"(dst),
      "l"(map), "r"(x), "r"(head), "r"(token), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}

// ------------------------------------------------------------- work of other CTAs
// Takes over the work of a CTA of this grid that has not started: its index
// arrives in the 16 bytes at `response`, completing `bar`.  Not to be asked
// again after a refusal.
__device__ __forceinline__ void take_cta(uint32_t response, uint32_t bar) {
  bar_expect(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(
                   response),
               "r"(bar)
               : "memory");
}
// The index taken over, or -1 if there was none.
__device__ __forceinline__ int taken_cta(uint32_t response) {
  int x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 r;\n .reg .b32 y, z, w;\n ld.shared.b128 r, [%1];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n mov.b32 %0, -1;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, r;\n"
      " fence.proxy.async.shared::cta;\n}\n"
      : "=r"(x)
      : "r"(response)
      : "memory");
  return x;
}

// ------------------------------------------------------------- tensor memory
__device__ __forceinline__ void tmem_alloc(uint32_t result, uint32_t columns) {   // one whole warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(result), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {      // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

#define CONFKV_IO4(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3])
#define CONFKV_OUT4(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3])
#define CONFKV_IN4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])
// 32 consecutive columns of the warp's 32 lanes, one lane per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31}, [%32];\n"
      : CONFKV_OUT4(r, 0), CONFKV_OUT4(r, 4), CONFKV_OUT4(r, 8), CONFKV_OUT4(r, 12), CONFKV_OUT4(r, 16),
        CONFKV_OUT4(r, 20), CONFKV_OUT4(r, 24), CONFKV_OUT4(r, 28)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : CONFKV_OUT4(r, 0), CONFKV_OUT4(r, 4), CONFKV_OUT4(r, 8), CONFKV_OUT4(r, 12)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n" ::CONFKV_IN4(r, 0),
      CONFKV_IN4(r, 4), CONFKV_IN4(r, 8), CONFKV_IN4(r, 12), "r"(addr)
      : "memory");
}
// Waits for the loads so far.  The registers are operands, so that nothing
// that reads them is moved up across the wait.
__device__ __forceinline__ void wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : CONFKV_IO4(r, 0), CONFKV_IO4(r, 4), CONFKV_IO4(r, 8), CONFKV_IO4(r, 12), CONFKV_IO4(r, 16),
                 CONFKV_IO4(r, 20), CONFKV_IO4(r, 24), CONFKV_IO4(r, 28)
               :
               : "memory");
}
__device__ __forceinline__ void wait_ld16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : CONFKV_IO4(r, 0), CONFKV_IO4(r, 4), CONFKV_IO4(r, 8), CONFKV_IO4(r, 12)
               :
               : "memory");
}
#undef CONFKV_IO4
#undef CONFKV_OUT4
#undef CONFKV_IN4

// ------------------------------------------------------------- tcgen05.mma
// Shared-memory matrix descriptor of a 128-byte-swizzled tile: rows of 128
// bytes in groups of 8 (1024 bytes).  `group` is the distance of consecutive
// 8-row groups, `block` that of consecutive 64-element column blocks of an
// operand whose contiguous axis is M or N (not read for one whose contiguous
// axis is K, where a K step advances inside the 128-byte row).
// The address is in the low word, in units of 16 bytes; the high word is the
// same for every tile.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t block) {
  return ((addr & 0x3FFFF) >> 4) | ((block >> 4) << 16);
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t group) { return (group >> 4) | (1u << 14) | (2u << 29); }
// Instruction descriptor of kind::f16: fp32 accumulators, A and B both fp16
// or both bf16, A with contiguous K, B with contiguous K or N.
__host__ __device__ constexpr uint32_t mma_desc(int M, int N, bool bf16, bool b_n_contiguous) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_n_contiguous ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tensor memory] (+)= A[shared] * B[shared]; low words of the descriptors,
// whose high word is `hi`.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t desc,
                                       bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.u32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(desc), "r"((uint32_t)accumulate)
      : "memory");
}
// D[tensor memory] (+)= A[tensor memory] * B[shared]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t desc,
                                       bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.u32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(desc), "r"((uint32_t)accumulate)
      : "memory");
}
// Arrives on `bar` once every tcgen05 operation this thread issued so far is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}

// True in one lane of a converged warp, always the same one: the code that
// it guards is issued once, from uniform registers.
__device__ __forceinline__ bool elect() {
  uint32_t one;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one)::"memory");
  return one != 0;
}

// ------------------------------------------------------------- registers
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// 32 bytes in one store (32-byte aligned).
__device__ __forceinline__ void st_global32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Two fp32 values as fp16 or bf16 pairs, `lo` in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace tc
}  // namespace confkv

// tcgen05 (5th-generation tensor core), TMEM and tensor-map TMA helpers.
//
// Shared-memory operands are 128-byte-swizzled (64-byte for 64-byte rows)
// tiles as tensor-map TMA writes them: rows of 128 (64) bytes, the 16-byte
// chunk index xor-ed with the row (row / 2) modulo 8 (4), tiles on 1024-byte
// boundaries. A tile serves as a K-major operand (rows are M or N, bytes along
// K) or, transposed, as an MN-major one (rows are K, bytes along M or N).
#pragma once

#include "sv_common.cuh"

namespace sv {

// ------------------------------------------------------------- descriptors

// Matrix descriptor of a swizzled tile: start address, strides (bytes),
// swizzle (2 = 128 B, 4 = 64 B). For both majors the stride between groups of
// eight rows is `sbo`; `lbo` is the stride between 128-byte (64-byte) blocks
// along M / N of an MN-major operand.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | static_cast<uint64_t>(lbo >> 4) << 16 |
         static_cast<uint64_t>(sbo >> 4) << 32 | 1ull << 46 | static_cast<uint64_t>(swizzle) << 61;
}

// Instruction descriptor: fp32 accumulators, operand type code for A and B
// (kind::f8f6f4: 0 = e4m3; kind::f16: 0 = f16), MN-major flags, sizes.
__host__ __device__ constexpr uint32_t tc_idesc(uint32_t type, bool a_mn, bool b_mn, uint32_t m, uint32_t n) {
  return 1u << 4 | type << 7 | type << 10 | static_cast<uint32_t>(a_mn) << 15 | static_cast<uint32_t>(b_mn) << 16 |
         (n >> 3) << 17 | (m >> 4) << 24;
}

// D (TMEM) = A B (+ D if acc), both operands in shared memory, e4m3 x e4m3.
__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}

// All tcgen05 operations this thread issued so far: arrive on bar when done.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ------------------------------------------------------------------- TMEM

// Warp-collective; cols a power of two >= 32. The address lands at smem word `slot`.
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 consecutive columns of the warp's 32 lanes (address: column, plus the
// warp's first lane << 16). Results are valid after tmem_ld_wait.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
// Ties register values to the point after the wait: the compiler must not read them before it.
template <int N>
__device__ __forceinline__ void tmem_use(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// -------------------------------------------------------------------- TMA

// Box of a 3-D tensor map (byte column 0, row y, page-head z) into shared
// memory; completion counted on bar.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(0), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Barrier over `threads` threads with an OR of a predicate.
__device__ __forceinline__ bool named_barrier_or(int id, int threads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.b32 a, %3, 0;\n\tbar.red.or.pred b, %1, %2, a;\n\tselp.b32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0;
}

// mbarrier wait that may sleep in hardware for about `ns` before it answers.
__device__ __forceinline__ bool mbar_try_wait_for(uint32_t bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2, %3;\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}

// A bounded mbarrier wait that also gives up once another thread has: `fail`
// is a word of shared memory. The loop is one function for all waits of a
// kernel: these kernels' roles run different code at once, and their speed
// hangs on all of it staying in the instruction cache.
constexpr uint32_t kWaitSleepNs = 20000;

static __device__ __noinline__ bool wait_or_fail_slow(uint32_t bar, uint32_t parity, volatile uint32_t* fail) {
  uint64_t prev = global_timer_ns(), spent = 0;
  for (uint32_t it = 1; it < kWaitIters; ++it) {
    if (mbar_try_wait_for(bar, parity, kWaitSleepNs)) return true;
    if (*fail) return false;
    const uint64_t now = global_timer_ns();
    const uint64_t gap = now - prev;
    spent += gap < kWaitGapNs ? gap : kWaitGapNs;
    prev = now;
    if (spent > kWaitNs) break;
  }
  *fail = 1;
  return false;
}

__device__ __forceinline__ bool wait_or_fail(uint32_t bar, uint32_t parity, volatile uint32_t* fail) {
  return mbar_try_wait_for(bar, parity, kWaitSleepNs) || wait_or_fail_slow(bar, parity, fail);
}

}  // namespace sv

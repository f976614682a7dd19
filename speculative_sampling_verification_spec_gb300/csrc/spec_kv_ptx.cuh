#pragma once
// spec_kv_ptx.cuh -- wrappers of the PTX the tensor-core attention kernel is made
// of: mbarriers with bounded waits, tensor-map copies, tensor memory and the
// fifth-generation matrix instruction with its descriptors.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace spec_kv_detail {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---- mbarriers -------------------------------------------------------------
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void bar_arrive_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits at most about two seconds, and no longer than until *gave_up is set (by
// whichever wait of the CTA ran out first, so that all of them end).  False: gave up.
static __device__ __noinline__ bool bar_wait_slow(uint64_t* b, uint32_t parity, volatile int* gave_up) {
  const uint64_t t0 = now_ns();
  for (uint32_t i = 0; i < 100000u; ++i) {
    if (bar_try(b, parity)) return true;
    if (*gave_up || now_ns() - t0 > 2000000000ull) break;
  }
  *gave_up = 1;
  return false;
}
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, volatile int* gave_up) {
  if (bar_try(b, parity)) return true;
  return bar_wait_slow(b, parity, gave_up);
}

__device__ __forceinline__ void fence_bar_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
// orders this thread's plain accesses of shared memory before later asynchronous ones
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- tensor-map copies -----------------------------------------------------
// a policy for lines that are read once and need not stay in the L2 cache
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], "
      "[%6], %7;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tensor memory ---------------------------------------------------------
// allocation, release: one whole warp; columns a power of two from 32
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
// N consecutive columns of the thread's lane
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float* x);
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t addr, const float* x);
template <int N>
__device__ __forceinline__ void tmem_tie(float* x);
template <>
__device__ __forceinline__ void tmem_ld<8>(uint32_t addr, float* x) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "r"(addr));
}
template <>
__device__ __forceinline__ void tmem_st<8>(uint32_t addr, const float* x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}
template <>
__device__ __forceinline__ void tmem_ld<4>(uint32_t addr, float* x) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
               : "r"(addr));
}
template <>
__device__ __forceinline__ void tmem_st<4>(uint32_t addr, const float* x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3])
               : "memory");
}
template <>
__device__ __forceinline__ void tmem_tie<4>(float* x) {
  asm volatile("" : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]));
}
// nothing that uses these values moves ahead of the wait before it
template <>
__device__ __forceinline__ void tmem_tie<8>(float* x) {
  asm volatile("" : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---- the matrix instruction ------------------------------------------------
// Shared-memory operand descriptor: start address, leading and stride byte offsets
// (all in 16-byte units), the fixed bit of this generation, the swizzle.
enum { kSwizzleNone = 0, kSwizzle128 = 2, kSwizzle64 = 4 };
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead_bytes, uint32_t stride_bytes, int swizzle) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>((lead_bytes >> 4) & 0x3fffu) << 16) |
         (static_cast<uint64_t>((stride_bytes >> 4) & 0x3fffu) << 32) | (uint64_t(1) << 46) |
         (static_cast<uint64_t>(swizzle) << 61);
}
// Instruction descriptor: e4m3 times e4m3 or e5m2, float accumulators, M x N; an
// operand is K-major (its K runs along the contiguous bytes) or else transposed.
enum { kE4m3 = 0, kE5m2 = 1 };
__host__ __device__ constexpr uint32_t instr_desc(int M, int N, bool a_transposed, bool b_transposed, int b_type) {
  return (1u << 4) | (static_cast<uint32_t>(b_type) << 10) | ((a_transposed ? 1u : 0u) << 15) |
         ((b_transposed ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D (+)= A B, 32 of K at a time; one thread issues it
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// arrives on the barrier when all matrix instructions issued before are complete
__device__ __forceinline__ void mma_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b))
               : "memory");
}

}  // namespace spec_kv_detail

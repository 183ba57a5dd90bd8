// Barriers and tensor-core instructions that the tcgen05 kernels share.
#pragma once

#include "tks_attn.cuh"

namespace tks {
namespace attn {

__device__ __forceinline__ void bar_init(uint32_t a, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(a), "r"(n) : "memory");
}
// Barrier and tensor instructions take their addresses from uniform registers: with an address
// that the compiler cannot see to be the same for the whole warp, each becomes a loop over its
// lanes (some 200 cycles). So whole warps come here, with addresses made of uniform values, and
// one elected lane acts.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
// One arrival for the warp.
__device__ __forceinline__ void bar_arrive(uint32_t a) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(a)
      : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t a, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred q;\n\tmbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(ok) : "r"(a), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ long long now_ns() {
  long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// A place in a ring of N, and the parity of its use: (x mod N, x / N mod 2) for x = 0, 1, ...
template <int N>
struct Ring {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      parity ^= 1;
    }
  }
};

// Whether a barrier's phase of this parity is over, waiting for it up to the time limit (then it is
// reported). The answer is the same for all lanes of the warp. NAP: a wait that may be answered
// late sleeps between its looks, and leaves the issue slots to the others.
template <bool NAP>
__device__ __forceinline__ bool bar_wait(uint32_t a, uint32_t parity, long long limit, unsigned* status) {
  long long t0 = 0;
  for (unsigned looks = 1; !__all_sync(0xffffffffu, bar_try(a, parity)); ++looks) {
    if (NAP) __nanosleep(100);
    if (looks % 64 == 0) {  // (the clock is read now and then)
      const long long t = now_ns();
      if (t0 == 0) t0 = t;
      if (__any_sync(0xffffffffu, t - t0 > limit)) {
        if ((threadIdx.x & 31) == 0) report(status, kStatTimeoutBit);
        return false;
      }
    }
  }
  return true;
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// Between the producers' ordinary stores to a stage and the products' reads of it. The warp that
// issues the products executes it, after the barrier: a producer's own would also wait for the
// loads that it has under way for the next tile (the wide tree of 64 drafts: 224 us, so 218).
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
#define TKS_R32(M) M(0), M(1), M(2), M(3), M(4), M(5), M(6), M(7), M(8), M(9), M(10), M(11), M(12), M(13), M(14), M(15), \
                   M(16), M(17), M(18), M(19), M(20), M(21), M(22), M(23), M(24), M(25), M(26), M(27), M(28), M(29), M(30), M(31)
// 32 columns of the warp's 32 lanes: a thread's lane, one register each.
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t addr) {
#define TKS_OUT(i) "=r"(r[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : TKS_R32(TKS_OUT) : "r"(addr) : "memory");
#undef TKS_OUT
}

// A shared-memory operand of 128-byte rows, 128-byte swizzled. K-major (keys): 8-row
// groups 1024 bytes apart. MN-major (values, transposed): 64-element blocks of the
// row `lead` bytes apart, 8-key groups 1024 bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// 32-bit accumulators; both inputs half or bfloat16; B K-major or transposed; M = 128.
__device__ __forceinline__ constexpr uint32_t instr(bool half, bool trans_b, int n) {
  return (1u << 4) | ((half ? 0u : 1u) << 7) | ((half ? 0u : 1u) << 10) | ((trans_b ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

}  // namespace attn
}  // namespace tks

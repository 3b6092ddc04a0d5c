// What the tcgen05 kernels of the FP8 product and of group-limited routing's product share: barriers
// and bounded waits, bulk and TMA copies, matrix descriptors, TMEM ordering (internal to libmoe).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"

namespace moe {

constexpr uint64_t kTcWaitNs = 2000000000ull;   // a wait gives up after 2 s

static __device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
static __device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
static __device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}
// One arrival of the warp: lane 0, by predicate (a branch would cost a reconvergence).
static __device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.eq.s32 q, %1, 0;\n"
      "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(lane)
      : "memory");
}
static __device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
// One try by the lane whose `who` is 0 only, by predicate: 32 lanes polling one barrier are 32
// operations on it.
static __device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity, int who) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.eq.s32 q, %3, 0;\nsetp.ne.s32 p, 0, 0;\n"
      "@q mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(who)
      : "memory");
  return ok != 0;
}
// The same without suspending the thread, for a look ahead of the wait.
static __device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity, int who) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.eq.s32 q, %3, 0;\nsetp.ne.s32 p, 0, 0;\n"
      "@q mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(who)
      : "memory");
  return ok != 0;
}
// Bounded wait of a converged warp (votes decide: the warp never diverges); `early`: the result of
// a look at this phase already taken, whose latency other work has covered.  A vote orders no
// memory: what the barrier guards is only the polling lane's (`who` 0) to touch.
static __device__ __forceinline__ bool lead_wait(uint64_t* b, uint32_t parity, int32_t* err,
                                                 int code, int who, bool early = false) {
  const uint32_t bar = smem_u32(b);
  if (__any_sync(0xffffffffu, early)) return true;
  if (__any_sync(0xffffffffu, mbar_try(bar, parity, who))) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (__any_sync(0xffffffffu, mbar_try(bar, parity, who))) return true;
    if ((i & 255) == 0 && __any_sync(0xffffffffu, globaltimer() - t0 > kTcWaitNs)) {
      pdl_wait();                               // (the word may still be being cleared)
      if (who == 0) atomicExch(err, code);
      return false;
    }
  }
}
// The same for all lanes: __syncwarp passes on to them what lane 0 has acquired.
static __device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t parity, int32_t* err,
                                                 int code, bool early = false) {
  const bool ok = lead_wait(b, parity, err, code, threadIdx.x & 31, early);
  __syncwarp();
  return ok;
}
static __device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes,
                                                uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
static __device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                              uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}
static __device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// One lane of a converged warp, the same one every time.
static __device__ __forceinline__ bool elect_one() {
  uint32_t pred = 0;
  asm volatile(
      "{\n.reg .pred p;\n.reg .b32 r;\nelect.sync r|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(pred));
  return pred != 0;
}
// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 B apart.
static __device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
static __device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
static __device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
static __device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
static __device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// cuTensorMapEncodeTiled, or NULL where the driver has none.
static inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

}  // namespace moe

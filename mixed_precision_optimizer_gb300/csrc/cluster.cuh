// Thread-block clusters: the rank and size, the barrier, stores into another CTA's
// shared memory (mapa, st.shared::cluster), and mail: values that arrive there with
// an mbarrier that counts their bytes (st.async).  The cluster's barrier makes a
// CTA wait until its stores to global memory are done, a few microseconds under
// load; mail orders nothing but itself.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace mpopt {
namespace {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Also orders the global and shared memory accesses of the cluster's threads.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of CTA `rank`'s copy of a place in shared memory.
__device__ __forceinline__ uint32_t at_peer(const void* p, uint32_t rank) {
  uint32_t m;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(m)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return m;
}
__device__ __forceinline__ void store_peer(uint32_t at, int64_t v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ void store_peer(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// One mbarrier for each of two alternating places.  init() by one thread, a
// cluster_sync() of all before the first use; for message k (0, 1, 2, ...) one
// thread of each CTA calls expect(k, bytes) with what all CTAs send it, the
// senders send(), the readers wait(k).  A place is used again for message k + 2:
// who sends that has to have waited for message k + 1, and its readers to have
// read message k before they sent theirs.
struct Mailbox {
  uint64_t* bar;         // [2] in shared memory

  static __device__ __forceinline__ uint32_t u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
  __device__ __forceinline__ void init() const {
    for (int i = 0; i < 2; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(u32(bar + i)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __device__ __forceinline__ void expect(int k, uint32_t bytes) const {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(u32(bar + (k & 1))), "r"(bytes) : "memory");
  }
  // v into CTA `rank`'s copy of *to, as a part of message k.
  __device__ __forceinline__ void send(int k, const void* to, uint32_t rank, float2 v) const {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at_peer(to, rank)),
                 "f"(v.x), "f"(v.y), "r"(at_peer(bar + (k & 1), rank))
                 : "memory");
  }
  // Whether message k is there: every try may suspend the thread for a while, and
  // after kTries of them (a second or more) the wait gives up.
  static constexpr int kTries = 1 << 20;
  __device__ __forceinline__ bool wait(int k) const {
    const uint32_t at = u32(bar + (k & 1)), parity = static_cast<uint32_t>(k >> 1) & 1u;
    for (int i = 0; i < kTries; ++i) {
      uint32_t there;
      asm volatile(
          "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
          " selp.u32 %0, 1, 0, p;\n}"
          : "=r"(there)
          : "r"(at), "r"(parity)
          : "memory");
      if (there) return true;
    }
    return false;
  }
};

}  // namespace
}  // namespace mpopt

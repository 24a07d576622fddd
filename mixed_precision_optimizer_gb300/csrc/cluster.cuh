// Thread-block clusters: the rank and size, the barrier, stores into another CTA's
// shared memory (mapa, st.shared::cluster), and mail: values that arrive there with
// an mbarrier that counts their bytes (st.async).  The cluster's barrier makes a
// CTA wait until its stores to global memory are done, a few microseconds under
// load; mail orders nothing but itself.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "mail.h"

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
__device__ __forceinline__ void store_peer(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// One mbarrier for each of two alternating places.  init() by one thread, a
// cluster_sync() of all before the first use; for message k (0, 1, 2, ...) one
// thread of each CTA calls expect(k, bytes) with what all CTAs send it, the
// senders send(), the readers wait(k).  A place is used again for message k + 2:
// who sends that has to have waited for message k + 1, and its readers to have
// read message k before they sent theirs (exchange_message in mail.h sees to both,
// where waits run out too).
struct Mailbox {
  uint64_t* bar;         // [2] in shared memory
  unsigned long long limit_ns = 2000000000ull;

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
  // Whether message k is there; a wait gives up after two seconds (limit_ns).
  __device__ __forceinline__ bool wait(int k) const {
    const uint32_t at = u32(bar + (k & 1)), parity = static_cast<uint32_t>(k >> 1) & 1u;
    if (there(at, parity)) return true;
    const unsigned long long t0 = nanoseconds();
    for (uint32_t i = 1;; ++i) {
      if (there(at, parity)) return true;
      if ((i & 63u) == 0 && nanoseconds() - t0 > limit_ns) return false;
    }
  }

 private:
  static __device__ __forceinline__ bool there(uint32_t at, uint32_t parity) {
    uint32_t yes;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(yes)
        : "r"(at), "r"(parity)
        : "memory");
    return yes != 0;
  }
  static __device__ __forceinline__ unsigned long long nanoseconds() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
  }
};

// Clusters of a kernel that the GPU holds at once (asked once for each device and
// size; smem: the most that the kernel is launched with).
constexpr int kMostClusterCtas = 8;
template <auto kKernel>
cudaError_t clusters_at_once(int cluster, int threads, size_t smem, int* clusters) {
  static thread_local int known_device = -1, known[kMostClusterCtas + 1];
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device != known_device) {
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    for (int& k : known) k = 0;
    known_device = device;
  }
  if (known[cluster] == 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg);
    if (e != cudaSuccess) return e;
    known[cluster] = n > 0 ? n : 1;
  }
  *clusters = known[cluster];
  return cudaSuccess;
}

}  // namespace
}  // namespace mpopt

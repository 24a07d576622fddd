// Self-test of the messages between the CTAs of a cluster (sm_103a): one of them is
// held back, so that a wait for it runs out.

#include "cluster.cuh"
#include "internal.h"

namespace mpopt {
namespace {

constexpr int kThreads = kMailSelftestThreads;
constexpr unsigned long long kShortLimitNs = 200000000ull;

__global__ void __launch_bounds__(kThreads) mail_selftest_kernel(float* sums, int ctas, int messages, int held_back) {
  __shared__ float2 inbox[2][kMostClusterCtas][kThreads];
  __shared__ uint64_t bars[2];
  const int t = threadIdx.x, rank = static_cast<int>(cluster_rank());
  const Mailbox mail{bars, kShortLimitNs};
  if (t == 0) mail.init();
  cluster_sync();
  int lost_at = kNoneLost;
  for (int k = 0; k < messages; ++k) {
    float2(&in)[kMostClusterCtas][kThreads] = inbox[k & 1];
    const bool there = exchange_message(mail, k, t == 0, static_cast<uint32_t>(ctas * kThreads) * 8, lost_at, [&] {
      for (int i = 0; i < ctas; ++i)
        if (!(k == held_back && rank == ctas - 1 && t == 0 && i == 0))
          mail.send(k, &in[rank][t], i, make_float2(static_cast<float>(k), static_cast<float>(rank * kThreads + t)));
    });
    float sum = 0.f;
    for (int i = 0; i < ctas; ++i) sum += 1000.f * in[i][t].x + in[i][t].y;
    sums[(rank * messages + k) * kThreads + t] = there ? sum : __uint_as_float(0x7fc00000u);
  }
  cluster_sync();
  leave_mail(mail, lost_at);
}

}  // namespace

cudaError_t launch_mail_selftest(float* sums, int ctas, int messages, int held_back, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mail_selftest_kernel, sums, ctas, messages, held_back);
}

}  // namespace mpopt

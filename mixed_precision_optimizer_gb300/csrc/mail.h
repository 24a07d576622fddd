// A part in messages that every one of several threads (or warps) of a cluster sends
// to every CTA, numbered 0, 1, 2, ..., over a Mail (Mailbox in cluster.cuh) whose two
// places alternate.  Plain C++ as well as device code.
//
// Whoever has not received a message in time takes part in no later one.  So nobody
// receives the next one either, since its bytes do not arrive in full, and each place
// holds one message at a time whatever is late:  message k + 2 is sent by those who
// have received k + 1 in full, to which everyone belongs who has received k.  What is
// received is therefore what was sent as that message, and after a loss nothing is.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MPOPT_MAIL __device__ __forceinline__
#else
#define MPOPT_MAIL inline
#endif

namespace mpopt {
namespace {

constexpr int kNoneLost = -1;

// Message k; `counts`: this thread expects its CTA's `bytes`; send() sends this part's.
// lost_at: kNoneLost, or the message that has not come.  Whether message k is there.
template <typename Mail, typename Send>
MPOPT_MAIL bool exchange_message(const Mail& mail, int k, bool counts, uint32_t bytes, int& lost_at, Send&& send) {
  if (lost_at != kNoneLost) return false;
  if (counts) mail.expect(k, bytes);
  send();
  if (mail.wait(k)) return true;
  lost_at = k;
  return false;
}

// Behind the last message and a barrier of the cluster, behind which nothing is sent:
// mail that was late may still be on its way here.
template <typename Mail>
MPOPT_MAIL void leave_mail(const Mail& mail, int lost_at) {
  if (lost_at != kNoneLost) mail.wait(lost_at);
}

}  // namespace
}  // namespace mpopt

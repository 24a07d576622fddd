// The messages between the CTAs of a cluster on the host: the rule of mail.h over a model
// of the mbarriers, a thread for each part that sends and waits.  A barrier counts the
// bytes that are still to come and one arrival, and begins its next phase when both are
// there, as the hardware's does; a wait asks for a phase's parity.
//   mail_model CTAS THREADS MESSAGES LIMIT_MS LATE_CTA LATE_MESSAGE DELIVERY
// The last thread of LATE_CTA (-1: none) comes to LATE_MESSAGE only when another part has
// given up on it; with DELIVERY its part of that message to CTA 0 arrives when every
// part has come to the last barrier.  Prints what each part received, as far as it came.
// Ends with 1 if a part took anything for a message that was not sent as that one, or
// a CTA left before mail to it had arrived.
#include <atomic>
#include <barrier>
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <memory>
#include <mutex>
#include <thread>
#include <vector>

#include "../mixed_precision_optimizer_gb300/csrc/mail.h"

using namespace std::chrono;

struct Bar {
  int pending = 1, phase = 0;
  long bytes = 0;
  void look() {
    if (pending == 0 && bytes == 0) ++phase, pending = 1;
  }
};

struct Cta {
  Bar bar[2];
  std::vector<int> inbox[2];
  int inside = 0;                    // its threads
};

struct Cluster {
  std::mutex m;
  std::condition_variable moved;
  std::vector<Cta> ctas;
  int threads, limit_ms;
  std::atomic<bool> gave_up{false}, wrong{false};
};

struct Mail {
  Cluster* c;
  int rank;
  void expect(int k, uint32_t bytes) const {
    std::lock_guard<std::mutex> l(c->m);
    Bar& b = c->ctas[rank].bar[k & 1];
    --b.pending;
    b.bytes += bytes;
    b.look();
    c->moved.notify_all();
  }
  void deliver(int k, int part, int to) const {
    std::lock_guard<std::mutex> l(c->m);
    Cta& t = c->ctas[to];
    if (t.inside == 0) c->wrong = true, std::puts("mail to a CTA that has left");
    t.inbox[k & 1][part] = k;
    t.bar[k & 1].bytes -= 8;
    t.bar[k & 1].look();
    c->moved.notify_all();
  }
  bool wait(int k) const {
    std::unique_lock<std::mutex> l(c->m);
    const bool there = c->moved.wait_for(l, milliseconds(c->limit_ms),
                                         [&] { return (c->ctas[rank].bar[k & 1].phase & 1) != ((k >> 1) & 1); });
    if (!there) c->gave_up = true;
    return there;
  }
};

// What the kernels did before: a part that has lost a message expects and sends all the same.
template <typename M, typename Send>
bool exchange_anyway(const M& mail, int k, bool counts, uint32_t bytes, int& lost_at, Send&& send) {
  if (counts) mail.expect(k, bytes);
  send();
  if (lost_at == mpopt::kNoneLost && !mail.wait(k)) lost_at = k;
  return lost_at == mpopt::kNoneLost;
}

int main(int argc, char** argv) {
  if (argc != 8) return 2;
  const int ctas = atoi(argv[1]), threads = atoi(argv[2]), messages = atoi(argv[3]), late_cta = atoi(argv[5]),
            late_message = atoi(argv[6]);
  const bool delivery = atoi(argv[7]) != 0;
  Cluster c;
  c.threads = threads;
  c.limit_ms = atoi(argv[4]);
  c.ctas.resize(ctas);
  for (Cta& t : c.ctas) {
    t.inside = threads;
    for (auto& in : t.inbox) in.assign(ctas * threads, -1);
  }
  std::barrier last(ctas * threads);
  std::vector<int> came(ctas * threads, 0);
  auto part = [&](int rank, int t) {
    const Mail mail{&c, rank};
    const int id = rank * threads + t;
    const bool late = rank == late_cta && t == threads - 1;
    bool held = false;
    int lost_at = mpopt::kNoneLost;
    for (int k = 0; k < messages; ++k) {
      if (late && k == late_message && !delivery) {
        for (int i = 0; i < 1000 && !c.gave_up; ++i) std::this_thread::sleep_for(milliseconds(10));
        std::this_thread::sleep_for(milliseconds(c.limit_ms / 2));       // the others go on as far as they do
      }
      auto send = [&] {
        for (int to = 0; to < ctas; ++to) {
          if (late && k == late_message && delivery && to == 0) held = true;
          else mail.deliver(k, id, to);
        }
      };
#ifdef PLANTED
      const bool there = exchange_anyway(mail, k, t == 0, 8u * ctas * threads, lost_at, send);
#else
      const bool there = mpopt::exchange_message(mail, k, t == 0, 8u * ctas * threads, lost_at, send);
#endif
      if (there) {
        std::lock_guard<std::mutex> l(c.m);
        for (int v : c.ctas[rank].inbox[k & 1])
          if (v != k) c.wrong = true, std::printf("CTA %d took message %d for %d\n", rank, v, k);
        came[id] = k + 1;
      }
    }
    last.arrive_and_wait();
    if (held) mail.deliver(late_message, id, 0);
    if (!(held && rank == 0)) {
#ifndef PLANTED
      mpopt::leave_mail(mail, lost_at);
#endif
    }
    std::lock_guard<std::mutex> l(c.m);
    --c.ctas[rank].inside;
  };
  std::vector<std::thread> all;
  for (int r = 0; r < ctas; ++r)
    for (int t = 0; t < threads; ++t) all.emplace_back(part, r, t);
  for (auto& t : all) t.join();
  for (int id = 0; id < ctas * threads; ++id) std::printf("%d ", came[id]);
  std::puts("");
  return c.wrong ? 1 : 0;
}

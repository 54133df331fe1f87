// CPU check of the product kernels' bounded wait
// (cluster_distributed_shared_gb300/csrc/bounded_wait.h), driven with made-up
// clocks.  Prints "ok" and exits 0 when every check holds.
#include <stdio.h>

#include "bounded_wait.h"

using namespace dsmh;

static int failures = 0;

#define CHECK(cond)                                              \
  do {                                                           \
    if (!(cond)) {                                               \
      printf("FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond);     \
      ++failures;                                                \
    }                                                            \
  } while (0)

// A thread for which every step (a probe, a look at the flag, a reading of
// the clock) takes one unit, but which is switched out for `away` units after
// step `out`.  The awaited arrival is at time `at`.
struct Thread {
  long long now = 0, out, away, at;
  int steps = 0;
  bool seen_late = false;  // a probe was made after the limit and failed
  Thread(long long out_, long long away_, long long at_) : out(out_), away(away_), at(at_) {}
  void step() {
    ++now;
    if (++steps == out) now += away;
  }
  Waited wait(long long limit, long long flag_at = 1LL << 60) {
    const long long end = now + limit;
    return bounded_wait(
        [&] {
          const bool here = now >= at;
          if (!here && now >= end) seen_late = true;
          step();
          return here;
        },
        [&] {
          const bool set = now >= flag_at;
          step();
          return set;
        },
        [&] {
          const long long t = now;
          step();
          return t;
        },
        limit);
  }
};

int main() {
  // Nothing in the way: arrivals within the limit are seen, the limit ends
  // the wait, and soon after it.
  for (long long at = 0; at < 90; ++at) CHECK(Thread(0, 0, at).wait(100) == Waited::kArrived);
  {
    Thread t(0, 0, 1LL << 50);
    CHECK(t.wait(100) == Waited::kGaveUp);
    CHECK(t.now < 120);
  }
  // Another wait that gave up ends it.
  CHECK(Thread(0, 0, 1LL << 50).wait(1000000, 50) == Waited::kLeft);
  // Switched out, after any step, for longer than the limit, while the
  // arrival comes in: it is seen.
  for (int out = 1; out < 40; ++out)
    for (long long at = 60; at < 5000; at += 61) CHECK(Thread(out, 10000, at).wait(100) == Waited::kArrived);
  // Whenever it gives up, a probe after the limit has failed.
  for (int out = 0; out < 200; ++out) {
    Thread t(out, 10000, 1LL << 50);
    CHECK(t.wait(100) == Waited::kGaveUp);
    CHECK(t.seen_late);
  }
  if (failures == 0) printf("ok\n");
  return failures != 0;
}

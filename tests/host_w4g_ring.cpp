// Host program for tests/test_w4g_ring_host.py: one ring of the integer 4-bit
// projection kernels (csrc/w4g_ring.h) with its loader, its reader and copies
// that land late, stepped in a random order.  The reader's wait can run out at
// a given use.  Counts what must never happen: a `full` or `empty` barrier
// that gets more arrivals than its phase has room for, a copy into a slot that
// is still being read or written, and a copy in flight when the loader ends.
#include <cstdint>
#include <cstdlib>
#include <random>
#include <vector>

#include "w4g_ring.h"

namespace {

// An mbarrier of one arrival per phase, and the copies its phase waits for.
struct Barrier {
  uint32_t phase = 0;  // completed phases
  int pending = 1, copies = 0;
  long overruns = 0;
  bool done(uint32_t parity) const { return (phase & 1u) != parity; }
  void settle() {
    if (pending == 0 && copies == 0) {
      ++phase;
      pending = 1;
    }
  }
  void arrive(int with_copies) {
    if (pending == 0) {
      ++overruns;
      return;
    }
    pending = 0;
    copies += with_copies;
    settle();
  }
  void land() {
    --copies;
    settle();
  }
};

}  // namespace

// uses: copies that the work needs; give_up: the use whose wait runs out (at
// or past `uses`: none).  drain: the loader waits for its copies at the end 0: if
// a wait of its own ran out, 1: always, 2: once the reader is done, if any ran
// out.  keep_releasing: so does a reader that gave up.  Out: barrier overruns, copies issued into a
// slot that has one in flight, copies in flight at the end, uses read in order.
extern "C" void run_ring(int uses, int slots, int give_up, unsigned seed, int drain, int keep_releasing,
                         long* out) {
  std::mt19937 rng(seed);
  std::vector<Barrier> full(slots), empty(slots);
  std::vector<int> flying(slots, 0);
  std::vector<int> queue;  // slots of the copies in flight
  long onto = 0, read = 0;
  bool abort_flag = false, dead = false, loader_ok = true;
  int issued = 0, taken = 0;
  auto land_one = [&] {
    if (queue.empty()) return;
    const size_t i = rng() % queue.size();
    const int s = queue[i];
    queue.erase(queue.begin() + (long)i);
    --flying[s];
    full[s].land();
  };
  bool loading = true;
  while (loading || taken < uses) {
    switch (rng() % 3) {
      case 0:
        if (!loading) break;
        if (issued == uses) {
          loading = false;
          break;
        }
        if (empty[issued % slots].done(((uint32_t)(issued / slots) & 1u) ^ 1u)) {
          const int s = issued % slots;
          onto += flying[s] != 0;
          full[s].arrive(1);
          ++flying[s];
          queue.push_back(s);
          ++issued;
        } else if (abort_flag) {
          loader_ok = false;
          loading = false;
        }
        break;
      case 1:
        if (taken == uses) break;
        if (!dead) {
          const int s = taken % slots;
          if (taken >= give_up) {  // its wait ran out
            dead = abort_flag = true;
          } else if (full[s].done((uint32_t)(taken / slots) & 1u)) {
            ++read;
          } else {
            break;
          }
        }
        if (keep_releasing || !dead) empty[taken % slots].arrive(0);
        ++taken;
        break;
      default:
        land_one();
    }
  }
  if (drain == 1 || (drain == 2 ? abort_flag : !loader_ok))
    bsr::drain_ring((uint32_t)issued, (uint32_t)slots, [&](uint32_t s, uint32_t parity) {
      for (int i = 0; i < 1000 && !full[s].done(parity); ++i) land_one();
      return full[s].done(parity);
    });
  out[0] = 0;
  for (int s = 0; s < slots; ++s) out[0] += full[s].overruns + empty[s].overruns;
  out[1] = onto;
  out[2] = (long)queue.size();
  out[3] = read;
}

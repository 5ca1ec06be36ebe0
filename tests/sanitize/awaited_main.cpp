// Walks a warp's loads on one barrier (cp_ring.h, Awaited) to every point where a wait may run out, with
// the load landing before or after the kernel's last wait, and checks that this last wait is answered by
// the load's own phase and by no other.  Built and run by tests/test_awaited.py.
#include <cstdint>
#include <cstdio>

#include "cp_ring.h"

// A barrier of one arrival and the bytes it announces: a phase is over when its load has landed.
struct Barrier {
  uint32_t over = 0;
  void land() { ++over; }
  // What a wait on a parity is told: whether the phase of that parity, the running one or the one
  // before it, is over.
  bool answers(uint32_t parity) const { return (over & 1) != parity; }
};

int main() {
  int fails = 0;
  // `good` loads arrive in time; then one begins whose wait runs out (late), or nothing more does
  for (uint32_t good = 0; good <= 9; ++good)
    for (int late = 0; late < 2; ++late) {
      Barrier b;
      cpl::Awaited a;
      for (uint32_t i = 0; i < good; ++i) {
        a.begun();
        if (!a.under_way || b.answers(a.parity)) ++fails;      // not yet: nothing has landed
        b.land();
        const bool arrived = b.answers(a.parity);
        if (!arrived) ++fails;
        a.waited(arrived);
        if (a.under_way) ++fails;
      }
      if (late == 0) continue;
      a.begun();
      a.waited(b.answers(a.parity));                           // ran out
      if (!a.under_way) ++fails;                               // the end waits for it,
      if (b.answers(a.parity)) ++fails;                        // not for the phase before,
      b.land();
      if (!b.answers(a.parity)) ++fails;                       // and is answered when it lands
    }
  if (fails) {
    std::fprintf(stderr, "%d checks failed\n", fails);
    return 1;
  }
  std::printf("awaited ok\n");
  return 0;
}

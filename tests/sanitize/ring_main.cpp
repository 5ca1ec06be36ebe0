// Walks two issuers of loads through a ring of stages (cp_ring.h) to every point where they may stop,
// and checks that what an ending kernel waits for covers every load begun, and that no parity can
// stand for an earlier phase.  Built and run by tests/test_ring.py.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "cp_ring.h"

int main() {
  int fails = 0;
  for (uint32_t stages = 1; stages <= 8; ++stages)
    for (uint32_t used = 0; used <= 3 * stages; ++used)           // fills that the products used up
      for (uint32_t a = used; a <= used + stages; ++a)            // each issuer: up to a ring ahead
        for (uint32_t b = used; b <= used + stages; ++b) {
          // per stage: fills by each issuer, counted one by one
          std::vector<uint32_t> fa(stages), fb(stages);
          for (uint32_t i = 0; i < a; ++i) ++fa[i % stages];
          for (uint32_t i = 0; i < b; ++i) ++fb[i % stages];
          for (uint32_t k = 0; k < stages; ++k) {
            if (cpl::ring_fills(a, stages, k) != fa[k]) ++fails;
            const uint32_t most = fa[k] > fb[k] ? fa[k] : fb[k], least = fa[k] + fb[k] - most;
            const cpl::LastFill last = cpl::last_fill(a, b, stages, k);
            if (last.any != (most != 0)) ++fails;
            if (!last.any) continue;
            // the phase waited for is the last that anyone began; all in front of it are complete
            // (both issuers' fills), so its parity cannot be answered by an older phase
            if (last.parity != ((most - 1) & 1)) ++fails;
            if (least + 1 < most) ++fails;
          }
        }
  if (fails) {
    std::fprintf(stderr, "%d checks failed\n", fails);
    return 1;
  }
  std::printf("ring ok\n");
  return 0;
}

// Which rows count as lying on 32-byte boundaries (cp_geometry.h, sectors_ok).  Built and run by
// tests/test_sectors.py.
#include <cstdint>
#include <cstdio>

#include "cp_geometry.h"

int main() {
  int fails = 0;
  alignas(64) static uint8_t at[128];
  for (uint64_t elt = 2; elt <= 4; elt += 2)
    for (uint64_t stride = 0; stride <= 64; ++stride) {
      const bool whole = stride * elt % 32 == 0;
      if (cpx::sectors_ok(at, stride, elt) != whole) ++fails;
      if (cpx::sectors_ok(at + 16, stride, elt)) ++fails;
      if (!cpx::sectors_ok(nullptr, stride, elt)) ++fails;   // an array that is not there
    }
  if (fails) {
    std::fprintf(stderr, "%d checks failed\n", fails);
    return 1;
  }
  std::printf("sectors ok\n");
  return 0;
}

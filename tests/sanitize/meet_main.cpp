// Whether two arrays of rows share a byte (cp_geometry.h, rows_meet), against counting the bytes.  Built
// and run by tests/test_rows_meet.py.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "cp_geometry.h"

static bool counted(const cpx::RowBytes& a, const cpx::RowBytes& b, const uint8_t* base) {
  std::vector<int> seen(4096);
  for (uint64_t r = 0; r < a.rows; ++r)
    for (uint64_t c = 0; c < a.width; ++c)
      seen[static_cast<const uint8_t*>(a.p) - base + r * a.stride + c] = 1;
  for (uint64_t r = 0; r < b.rows; ++r)
    for (uint64_t c = 0; c < b.width; ++c)
      if (seen[static_cast<const uint8_t*>(b.p) - base + r * b.stride + c]) return true;
  return false;
}

int main() {
  static uint8_t base[4096];
  uint32_t x = 12345, fails = 0, met = 0, apart = 0;
  auto next = [&](uint32_t n) {
    x = x * 1664525u + 1013904223u;
    return (x >> 8) % n;
  };
  for (int i = 0; i < 400000; ++i) {
    cpx::RowBytes a{base + 600 + next(200), 1 + next(40), 0, next(6)};
    cpx::RowBytes b{base + 600 + next(200), a.stride, 0, next(6)};
    a.width = next(static_cast<uint32_t>(a.stride) + 1);
    b.width = next(static_cast<uint32_t>(b.stride) + 1);
    if (next(8) == 0) a.stride = 0;                        // one row for all
    if (next(8) == 0) a.rows = 1, a.stride = a.width + next(9), a.width = 1 + next(120);
    if (next(8) == 0) b.rows = 1, b.stride = next(5), b.width = 1 + next(120);
    const bool want = counted(a, b, base);
    (want ? met : apart) += 1;
    if (cpx::rows_meet(a, b) != want || cpx::rows_meet(b, a) != want) ++fails;
    if (cpx::rows_clash(a, a) || (cpx::rows_clash(a, b) && !want)) ++fails;
  }
  // other strides are not looked into, arrays that are not there or far away meet nothing
  if (cpx::rows_meet({nullptr, 8, 8, 3}, {base, 8, 8, 3})) ++fails;
  if (cpx::rows_meet({base, 8, 8, 3}, {base + 24, 16, 8, 3})) ++fails;
  if (fails || met < 10000 || apart < 10000) {
    std::fprintf(stderr, "%u checks failed, %u met, %u apart\n", fails, met, apart);
    return 1;
  }
  std::printf("meet ok\n");
  return 0;
}

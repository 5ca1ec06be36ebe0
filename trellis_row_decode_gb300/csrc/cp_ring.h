// cp_ring.h -- arithmetic of a ring of stages that loads fill in turn (plain C++: the product's
// kernels and the CPU tests share it).
#pragma once

#include <cstdint>

namespace cpl {

// How often stage `k` has been filled after `fills` loads went round a ring of `stages`.
constexpr uint32_t ring_fills(uint32_t fills, uint32_t stages, uint32_t k) {
  return fills / stages + (k < fills % stages ? 1 : 0);
}

// What a kernel that ends early waits for at stage `k`, before its shared memory is someone
// else's: the last fill that either of two issuers began (`mine`, `other`: their loads so far; an
// issuer alone gives its count twice).  `parity` is that of the fill's barrier phase.  An issuer
// is at most one fill of a stage ahead of the other (a stage is filled again once both fills of it
// are used up), so the phases in front of it are complete and the parity names no other phase.
struct LastFill {
  bool any;
  uint32_t parity;
};
constexpr LastFill last_fill(uint32_t mine, uint32_t other, uint32_t stages, uint32_t k) {
  const uint32_t n = ring_fills(mine > other ? mine : other, stages, k);
  return LastFill{n != 0, (n - 1) & 1};
}

}  // namespace cpl

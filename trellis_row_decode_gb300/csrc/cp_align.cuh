// cp_align.cuh -- rows on any byte boundary copied to rows on 16-byte ones, which tensor maps want
// (the products of 8 and of 16 bits): what the copying kernels share.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "cp_matmul_fp8.h"

namespace cpm {

// Sixteen bytes from row + col on, zeros behind the row's k bytes: shifted out of two aligned
// pieces, or byte by byte where those reach outside the row.
__device__ __forceinline__ uint4 load_any_piece(const uint8_t* row, uint32_t col, uint32_t k) {
  const uint8_t* p = row + col;
  const uint32_t skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15);
  if (col >= skew && static_cast<uint64_t>(col) + (skew != 0 ? 32 - skew : 16) <= k) {
    const uint4* q = reinterpret_cast<const uint4*>(p - skew);
    const uint4 lo = q[0], hi = skew != 0 ? q[1] : make_uint4(0, 0, 0, 0);
    uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (skew & 8) {
#pragma unroll
      for (int i = 0; i < 6; ++i) x[i] = x[i + 2];
    }
    if (skew & 4) {
#pragma unroll
      for (int i = 0; i < 5; ++i) x[i] = x[i + 1];
    }
    const uint32_t bits = 8 * (skew & 3);
    return make_uint4(__funnelshift_r(x[0], x[1], bits), __funnelshift_r(x[1], x[2], bits),
                      __funnelshift_r(x[2], x[3], bits), __funnelshift_r(x[3], x[4], bits));
  }
  uint32_t w[4] = {};
#pragma unroll
  for (int b = 0; b < 16; ++b)
    if (static_cast<uint64_t>(col) + b < k) w[b / 4] |= static_cast<uint32_t>(p[b]) << (8 * (b & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kAlignThreads = 256;
constexpr uint64_t kAlignCtas = 152 * 6;                  // as many as run at once
constexpr uint32_t kAlignPieces = 4;                      // 16-byte pieces of a lane
constexpr uint32_t kAlignBytes = 32 * 16 * kAlignPieces;  // of a row, by one warp at a time

struct AlignParams {
  AlignOperand of[2];
  uint32_t k, chunks;      // chunks of kAlignBytes in a row
  uint64_t pitch;
};

// CTA `cta` of `ctas` of kAlignThreads.
__device__ __forceinline__ void align_rows_of(const AlignParams& p, uint32_t cta, uint32_t ctas) {
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t warps = static_cast<uint64_t>(ctas) * (kAlignThreads / 32);
  const uint64_t units = (p.of[0].rows + p.of[1].rows) * p.chunks;
  for (uint64_t u = static_cast<uint64_t>(cta) * (kAlignThreads / 32) + threadIdx.x / 32;
       u < units; u += warps) {
    uint64_t row = u / p.chunks;
    const uint32_t col = static_cast<uint32_t>(u - row * p.chunks) * kAlignBytes + lane * 16;
    const bool second = row >= p.of[0].rows;
    if (second) row -= p.of[0].rows;
    const uint8_t* from = (second ? p.of[1].from : p.of[0].from) +
                          row * (second ? p.of[1].ld : p.of[0].ld);
    uint8_t* to = (second ? p.of[1].to : p.of[0].to) + row * p.pitch;
    uint4 v[kAlignPieces];
#pragma unroll
    for (uint32_t i = 0; i < kAlignPieces; ++i)
      if (col + i * 512 < p.k) v[i] = load_any_piece(from, col + i * 512, p.k);
#pragma unroll
    for (uint32_t i = 0; i < kAlignPieces; ++i)
      if (col + i * 512 < p.k) *reinterpret_cast<uint4*>(to + col + i * 512) = v[i];
  }
}

inline uint64_t aligned_pitch(uint64_t k) { return (k + 15) / 16 * 16; }

inline AlignParams align_params(const AlignOperand (&of)[2], uint32_t k, uint64_t pitch) {
  return AlignParams{{of[0], of[1]}, k, (k + kAlignBytes - 1) / kAlignBytes, pitch};
}
inline uint32_t align_ctas(const AlignParams& p) {
  const uint64_t units = (p.of[0].rows + p.of[1].rows) * p.chunks;
  const uint64_t ctas = (units + kAlignThreads / 32 - 1) / (kAlignThreads / 32);
  return static_cast<uint32_t>(ctas < kAlignCtas ? ctas : kAlignCtas);
}

}  // namespace cpm

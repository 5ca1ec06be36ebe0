// cp_matmul_tc.cu -- cp_matmul_fp8 on tensor memory (tcgen05), for operands whose rows lie on
// 16-byte boundaries (include/cp.h).
//
//   out[i][j] = sum over g of sa[i][g] sw[j / 128][g] * (a[i] . w[j] over group g)
#include <atomic>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "cp.h"
#include "cp_internal.h"
#include "cp_layer.cuh"
#include "cp_matmul_fp8.h"
#include "cp_ring.h"
#include "cp_tcgen05.cuh"

namespace {

using namespace cpl;
using cpm::MatmulParams;

// ------------------------------------------------- rows on 16-byte boundaries: tcgen05
//
// A pair of CTAs (two SMs) makes 256 x bn outputs, bn a multiple of 32 up to 256.  Each
// CTA stages its 128 rows of a and its half of the bn rows of w (128 bytes of k a stage,
// 128-byte swizzle), so a byte that enters an SM feeds both tensor cores.  Roles: one
// thread per CTA issues the TMA loads; one thread of the first CTA issues four
// tcgen05.mma (k = 32 each) per group of 128 into one of two tensor-memory buffers; eight
// warps per CTA read the other buffer, scale it and add it to their registers (a lane has
// a row, a warp half of the columns).  The scales differ from group to group, so the
// running sum cannot stay in tensor memory; the two buffers let the tensor core work on
// the next group meanwhile.  With few tiles, `splits` pairs of one cluster share a tile's
// groups and add their sums, in the order of the pairs, through distributed shared memory.
//
// 4096 x 4096 x 24576: 340-348 us in bursts of a dozen (2.4 PFLOP/s), 364-376 in calls that go on
// (2.2, at the power limit).  Bound by the summing warps:
// the tensor core alone takes 225 us (263 sustained, at the power limit), with the loads of
// tensor memory 250, with the fused multiply-adds 334 (224 of them an SM partition and group,
// issued at 0.8 a clock), with the loads of the scales 348.  2048^3: 14.0 us, 64 tiles of 16 groups
// in one turn, of which about 6 us are the start, the first loads and the outputs.

constexpr int kSumWarps = 8;
constexpr int kTcThreads = (kSumWarps + 4) * 32;       // + the TMA warp, the MMA warp and two idle
// Registers: launched with 168 a thread (65,536 over 12 warps); the summing warps (128 sums and 64
// values in flight a thread) take what the other four give up.
constexpr int kLaunchRegs = 168, kSumRegs = 208, kOtherRegs = 88;
static_assert(2 * kSumRegs + kOtherRegs <= 3 * kLaunchRegs, "a warpgroup's share of the launch");
constexpr uint32_t kMaxStages = 8;
constexpr uint32_t kTileA = 128 * 128;                 // bytes of a's rows per stage and CTA
constexpr uint32_t kSmemMost = 224 * 1024;             // dynamic shared memory of a CTA

// A wait that ran out sets this word; cp_matmul_fp8_status reads and clears it.
__device__ uint32_t g_matmul_gave_up;

struct TcParams {
  const float* sa;
  const float* sw;
  void* out;
  uint64_t ldo;
  uint32_t m, n, groups;
  int out_dtype;
  uint32_t tiles_m, tiles, stages, splits, tmem_columns;
  uint32_t out_align;       // 32, 16 or 0: bytes on whose boundaries out's rows lie
};

// Eight consecutive outputs of a row.
__device__ __forceinline__ void store8(const TcParams& p, uint32_t row, uint32_t col,
                                       const float* v) {
  const uint64_t at = static_cast<uint64_t>(row) * p.ldo + col;
  if (p.out_align >= 16 && col + 8 <= p.n) {
    if (p.out_dtype == CP_F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = v[e];
      if (p.out_dtype == CP_F16) store_octet(static_cast<__half*>(p.out) + at, pack<__half>(u));
      else store_octet(static_cast<__nv_bfloat16*>(p.out) + at, pack<__nv_bfloat16>(u));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < p.n) store_from_f32(p.out, at + e, p.out_dtype, v[e]);
  }
}

// Sixteen, whole 32-byte sectors of L2 where the rows allow it: a lane's outputs are its own
// row's, so only whole sectors keep the writes from being merged in L2.
__device__ __forceinline__ void store16(const TcParams& p, uint32_t row, uint32_t col,
                                        const float* v) {
  if (p.out_dtype != CP_F32 && p.out_align >= 32 && col + 16 <= p.n) {
    Packed<float> r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = v[8 * h + e];
      if (p.out_dtype == CP_F16) {
        const Packed<__half> x = pack<__half>(u);
#pragma unroll
        for (int e = 0; e < 4; ++e) r.w[4 * h + e] = x.w[e];
      } else {
        const Packed<__nv_bfloat16> x = pack<__nv_bfloat16>(u);
#pragma unroll
        for (int e = 0; e < 4; ++e) r.w[4 * h + e] = x.w[e];
      }
    }
    store_octet(reinterpret_cast<float*>(static_cast<uint16_t*>(p.out) +
                                         static_cast<uint64_t>(row) * p.ldo + col), r);
  } else {
    store8(p, row, col, v);
    store8(p, row, col + 8, v + 8);
  }
}

// Columns col to end, 32 at most, of the warp's 32 rows, where out's rows lie on no useful
// boundary: transposed by five exchanges between lanes, so that each store writes 32 consecutive outputs of one row
// (3000 x 700 x 900: 15.8 us, by each lane's single outputs of its own row 31.1; 3393 x 3777 x 384
// in fp32: 40 against 83).
__device__ __forceinline__ void store_transposed(const TcParams& p, uint32_t row0, uint32_t col,
                                                 uint32_t end, uint32_t lane, float (&x)[32]) {
#pragma unroll
  for (uint32_t s = 16; s > 0; s /= 2) {
    const bool high = (lane & s) != 0;
#pragma unroll
    for (uint32_t i = 0; i < 32; ++i) {
      if ((i & s) == 0) {
        const float got = __shfl_xor_sync(0xFFFFFFFFu, high ? x[i] : x[i + s], s);
        x[i] = high ? got : x[i];
        x[i + s] = high ? x[i + s] : got;
      }
    }
  }
  if (col + lane < end) {
    const uint32_t rows = min(p.m - row0, 32u);
    const uint64_t at = static_cast<uint64_t>(row0) * p.ldo + col + lane;
#pragma unroll
    for (uint32_t r = 0; r < 32; ++r)
      if (r < rows) store_from_f32(p.out, at + r * p.ldo, p.out_dtype, x[r]);
  }
}

// f(std::integral_constant) for 0 .. kCount - 1.
template <uint32_t kCount, typename F, uint32_t kFrom = 0>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (kFrom < kCount) {
    f(std::integral_constant<uint32_t, kFrom>{});
    static_for<kCount, F, kFrom + 1>(static_cast<F&&>(f));
  }
}

// Up to 32 columns of a warp's share of 8 * kEights, from column 32 * kChunk on.
template <uint32_t kEights, uint32_t kChunk>
__device__ __forceinline__ void load_chunk(float (&x)[32], uint32_t at) {
  constexpr uint32_t kLeft = kEights - 4 * kChunk;
  if constexpr (kLeft >= 4) {
    cpt::tmem_load32<0>(x, at + 32 * kChunk);
  } else {
    if constexpr ((kLeft & 2) != 0) cpt::tmem_load16<0>(x, at + 32 * kChunk);
    if constexpr ((kLeft & 1) != 0)
      cpt::tmem_load8<(kLeft & 2) * 8>(x, at + 32 * kChunk + (kLeft & 2) * 8);
  }
}

// acc += x * scale over those columns; those from `turn` eights on have the second scale.
template <uint32_t kEights, uint32_t kChunk>
__device__ __forceinline__ void add_chunk(float (&acc)[kEights * 8], const float (&x)[32],
                                          uint32_t turn, float scale0, float scale1) {
  constexpr uint32_t kLeft = kEights - 4 * kChunk, kHere = kLeft < 4 ? kLeft : 4;
#pragma unroll
  for (uint32_t c = 0; c < kHere; ++c) {
    const float f = 4 * kChunk + c < turn ? scale0 : scale1;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
      acc[32 * kChunk + 8 * c + i] = fmaf(x[8 * c + i], f, acc[32 * kChunk + 8 * c + i]);
  }
}

template <uint32_t kEights>            // columns of a warp's share / 8 = kBn / 16
__global__ void __launch_bounds__(kTcThreads, 1)
    matmul_tc_kernel(const __grid_constant__ CUtensorMap map_a,
                     const __grid_constant__ CUtensorMap map_w, const TcParams p) {
  constexpr uint32_t kBn = kEights * 16, kShare = kEights * 8;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 5];
  __shared__ uint32_t tmem_base;
  __shared__ uint32_t issued;              // this CTA's fills of stages
  __shared__ int gave_up;
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cpt::cluster_rank();
  const uint32_t half = rank & 1, split = rank >> 1, first = rank & ~1u;
  const uint32_t stage_bytes = kTileA + kBn * 64;
  const uint32_t full = cpt::smem_addr(bars), empty = full + 8 * kMaxStages;
  const uint32_t acc_full = empty + 8 * kMaxStages, acc_empty = acc_full + 16;
  const uint32_t drained = acc_empty + 16;
  // the first CTA's barriers hold the pair's loads and reads
  const uint32_t pair_full = cpt::map_rank(full, first);
  const uint32_t pair_acc_empty = cpt::map_rank(acc_empty, first);

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < p.stages; ++s) {
      cpt::mbar_init(full + 8 * s, 1);
      cpt::mbar_init(empty + 8 * s, 1);
    }
    for (uint32_t b = 0; b < 2; ++b) {
      cpt::mbar_init(acc_full + 8 * b, 1);
      cpt::mbar_init(acc_empty + 8 * b, 2 * kSumWarps);
    }
    cpt::mbar_init(drained, 1);
    cpt::mbar_init_fence();
    gave_up = 0;
  }
  if (warp == kSumWarps + 1) cpt::tmem_alloc_pair(cpt::smem_addr(&tmem_base), p.tmem_columns);
  cpt::tc_fence_before();
  __syncthreads();
  cpt::cluster_sync();
  cpt::tc_fence_after();
  wait_for_previous();          // (the set-up above runs while the kernel before this one ends)
  const uint32_t tmem = tmem_base;
  const uint32_t kb0 = static_cast<uint32_t>(static_cast<uint64_t>(p.groups) * split / p.splits);
  const uint32_t kb1 =
      static_cast<uint32_t>(static_cast<uint64_t>(p.groups) * (split + 1) / p.splits);
  const uint32_t step = gridDim.x / (2 * p.splits), tile0 = blockIdx.x / (2 * p.splits);
  // Every warp of the cluster comes here when its role ends.  If a wait of the pair's first CTA ran
  // out, whichever warp's, what the pair has in flight then ends before either CTA leaves its shared
  // and tensor memory (the second waits at the cluster's last barrier): loads up to the last fill
  // that either CTA began, all of which count on the first CTA's barriers, and every product
  // issued.  These waits have a limit too, one for each of the two warps that see to them; a fill
  // that only one CTA began runs it out, and has landed by then.  Where the first CTA has not given
  // up, its summing warps have seen every product done, so nothing is in flight.
  auto end_role = [&] {
    __syncwarp();
    cpt::tc_fence_before();
    asm volatile("barrier.sync 1, %0;" ::"n"(kTcThreads) : "memory");
    cpt::cluster_sync();
  };

  if (warp >= kSumWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // Both warps run their loops whole and elect a thread to issue.
    if (warp == kSumWarps) {
      // -------------------------------------------------------------- loads
      if (cpt::elect_one()) {
        cpt::tma_prefetch_map(&map_a);
        cpt::tma_prefetch_map(&map_w);
      }
      __syncwarp();
      const uint32_t w_bytes = kBn * 64;
      uint32_t s = 0, round = 0, fills = 0;
      bool ok = true;
      for (uint32_t tile = tile0; tile < p.tiles && ok; tile += step) {
        const uint32_t tile_n = tile / p.tiles_m;
        const uint32_t row0 = (tile - tile_n * p.tiles_m) * 256, col0 = tile_n * kBn;
        const bool a1 = row0 + 128 < p.m;               // the second CTA has rows of a
        const bool mine = half == 0 || a1;
        const uint32_t bytes = 2 * w_bytes + (a1 ? 2 : 1) * kTileA;
        for (uint32_t kb = kb0; kb < kb1; ++kb) {
          if (round > 0) {
            ok = cpt::mbar_wait(empty + 8 * s, (round - 1) & 1, &gave_up);
            if (!ok) break;
          }
          const uint32_t dst = cpt::smem_addr(tiles) + s * stage_bytes;
          if (cpt::elect_one()) {
            if (half == 0) cpt::mbar_expect(full + 8 * s, bytes);
            if (mine)
              cpt::tma_load_pair(dst, &map_a, kb * 128, row0 + half * 128, pair_full + 8 * s);
            cpt::tma_load_pair(dst + kTileA, &map_w, kb * 128, col0 + half * (kBn / 2),
                               pair_full + 8 * s);
          }
          __syncwarp();
          ++fills;
          if (++s == p.stages) {
            s = 0;
            ++round;
          }
        }
      }
      if (lane == 0) issued = fills;
      end_role();
      if (gave_up != 0 && half == 0) {
        const uint32_t other = cpt::load_cluster1(cpt::map_rank(cpt::smem_addr(&issued), rank + 1));
        int late = 0;
        for (uint32_t k = 0; k < p.stages; ++k) {
          const LastFill last = last_fill(fills, other, p.stages, k);
          if (last.any) cpt::mbar_wait(full + 8 * k, last.parity, &late);
        }
      }
    } else if (warp == kSumWarps + 1 && half == 0) {
      // ----------------------------------------------------------- products
      const uint32_t instr = cpt::e4m3_instr_desc(256, kBn);
      const uint16_t pair = static_cast<uint16_t>(3u << first);
      uint32_t it = 0, s = 0, round = 0;
      bool ok = true;
      for (uint32_t tile = tile0; tile < p.tiles && ok; tile += step) {
        for (uint32_t kb = kb0; kb < kb1; ++kb, ++it) {
          const uint32_t b = it & 1;
          ok = (it < 2 || cpt::mbar_wait(acc_empty + 8 * b, ((it >> 1) - 1) & 1, &gave_up)) &&
               cpt::mbar_wait(full + 8 * s, round & 1, &gave_up);
          if (!ok) break;
          cpt::tc_fence_after();
          const uint32_t at = cpt::smem_addr(tiles) + s * stage_bytes;
          const uint64_t da = cpt::operand_desc(at), dw = cpt::operand_desc(at + kTileA);
          if (cpt::elect_one()) {
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
              cpt::mma_pair(tmem + b * kBn, da + 2 * k, dw + 2 * k, instr, k != 0);
            cpt::mma_commit_pair(empty + 8 * s, pair);
            cpt::mma_commit_pair(acc_full + 8 * b, pair);
          }
          __syncwarp();
          if (++s == p.stages) {
            s = 0;
            ++round;
          }
        }
      }
      end_role();
      if (gave_up != 0) {
        int late = 0;
        if (cpt::elect_one()) cpt::mma_commit_pair(drained, static_cast<uint16_t>(1u << first));
        __syncwarp();
        cpt::mbar_wait(drained, 0, &late);
      }
    } else {
      end_role();
    }
  } else {
    // ----------------------------------------------------------------- sums
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    const uint32_t lanes = (warp & 3) * 32;              // tensor-memory lanes of this warp
    const uint32_t share = (warp >> 2) * kShare;         // its first column of the tile
    const uint32_t tmem_warp = tmem + (lanes << 16) + share;
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t tile = tile0; tile < p.tiles && ok; tile += step) {
      const uint32_t tile_n = tile / p.tiles_m;
      const uint32_t row0 = (tile - tile_n * p.tiles_m) * 256 + half * 128 + lanes;
      const uint32_t row = row0 + lane;
      const uint32_t col = tile_n * kBn + share;
      const bool any = row0 < p.m && col < p.n;          // the warp has outputs
      const uint32_t turn = (128 - col % 128) / 8;       // eights from here on are in the next block
      constexpr uint32_t kChunks = (kEights + 3) / 4;    // of 32 columns, the last may be shorter
      float acc[kShare];
#pragma unroll
      for (uint32_t i = 0; i < kShare; ++i) acc[i] = 0.0f;
      if (!any) {
        for (uint32_t kb = kb0; kb < kb1 && ok; ++kb, ++it) {
          ok = cpt::mbar_wait(acc_full + 8 * (it & 1), (it >> 1) & 1, &gave_up);
          if (ok && lane == 0) cpt::mbar_arrive_cluster(pair_acc_empty + 8 * (it & 1));
        }
      } else {
        // scales are loaded two groups ahead, each into the registers of its parity
        const float* sa = p.sa + static_cast<uint64_t>(min(row, p.m - 1)) * p.groups;
        const uint32_t last = (p.n + 127) / 128 - 1;
        const float* sw0 = p.sw + static_cast<uint64_t>(col / 128) * p.groups;
        const float* sw1 = p.sw + static_cast<uint64_t>(min(col / 128 + 1, last)) * p.groups;
        float fa[2] = {}, f0[2] = {}, f1[2] = {};
        auto load_scales = [&](uint32_t k, uint32_t kb) {
          if (kb < kb1) {
            fa[k] = sa[kb];
            f0[k] = sw0[kb];
            f1[k] = sw1[kb];
          }
        };
        load_scales(0, kb0);
        load_scales(1, kb0 + 1);
        float v[2][32];
        for (uint32_t kb = kb0; kb < kb1 && ok; kb += 2) {
#pragma unroll
          for (uint32_t k = 0; k < 2; ++k) {
            if (kb + k < kb1 && ok) {
              const uint32_t b = it & 1;
              const uint32_t at = tmem_warp + b * kBn;
              ok = cpt::mbar_wait(acc_full + 8 * b, (it >> 1) & 1, &gave_up);
              if (ok) {
                cpt::tc_fence_after();
                load_chunk<kEights, 0>(v[0], at);
                const float scale0 = fa[k] * f0[k], scale1 = fa[k] * f1[k];
                load_scales(k, kb + k + 2);
                static_for<kChunks>([&](auto chunk) {
                  constexpr uint32_t c = decltype(chunk)::value;
                  float(&x)[32] = v[c & 1];
                  cpt::tmem_load_wait(x);
                  if constexpr (c + 1 < kChunks) {
                    load_chunk<kEights, c + 1>(v[(c + 1) & 1], at);
                  } else {                // the buffer is read: the tensor core may have it back
                    cpt::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) cpt::mbar_arrive_cluster(pair_acc_empty + 8 * b);
                  }
                  add_chunk<kEights, c>(acc, x, turn, scale0, scale1);
                });
                ++it;
              }
            }
          }
        }
      }
      if (!ok) break;
      if (p.splits == 1) {
        if (any && p.out_align == 0) {
          static_for<kChunks>([&](auto chunk) {
            constexpr uint32_t c = decltype(chunk)::value;
            constexpr uint32_t kHere = kShare - 32 * c < 32 ? kShare - 32 * c : 32;
            float x[32];
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i)
              x[i] = i < kHere ? acc[32 * c + (i < kHere ? i : 0)] : 0.0f;
            const uint32_t from = col + 32 * c;
            if (from < p.n) store_transposed(p, row0, from, min(p.n, from + kHere), lane, x);
          });
        } else if (any && row < p.m) {
#pragma unroll
          for (uint32_t c = 0; c < kEights; c += 2)
            if (col + 8 * c < p.n) store16(p, row, col + 8 * c, acc + 8 * c);
        }
      } else if (any) {
        // this pair's sums, [row][kBn + 4] floats over the stages (all loads are used up)
        float* part = reinterpret_cast<float*>(tiles) + (lanes + lane) * (kBn + 4) + share;
#pragma unroll
        for (uint32_t i = 0; i < kEights * 2; ++i)
          *reinterpret_cast<float4*>(part + 4 * i) =
              make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
      }
    }
    if (!ok && lane == 0) atomicOr(&g_matmul_gave_up, 1u);
    end_role();
  }
  if (p.splits > 1 && gave_up == 0 && warp < kSumWarps) {
    // the pairs' sums, added in order: each pair takes a share of the tile's columns
    const uint32_t row0 = tile0 % p.tiles_m * 256 + half * 128, col0 = tile0 / p.tiles_m * kBn;
    const uint32_t rows = row0 < p.m ? min(128u, p.m - row0) : 0;
    const uint32_t c0 = kBn * split / p.splits, c1 = kBn * (split + 1) / p.splits;
    const uint32_t wide = c1 - c0, base = cpt::smem_addr(tiles);
    for (uint32_t i = threadIdx.x; i < rows * wide / 4; i += kSumWarps * 32) {
      const uint32_t r = i / (wide / 4), c = c0 + (i - r * (wide / 4)) * 4;
      if (col0 + c < p.n) {
        const uint32_t off = base + (r * (kBn + 4) + c) * 4;
        float4 v[4];
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q)
          if (q < p.splits) v[q] = cpt::load_cluster4(cpt::map_rank(off, 2 * q + half));
        float4 sum = v[0];
#pragma unroll
        for (uint32_t q = 1; q < 4; ++q) {
          if (q < p.splits) {
            sum.x += v[q].x;
            sum.y += v[q].y;
            sum.z += v[q].z;
            sum.w += v[q].w;
          }
        }
        const uint64_t at = static_cast<uint64_t>(row0 + r) * p.ldo + col0 + c;
        const float out[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
          if (col0 + c + e < p.n) store_from_f32(p.out, at + e, p.out_dtype, out[e]);
      }
    }
  }
  __syncwarp();
  cpt::cluster_sync();                 // no CTA leaves while another may read its shared memory
  if (warp == kSumWarps + 1) cpt::tmem_free_pair(tmem, p.tmem_columns);
}

// ----------------------------------------------- few rows of a, many bytes of w: tcgen05
//
// With at most 128 rows of a (launch_thin) the operands change places: 128 rows of w are the tensor core's
// 128 x 32 operand, up to 64 rows of a its N (16, 32 or 64) columns, and the kernel is bound by
// the stream of w (a second tile of rows of a finds it in L2).  A unit is 128 columns of tensor
// memory, 128 / kN groups side by side, so the sums (a lane has a row of w) wait once a unit; two
// units alternate.  Two CTAs share an SM; `splits` CTAs of a cluster share a tile's groups and
// add their sums in order through distributed shared memory.
//
// 1 x 4096 x 24576: 19.9 us, 101 MB at 5.1 TB/s; 48 rows of a: 22.8 us; 1 x 4096 x 4096: 6.3 us.  The
// fixed part is about 4 us (launch, tensor maps, the first loads, the exchange); the stream
// itself runs at the copy rate.

constexpr int kThinThreads = 256;      // four summing warps, TMA, MMA, scales, one idle
constexpr uint32_t kThinUnit = 128;    // columns of tensor memory
constexpr uint32_t kThinMaxStages = 6;
constexpr uint32_t kThinSmem = 111616;  // dynamic shared memory of a CTA, two to an SM

struct ThinParams {
  const float* sa;
  const float* sw;
  void* out;
  uint64_t ldo;
  uint32_t m, n, groups, splits, stages, tiles_m;
  int out_dtype;
};

template <uint32_t kN>
__global__ void __launch_bounds__(kThinThreads, 2)
    matmul_thin_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_w, const ThinParams p) {
  constexpr uint32_t kPer = kThinUnit / kN;            // groups of a unit
  constexpr uint32_t kStage = kTileA + kN * 128;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[2 * kThinMaxStages + 7];
  __shared__ __align__(16) float scales[2][kThinUnit];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = p.splits == 1 ? 0 : cpt::cluster_rank();
  const uint32_t tile = blockIdx.x / p.splits;       // those of one part of w come together
  const uint32_t row0 = tile / p.tiles_m * 128;
  const uint32_t token0 = tile % p.tiles_m * kN, tokens = min(p.m - token0, kN);
  const uint32_t full = cpt::smem_addr(bars), empty = full + 8 * kThinMaxStages;
  const uint32_t acc_full = empty + 8 * kThinMaxStages, acc_empty = acc_full + 16;
  const uint32_t scale_full = acc_empty + 16, drained = scale_full + 16;
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < p.stages; ++s) {
      cpt::mbar_init(full + 8 * s, 1);
      cpt::mbar_init(empty + 8 * s, 1);
    }
    for (uint32_t b = 0; b < 2; ++b) {
      cpt::mbar_init(acc_full + 8 * b, 1);
      cpt::mbar_init(acc_empty + 8 * b, 4);
      cpt::mbar_init(scale_full + 8 * b, 32);
    }
    cpt::mbar_init(drained, 1);
    cpt::mbar_init_fence();
    gave_up = 0;
  }
  if (warp == 5) cpt::tmem_alloc(cpt::smem_addr(&tmem_base), 2 * kThinUnit);
  cpt::tc_fence_before();
  __syncthreads();
  cpt::tc_fence_after();
  wait_for_previous();
  const uint32_t tmem = tmem_base;
  // whole units go to each CTA of the cluster
  const uint32_t units = (p.groups + kPer - 1) / kPer;
  const uint32_t u0 = units * rank / p.splits, u1 = units * (rank + 1) / p.splits;
  const uint32_t kb0 = u0 * kPer, kb1 = min(u1 * kPer, p.groups);
  float acc[kN];
#pragma unroll
  for (uint32_t i = 0; i < kN; ++i) acc[i] = 0.0f;
  bool ok = true;
  // Every warp comes here when its role ends.  If a wait ran out, whichever warp's, the loads and
  // products in flight then end (their waits have a limit too) before the stages and tensor memory are
  // used for anything else: the warps that issued them see to it within their own branches, where
  // the sums are not held.
  auto end_role = [&] {
    if (!ok && lane == 0) atomicOr(&g_matmul_gave_up, 1u);
    __syncwarp();
    cpt::tc_fence_before();
    asm volatile("barrier.sync 1, %0;" ::"n"(kThinThreads) : "memory");
  };

  if (warp == 4) {
    // ------------------------------------------------------------------ loads
    if (cpt::elect_one()) {
      cpt::tma_prefetch_map(&map_a);
      cpt::tma_prefetch_map(&map_w);
    }
    __syncwarp();
    uint32_t s = 0, round = 0, fills = 0;
    for (uint32_t kb = kb0; kb < kb1; ++kb) {
      if (round > 0) {
        ok = cpt::mbar_wait(empty + 8 * s, (round - 1) & 1, &gave_up);
        if (!ok) break;
      }
      const uint32_t dst = cpt::smem_addr(tiles) + s * kStage;
      if (cpt::elect_one()) {
        cpt::mbar_expect(full + 8 * s, kStage);
        cpt::tma_load(dst, &map_w, kb * 128, row0, full + 8 * s);
        cpt::tma_load(dst + kTileA, &map_a, kb * 128, token0, full + 8 * s);
      }
      __syncwarp();
      ++fills;
      if (++s == p.stages) {
        s = 0;
        ++round;
      }
    }
    end_role();
    if (gave_up != 0) {
      int late = 0;
      for (uint32_t k = 0; k < p.stages; ++k) {
        const LastFill last = last_fill(fills, fills, p.stages, k);
        if (last.any) cpt::mbar_wait(full + 8 * k, last.parity, &late);
      }
    }
  } else if (warp == 5) {
    // --------------------------------------------------------------- products
    constexpr uint32_t instr = cpt::e4m3_instr_desc(128, kN);
    uint32_t s = 0, round = 0, kb = kb0;
    for (uint32_t u = 0; kb < kb1; ++u) {
      const uint32_t b = u & 1;
      ok = u < 2 || cpt::mbar_wait(acc_empty + 8 * b, ((u >> 1) - 1) & 1, &gave_up);
      for (uint32_t g = 0; g < kPer && kb < kb1 && ok; ++g, ++kb) {
        ok = cpt::mbar_wait(full + 8 * s, round & 1, &gave_up);
        if (!ok) break;
        cpt::tc_fence_after();
        const uint32_t at = cpt::smem_addr(tiles) + s * kStage;
        const uint64_t dw = cpt::operand_desc(at), da = cpt::operand_desc(at + kTileA);
        if (cpt::elect_one()) {
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k)
            cpt::mma_one(tmem + b * kThinUnit + g * kN, dw + 2 * k, da + 2 * k, instr, k != 0);
          cpt::mma_commit(empty + 8 * s);
          if (g + 1 == kPer || kb + 1 == kb1) cpt::mma_commit(acc_full + 8 * b);
        }
        __syncwarp();
        if (++s == p.stages) {
          s = 0;
          ++round;
        }
      }
      if (!ok) break;
    }
    end_role();
    if (gave_up != 0) {
      int late = 0;
      if (cpt::elect_one()) cpt::mma_commit(drained);
      __syncwarp();
      cpt::mbar_wait(drained, 0, &late);
    }
  } else if (warp == 6) {
    // ----------------------------------------------------------------- scales
    const float* sw = p.sw + static_cast<uint64_t>(row0 / 128) * p.groups;
    uint32_t u = 0;
    for (uint32_t kb = kb0; kb < kb1; kb += kPer, ++u) {
      const uint32_t b = u & 1;
      float f[4];
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t e = lane + 32 * i, group = kb + e / kN, token = e % kN;
        f[i] = group < kb1 && token < tokens
                   ? p.sa[static_cast<uint64_t>(token0 + token) * p.groups + group] * sw[group]
                   : 0.0f;
      }
      if (u >= 2) {
        ok = cpt::mbar_wait(acc_empty + 8 * b, ((u >> 1) - 1) & 1, &gave_up);
        if (!ok) break;
      }
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) scales[b][lane + 32 * i] = f[i];
      cpt::mbar_arrive(scale_full + 8 * b);
    }
    end_role();
  } else if (warp < 4) {
    // ------------------------------------------------------------------- sums
    const uint32_t tmem_warp = tmem + ((warp * 32) << 16);
    uint32_t u = 0;
    for (uint32_t kb = kb0; kb < kb1; kb += kPer, ++u) {
      const uint32_t b = u & 1;
      ok = cpt::mbar_wait(scale_full + 8 * b, (u >> 1) & 1, &gave_up) &&
           cpt::mbar_wait(acc_full + 8 * b, (u >> 1) & 1, &gave_up);
      if (!ok) break;
      cpt::tc_fence_after();
      const uint32_t columns = min(kPer, kb1 - kb) * kN;     // of the unit that are filled
#pragma unroll
      for (uint32_t c = 0; c < 4; ++c) {
        if (32 * c < columns) {          // (a last unit of 16-column groups may fill half of it)
          float x[32];
          cpt::tmem_load32<0>(x, tmem_warp + b * kThinUnit + 32 * c);
          float f[32];
#pragma unroll
          for (uint32_t i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(&f[4 * i]) =
                *reinterpret_cast<const float4*>(&scales[b][32 * c + 4 * i]);
          cpt::tmem_load_wait(x);
          const uint32_t here = min(32u, columns - 32 * c);
#pragma unroll
          for (uint32_t i = 0; i < 32; ++i)
            if (kN >= 32 || i < 16 || here == 32)
              acc[(32 * c + i) % kN] = fmaf(x[i], f[i], acc[(32 * c + i) % kN]);
        }
      }
      cpt::tc_fence_before();
      __syncwarp();
      if (lane == 0) cpt::mbar_arrive(acc_empty + 8 * b);
    }
    end_role();
  } else {
    end_role();
  }
  if (gave_up != 0) __syncthreads();
  const uint32_t row = row0 + threadIdx.x;       // (of the summing warps)
  if (p.splits == 1) {
    if (warp < 4 && row < p.n) {
#pragma unroll
      for (uint32_t i = 0; i < kN; ++i)
        if (i < tokens)
          store_from_f32(p.out, static_cast<uint64_t>(token0 + i) * p.ldo + row, p.out_dtype,
                         acc[i]);
    }
  } else {
    // sums as [row of a][row of w] over the stages (all loads are used up); each CTA of the cluster
    // then adds a share of the tokens
    float* part = reinterpret_cast<float*>(tiles);
    if (warp < 4) {
#pragma unroll
      for (uint32_t i = 0; i < kN; ++i) part[i * 128 + threadIdx.x] = acc[i];
    }
    __syncthreads();
    cpt::cluster_sync();
    const uint32_t i0 = tokens * 32 * rank / p.splits, i1 = tokens * 32 * (rank + 1) / p.splits;
    for (uint32_t i = i0 + threadIdx.x; i < i1; i += kThinThreads) {
      const uint32_t at = cpt::smem_addr(part + 4 * i);
      float4 v[8];
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q)
        if (q < p.splits) v[q] = cpt::load_cluster4(cpt::map_rank(at, q));
      float4 sum = v[0];
#pragma unroll
      for (uint32_t q = 1; q < 8; ++q) {
        if (q < p.splits) {
          sum.x += v[q].x;
          sum.y += v[q].y;
          sum.z += v[q].z;
          sum.w += v[q].w;
        }
      }
      const uint32_t token = token0 + i / 32, r = row0 + i % 32 * 4;
      const float out[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e)
        if (r + e < p.n)
          store_from_f32(p.out, static_cast<uint64_t>(token) * p.ldo + r + e, p.out_dtype, out[e]);
    }
    __syncwarp();
    cpt::cluster_sync();             // no CTA leaves while another may read its shared memory
  }
  if (warp == 5) cpt::tmem_free(tmem, 2 * kThinUnit);
}

// What a launch needs to know of the device, found once.
using TcKernel = void (*)(CUtensorMap, CUtensorMap, TcParams);
constexpr TcKernel kTcKernels[8] = {      // tiles of 32, 64, .. 256 columns
    &matmul_tc_kernel<2>,  &matmul_tc_kernel<4>,  &matmul_tc_kernel<6>,  &matmul_tc_kernel<8>,
    &matmul_tc_kernel<10>, &matmul_tc_kernel<12>, &matmul_tc_kernel<14>, &matmul_tc_kernel<16>};

struct TcDevice {
  std::atomic<int> state{0};           // 1: found
  int clusters[3] = {0, 0, 0};         // clusters of 2, 4, 8 CTAs that run at once
};
TcDevice g_devices[64];
std::mutex g_device_lock;

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::atomic<EncodeTiled> g_encode{nullptr};

void launch_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, uint32_t cluster,
                   uint32_t ctas, size_t smem, cudaStream_t s) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3(ctas);
  cfg->blockDim = dim3(kTcThreads);
  cfg->dynamicSmemBytes = smem;
  cfg->stream = s;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

const TcDevice* tc_device(cudaError_t* err) {
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err == cudaSuccess && dev >= 64) *err = cudaErrorInvalidDevice;
  if (*err != cudaSuccess) return nullptr;
  TcDevice& d = g_devices[dev];
  if (d.state.load(std::memory_order_acquire) == 1) return &d;
  const std::lock_guard<std::mutex> one(g_device_lock);
  if (d.state.load(std::memory_order_acquire) == 1) return &d;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  *err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                          &found);
  if (*err != cudaSuccess) return nullptr;
  if (fn == nullptr || found != cudaDriverEntryPointSuccess) {
    *err = cudaErrorNotSupported;
    return nullptr;
  }
  g_encode.store(reinterpret_cast<EncodeTiled>(fn));
  for (TcKernel kernel : kTcKernels) {
    const void* k = reinterpret_cast<const void*>(kernel);
    cudaFuncAttributes attrs{};
    *err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSmemMost));
    if (*err == cudaSuccess) *err = cudaFuncGetAttributes(&attrs, k);
    if (*err == cudaSuccess && attrs.numRegs != kLaunchRegs) *err = cudaErrorInvalidConfiguration;
    if (*err != cudaSuccess) return nullptr;
  }
  for (const void* k : {reinterpret_cast<const void*>(&matmul_thin_kernel<16>),
                        reinterpret_cast<const void*>(&matmul_thin_kernel<32>),
                        reinterpret_cast<const void*>(&matmul_thin_kernel<64>)}) {
    *err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kThinSmem));
    if (*err != cudaSuccess) return nullptr;
  }
  for (int i = 0; i < 3 && *err == cudaSuccess; ++i) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    launch_config(&cfg, attr, 2u << i, (2u << i) * 64, kSmemMost, nullptr);
    int most = 0;
    *err = cudaOccupancyMaxActiveClusters(&most, reinterpret_cast<const void*>(kTcKernels[7]),
                                          &cfg);
    d.clusters[i] = most;
  }
  if (*err != cudaSuccess) return nullptr;
  if (d.clusters[0] < 1) {
    *err = cudaErrorInvalidConfiguration;
    return nullptr;
  }
  d.state.store(1, std::memory_order_release);
  return &d;
}

bool encode_map(CUtensorMap* map, const uint8_t* base, uint64_t k, uint64_t rows, uint64_t ld,
                uint32_t box_rows) {
  const cuuint64_t dims[2] = {k, rows};
  const cuuint64_t strides[1] = {rows == 1 ? (k + 15) / 16 * 16 : ld};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t elem[2] = {1, 1};
  return g_encode.load()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims,
                         strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Columns of a tile and pairs that share one, by the time that the busiest pair needs.  In
// nanoseconds, measured on tiles of one turn (k = 4096 and 24576, 64 to 256 columns): a group
// takes 250 + 0.85 a column, a tile's outputs 14 a column, and sharing a tile 4000.
void choose_tile(const TcDevice& d, uint32_t m, uint32_t n, uint32_t groups, uint32_t* bn,
                 uint32_t* splits) {
  const uint64_t tiles_m = (static_cast<uint64_t>(m) + 255) / 256;
  double best = 1e300;
  for (uint32_t i = 0; i < 3; ++i) {
    const uint32_t s = 1u << i;
    if (s > 1 && groups < 4 * s) break;
    for (uint32_t b = 256; b >= 32; b -= 32) {
      const uint64_t tiles = tiles_m * ((static_cast<uint64_t>(n) + b - 1) / b);
      const uint64_t at_once = static_cast<uint64_t>(d.clusters[i]);
      if (at_once == 0 || (s > 1 && tiles > at_once)) continue;
      const double turns = static_cast<double>((tiles + at_once - 1) / at_once);
      const double cost =
          turns * ((groups + s - 1) / s * (250.0 + 0.85 * b) + 14.0 * b) + (s > 1 ? 4000.0 : 0.0);
      if (cost < best) {
        best = cost;
        *bn = b;
        *splits = s;
      }
    }
  }
}

}  // namespace

namespace cpm {

cp_status launch_pairs(const MatmulParams& q, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const TcDevice* d = tc_device(&e);
  if (d == nullptr) return cpx::cuda_fail(e, "fp8 matmul device query");
  uint32_t bn = 32, splits = 1;
  choose_tile(*d, q.m, q.n, q.groups, &bn, &splits);
  TcParams p{};
  p.sa = q.sa;
  p.sw = q.sw;
  p.out = q.out;
  p.ldo = q.ldo;
  p.m = q.m;
  p.n = q.n;
  p.groups = q.groups;
  p.out_dtype = q.out_dtype;
  p.splits = splits;
  p.tiles_m = (q.m + 255) / 256;
  const uint64_t tiles = static_cast<uint64_t>(p.tiles_m) * ((q.n + bn - 1) / bn);
  if (tiles >= (1ull << 31)) {
    cpx::set_error("m and n make more than 2^31 tiles");
    return CP_ERR_INVALID_ARG;
  }
  p.tiles = static_cast<uint32_t>(tiles);
  const uint32_t stage = kTileA + bn * 64;
  p.stages = (kSmemMost - 1024) / stage;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.tmem_columns = 64;
  while (p.tmem_columns < 2 * bn) p.tmem_columns *= 2;
  const uint64_t elt = dtype_size(q.out_dtype);
  p.out_align = cpx::aligned(q.out, 32) && q.ldo * elt % 32 == 0   ? 32
                : cpx::aligned(q.out, 16) && q.ldo * elt % 16 == 0 ? 16
                                                                   : 0;
  CUtensorMap map_a, map_w;
  if (!encode_map(&map_a, q.a, q.k, q.m, q.lda, 128) ||
      !encode_map(&map_w, q.w, q.k, q.n, q.ldw, bn / 2)) {
    cpx::set_error("tensor map refused");
    return CP_ERR_CUDA;
  }
  const uint32_t at_once = static_cast<uint32_t>(d->clusters[splits == 1 ? 0 : splits == 2 ? 1 : 2]);
  const uint32_t clusters = splits > 1 || p.tiles < at_once ? p.tiles : at_once;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  launch_config(&cfg, attr, 2 * splits, 2 * splits * clusters, kSmemMost, s);
  e = cudaLaunchKernelEx(&cfg, kTcKernels[bn / 32 - 1], map_a, map_w, p);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul launch");
  return CP_OK;
}

cp_status launch_thin(const MatmulParams& q, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (tc_device(&e) == nullptr) return cpx::cuda_fail(e, "fp8 matmul device query");
  const uint32_t kn = q.m <= 16 ? 16 : q.m <= 32 ? 32 : 64;
  const uint32_t units = (q.groups + kThinUnit / kn - 1) / (kThinUnit / kn);
  const uint32_t tiles_m = (q.m + kn - 1) / kn;
  const uint32_t tiles = (q.n + 127) / 128 * tiles_m;
  // CTAs share a tile until there are enough to keep every SM's loads in flight.
  uint32_t splits = 1;
  while (splits < 8 && static_cast<uint64_t>(tiles) * splits * 2 <= 304 && units >= 2 * splits)
    splits *= 2;
  ThinParams p{q.sa, q.sw, q.out, q.ldo, q.m, q.n, q.groups, splits, 0, tiles_m, q.out_dtype};
  const uint32_t stage = kTileA + kn * 128;
  p.stages = (kThinSmem - 1024) / stage;
  if (p.stages > kThinMaxStages) p.stages = kThinMaxStages;
  CUtensorMap map_a, map_w;
  if (!encode_map(&map_a, q.a, q.k, q.m, q.lda, kn) ||
      !encode_map(&map_w, q.w, q.k, q.n, q.ldw, 128)) {
    cpx::set_error("tensor map refused");
    return CP_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  launch_config(&cfg, attr, splits, splits * tiles, kThinSmem, s);
  cfg.blockDim = dim3(kThinThreads);
  auto* fn = kn == 16 ? &matmul_thin_kernel<16> : kn == 32 ? &matmul_thin_kernel<32>
                                                            : &matmul_thin_kernel<64>;
  e = cudaLaunchKernelEx(&cfg, fn, map_a, map_w, p);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul launch");
  return CP_OK;
}

}  // namespace cpm

extern "C" cp_status cp_matmul_fp8_status(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul");
  uint32_t word = 0;
  e = cudaMemcpyFromSymbol(&word, g_matmul_gave_up, sizeof(word));
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul status");
  if (word == 0) return CP_OK;
  const uint32_t zero = 0;
  e = cudaMemcpyToSymbol(g_matmul_gave_up, &zero, sizeof(zero));
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul status");
  cpx::set_error("a wait inside cp_matmul_fp8 ran out of time; its output is not valid");
  return CP_ERR_CUDA;
}

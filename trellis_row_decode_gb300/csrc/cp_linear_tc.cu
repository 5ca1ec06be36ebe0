// cp_linear_tc.cu -- the 16-bit products of cp_linear and cp_linear_grad on tensor memory
// (tcgen05), for operands whose rows lie on 16-byte boundaries (include/cp.h).
//
//   out[i][j] = epilogue(sum over k of a[i][k] b[j][k])
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "cp.h"
#include "cp_epilogue.cuh"
#include "cp_internal.h"
#include "cp_layer.cuh"
#include "cp_linear.h"
#include "cp_ring.h"
#include "cp_tcgen05.cuh"

namespace {

using namespace cpl;
using cpe::DropKey;
using cpe::Epilogue;
using cplin::ColumnSums;
using cplin::kMostProducts;
using cplin::Tiling;

// A wait that ran out sets this word; cp_linear_status reads and clears it.
__device__ uint32_t g_linear_gave_up;

// --------------------------------------------------------------- pairs of SMs
//
// A pair of CTAs (two SMs) makes 256 x bn sums, bn a multiple of 32 up to 256.  Each CTA stages
// its 128 rows of a and its half of the bn rows of b, 64 of k a stage.  An operand that is stored
// along k comes as rows of 128 bytes; one that is stored across k (the gradient's: dz and x for dw,
// w for dx) as blocks of 64 by 64 that the tensor core transposes as it reads them, so neither
// is ever transposed in memory.  Roles: a thread each issues the TMA loads of a and of b, one of the
// first CTA the tcgen05.mma, sixteen warps per CTA finish the sums of one of two tensor-memory
// buffers while the tensor core fills the other (a lane has a row, four warps every fourth block of
// 32 columns), one adds up the column sums that the kernel before left in parts.  A CTA pair
// walks over its units: tiles of up to two products (dx and dw of one call), the k of each
// shared by `splits` units where there are few; their sums go to a workspace, and finish_kernel adds
// them in order.
//
// bf16, plain outputs, in bursts: 4096^3 72-73 us (1.9 PFLOP/s), k = 24576 429-434 (with bias and residual
// 432-438), in calls that go on, at the power limit, 83 and 503; fp16 76-77 and, read in segments,
// 467-473; both gradients of 4096^3: 142 us (1.94).  Bound by the tensor core there (85-89 % of
// its cycles): loads alone would take 216 ns for 64 of k at 256 columns, products alone 265, together
// 300.  What each piece is for: the issuing warps run whole on a warp-uniform index, so their
// operands are in uniform registers (64 of k at 64 columns: 230 -> 162 ns), narrow tiles stage 128 of
// k (162 -> 144; at 256 columns nothing), sixteen finishing warps and not eight hide the epilogue's
// chains, and the ring keeps what the slots leave (five stages and not six of 30 KB: 457 -> 497 us at
// k = 24576).  Short k is bound by the epilogue: 4096 x 4096 x 1024 plain 24.6 us, with silu 24.8, gelu
// 26.6, dropout 35, with everything 45 (the generator's products on their pipe, then the activations').

constexpr int kSumWarps = 16;
constexpr uint32_t kGroups = kSumWarps / 4;            // of four warps, one for each 32 lanes
constexpr uint32_t kLoadA = 0, kMmaWarp = 1, kLoadB = 2, kSumsWarp = 3, kFirstFinish = 4;
constexpr int kThreads = (kFirstFinish + kSumWarps) * 32;
constexpr uint32_t kStageK = 64;                       // of k in a stage, or a part of it: 128 bytes
constexpr uint32_t kMaxStages = 8;
constexpr uint32_t kTileA = 128 * 128;                 // bytes of a's rows per stage and CTA
constexpr uint32_t kBlock = 64 * 128;                  // bytes of a 64 x 64 block stored across k
constexpr uint32_t kSmemUsed = 225 * 1024;             // dynamic shared memory of a CTA
constexpr uint32_t kSmemMost = kSmemUsed + 1023;       // (and what it takes to start on 1024 bytes)
constexpr uint32_t kQuickK = 512;                      // k up to here: two slots a warp for residuals
constexpr uint32_t kTwoBytes = 24 * 1024;              // stages up to here hold two parts
constexpr uint32_t kBuffer = 256;                      // columns of tensor memory of a buffer
constexpr uint32_t kSegment = cplin::long_sum(CP_F32); // of k that the tensor core adds up alone
// Registers with segments: launched with 96 a thread (65,536 over 20 warps); the finishing warps
// (64 sums a thread) take what the other four give up.
constexpr int kLaunchRegs = 96, kFinishRegs = 104, kOtherRegs = 64;
static_assert(4 * kFinishRegs + kOtherRegs <= 5 * kLaunchRegs, "a warpgroup's share of the launch");
constexpr uint32_t kRasterRows = 16;                   // tiles along m that are walked together

struct PairProduct {
  Epilogue e;
  float* part;               // sums of the splits, [splits][m][pitch]
  uint64_t pitch;
  uint32_t kblocks, bn, splits, tiles_m, tiles_n, tiles;
  uint32_t b_bytes, b_boxes; // of b, a stage and CTA
  uint32_t instr;
  int a_across, b_across;
  int tma_out, tma_residual; // outputs leave, the residual comes, through shared memory and TMA
};

struct PairParams {
  CUtensorMap map_a[kMostProducts], map_b[kMostProducts], map_out[kMostProducts],
      map_residual[kMostProducts];
  PairProduct q[kMostProducts];
  ColumnSums sums;
  uint32_t first_units, units, stages, stage_bytes;
  uint32_t two;                // a stage holds 128 of k, in two parts
  uint32_t slots_at, slots;    // behind the stages: each finishing warp's bytes for its blocks
};

struct Unit {
  uint32_t which, split, row0, col0, kb0, kb1;
};

__device__ __forceinline__ Unit unit_of(const PairParams& p, uint32_t u) {
  Unit r;
  r.which = u < p.first_units ? 0 : 1;
  if (r.which != 0) u -= p.first_units;
  const PairProduct& q = p.q[r.which];
  r.split = u / q.tiles;
  const uint32_t tile = u - r.split * q.tiles;
  const uint32_t wide = kRasterRows * q.tiles_n, g = tile / wide, at = tile - g * wide;
  const uint32_t rows = min(kRasterRows, q.tiles_m - g * kRasterRows), tn = at / rows;
  r.row0 = (g * kRasterRows + at - tn * rows) * 256;
  r.col0 = tn * q.bn;
  r.kb0 = static_cast<uint32_t>(static_cast<uint64_t>(q.kblocks) * r.split / q.splits);
  r.kb1 = static_cast<uint32_t>(static_cast<uint64_t>(q.kblocks) * (r.split + 1) / q.splits);
  return r;
}

// 32 rows of 64 bytes of outputs (32 columns of 16 bits, the first 16 of v in 32 bits) in a slot, as
// a tensor map with the 64-byte swizzle lays them out; a lane has a row.  `add`: the residual's
// block lies there already.
constexpr uint32_t kSlot = 32 * 64;
__device__ __forceinline__ void write_slot(uint32_t slot, uint32_t lane, int dtype, bool add,
                                           float (&v)[32]) {
  if (dtype == CP_F32) {
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c)
      cpt::store_shared4(slot + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4), __float_as_uint(v[4 * c]),
                         __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                         __float_as_uint(v[4 * c + 3]));
    return;
  }
#pragma unroll
  for (uint32_t c = 0; c < 4; ++c) {
    const uint32_t at = slot + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4);
    if (add) {
      const uint4 r = cpt::load_shared4(at);
      cpe::add_pair(v[8 * c], v[8 * c + 1], r.x, dtype);
      cpe::add_pair(v[8 * c + 2], v[8 * c + 3], r.y, dtype);
      cpe::add_pair(v[8 * c + 4], v[8 * c + 5], r.z, dtype);
      cpe::add_pair(v[8 * c + 6], v[8 * c + 7], r.w, dtype);
    }
    uint32_t w[4];
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      w[i] = dtype == CP_F16 ? pack_pair<__half>(v[8 * c + 2 * i], v[8 * c + 2 * i + 1])
                             : pack_pair<__nv_bfloat16>(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
    cpt::store_shared4(at, w[0], w[1], w[2], w[3]);
  }
}

// A warp's 32 columns (c on) of sums over rows of 16 bits on 16-byte boundaries: four lanes a row,
// eight rows at a time, eight such loads under way.
template <typename T>
__device__ __forceinline__ void add_rows(const ColumnSums& p, uint32_t col, uint32_t first,
                                         float (&acc)[8]) {
  const T* at = static_cast<const T*>(p.rows) + col;
  const uint32_t here = min(p.n - col, 8u);
  for (uint32_t r = first; r < p.count; r += 64) {
    Packed<T> x[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      x[i] = zero_octet<T>();
      if (r + 8 * i < p.count && here == 8) x[i] = load_octet(at + (r + 8 * i) * p.pitch);
    }
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      float v[8];
      unpack(x[i], v);
      if (r + 8 * i < p.count && here < 8) {           // (the columns' last octet)
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e)
          if (e < here) v[e] = to_f32(at[(r + 8 * i) * p.pitch + e]);
      }
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) acc[e] += v[e];
    }
  }
}
__device__ __forceinline__ void sum_rows(const ColumnSums& p, uint32_t c, uint32_t lane) {
  const uint32_t col = c + 8 * (lane & 3);
  float acc[8] = {};
  if (col < p.n) {
    if (p.rows_dtype == CP_F16) add_rows<__half>(p, col, lane >> 2, acc);
    else add_rows<__nv_bfloat16>(p, col, lane >> 2, acc);
  }
  __syncwarp();
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e) {
#pragma unroll
    for (uint32_t s = 4; s < 32; s *= 2) acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], s);
  }
  if (lane < 4) {
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) {
      if (col + e < p.n) {
        if (p.accumulate) acc[e] += load_as_f32(p.out, col + e, p.dtype);
        store_from_f32(p.out, col + e, p.dtype, acc[e]);
      }
    }
  }
  __syncwarp();
}

// kRich: some product has an activation, dropout, or sums to keep.
// kSegments: some product has more of k in a unit than its outputs' type allows (long_sum).  The tensor
// core cuts what it adds instead of rounding it, an error that grows with k (relative, random bf16
// operands: 1.07e-9 k, 4.4e-6 at k = 4096, where fp32 additions that round leave 6e-7; positive ones
// 6e-9 k, all to one side); so the sum is read every kSegment of k and added up in registers.
template <bool kRich, bool kSegments>
__global__ void __launch_bounds__(kThreads, 1) pairs_kernel(const __grid_constant__ PairParams p) {
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 5];
  __shared__ __align__(8) uint64_t residual_bars[kSumWarps];
  __shared__ uint32_t tmem_base;
  __shared__ uint32_t issued[2];           // this CTA's fills of stages, by either issuer
  __shared__ int gave_up;
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t warp = cpt::warp_index(), lane = threadIdx.x & 31;
  const uint32_t half = cpt::cluster_rank();
  const uint32_t full = cpt::smem_addr(bars), empty = full + 8 * kMaxStages;
  const uint32_t acc_full = empty + 8 * kMaxStages, acc_empty = acc_full + 16;
  const uint32_t drained = acc_empty + 16;
  // the first CTA's barriers hold the pair's loads and reads
  const uint32_t pair_full = cpt::map_rank(full, 0);
  const uint32_t pair_acc_empty = cpt::map_rank(acc_empty, 0);

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
    for (uint32_t w = 0; w < kSumWarps; ++w) cpt::mbar_init(cpt::smem_addr(&residual_bars[w]), 1);
    cpt::mbar_init_fence();
    gave_up = 0;
  }
  if (warp == kMmaWarp) cpt::tmem_alloc_pair(cpt::smem_addr(&tmem_base), 2 * kBuffer);
  cpt::tc_fence_before();
  __syncthreads();
  cpt::cluster_sync();
  cpt::tc_fence_after();
  wait_for_previous();          // (the set-up above runs while the kernel before this one ends)
  let_next_start();
  const uint32_t tmem = tmem_base;
  const uint32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  // Every warp of the pair comes here when its role ends.  If a wait of the first CTA ran out,
  // whichever warp's, what the pair has in flight then ends before either CTA leaves its shared and
  // tensor memory (the second waits at the cluster's last barrier): loads up to the last fill that
  // either CTA began, all of which count on the first CTA's barriers, and every product issued.
  // These waits have a limit too.  Where the first CTA has not given up, its finishing warps have
  // seen every product done, so nothing is in flight.
  auto end_role = [&] {
    __syncwarp();
    cpt::tc_fence_before();
    asm volatile("barrier.sync 1, %0;" ::"n"(kThreads) : "memory");
    cpt::cluster_sync();
  };

  if (warp < kFirstFinish) {
    if constexpr (kSegments) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadA || warp == kLoadB) {
      // ---------------------------------------------------------------- loads
      // (a warp for a, one for b; each runs its loop whole and elects a thread to issue)
      const bool is_a = warp == kLoadA;
      if (p.units != 0 && cpt::elect_one()) {    // (column sums alone come without a map)
        for (int i = 0; i < kMostProducts; ++i)
          cpt::tma_prefetch_map(is_a ? &p.map_a[i] : &p.map_b[i]);
      }
      __syncwarp();
      const uint32_t base = cpt::smem_addr(tiles) + (is_a ? 0 : kTileA), k_shift = 6 + p.two;
      uint32_t s = 0, parity = 1, fills = 0;     // (parity 1: a stage that was never filled is free)
      bool ok = true;
      for (uint32_t u = pair; u < p.units && ok; u += pairs) {
        const Unit t = unit_of(p, u);
        const PairProduct& q = p.q[t.which];
        const CUtensorMap* map = is_a ? &p.map_a[t.which] : &p.map_b[t.which];
        const bool a1 = t.row0 + 128 < q.e.m;             // the second CTA has rows of a
        const bool across = (is_a ? q.a_across : q.b_across) != 0;
        const uint32_t boxes = is_a ? (half == 0 || a1 ? (across ? 2 : 1) : 0) : q.b_boxes;
        const uint32_t bytes = (2 * q.b_bytes + (a1 ? 2 : 1) * kTileA) << p.two;
        const uint32_t at = is_a ? t.row0 + half * 128 : t.col0 + half * (q.bn / 2);
        const bool expect = is_a && half == 0;
        for (uint32_t kb = t.kb0; kb < t.kb1; ++kb) {
          ok = cpt::mbar_wait(empty + 8 * s, parity, &gave_up);
          if (!ok) break;
          const uint32_t dst = base + s * p.stage_bytes, k0 = kb << k_shift;
          const uint32_t dst2 = dst + p.stage_bytes / 2, bar = pair_full + 8 * s;
          if (cpt::elect_one()) {
            if (expect) cpt::mbar_expect(full + 8 * s, bytes);
            if (across) {
              for (uint32_t i = 0; i < boxes; ++i) {
                cpt::tma_load_pair(dst + i * kBlock, map, at + 64 * i, k0, bar);
                if (p.two) cpt::tma_load_pair(dst2 + i * kBlock, map, at + 64 * i, k0 + kStageK, bar);
              }
            } else if (boxes != 0) {
              cpt::tma_load_pair(dst, map, k0, at, bar);
              if (p.two) cpt::tma_load_pair(dst2, map, k0 + kStageK, at, bar);
            }
          }
          __syncwarp();
          ++fills;
          if (++s == p.stages) {
            s = 0;
            parity ^= 1;
          }
        }
      }
      if (lane == 0) issued[is_a ? 0 : 1] = fills;
      end_role();
      if (gave_up != 0 && half == 0 && is_a) {
        const uint32_t other = cpt::map_rank(cpt::smem_addr(issued), 1);
        const uint32_t mine = max(issued[0], issued[1]);
        const uint32_t theirs = max(cpt::load_cluster1(other), cpt::load_cluster1(other + 4));
        int late = 0;
        for (uint32_t k = 0; k < p.stages; ++k) {
          const LastFill last = last_fill(mine, theirs, p.stages, k);
          if (last.any) cpt::mbar_wait(full + 8 * k, last.parity, &late);
        }
      }
    } else if (warp == kMmaWarp && half == 0) {
      // ------------------------------------------------------------- products
      const uint32_t segment = kSegment / kStageK >> p.two;
      uint32_t it = 0, s = 0, parity = 0;
      bool ok = true;
      for (uint32_t u = pair; u < p.units && ok; u += pairs) {
        const Unit t = unit_of(p, u);
        const PairProduct& q = p.q[t.which];
        const uint32_t instr = q.instr;
        const uint32_t a_step = q.a_across ? 128 : 2, b_step = q.b_across ? 128 : 2;
        const uint32_t a_low = cpt::desc_low(cpt::smem_addr(tiles), q.a_across != 0);
        const uint32_t b_low = cpt::desc_low(cpt::smem_addr(tiles) + kTileA, q.b_across != 0);
        for (uint32_t kb = t.kb0; kb < t.kb1 && ok; ++it) {
          const uint32_t b = it & 1, to = tmem + b * kBuffer;
          const uint32_t end = kSegments ? min(kb + segment, t.kb1) : t.kb1;
          ok = it < 2 || cpt::mbar_wait(acc_empty + 8 * b, ((it >> 1) - 1) & 1, &gave_up);
          if (!ok) break;
          uint32_t more = 0;
          for (; kb < end; ++kb) {
            ok = cpt::mbar_wait(full + 8 * s, parity, &gave_up);
            if (!ok) break;
            cpt::tc_fence_after();
            const uint32_t at = s * (p.stage_bytes >> 4), at2 = at + (p.stage_bytes >> 5);
            if (cpt::elect_one()) {
              cpt::mma_half_pair(to, cpt::desc_of(a_low + at), cpt::desc_of(b_low + at), instr, more);
#pragma unroll
              for (uint32_t k = 1; k < 4; ++k)
                cpt::mma_half_pair(to, cpt::desc_of(a_low + at + k * a_step),
                                   cpt::desc_of(b_low + at + k * b_step), instr, 1);
              if (p.two) {
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k)
                  cpt::mma_half_pair(to, cpt::desc_of(a_low + at2 + k * a_step),
                                     cpt::desc_of(b_low + at2 + k * b_step), instr, 1);
              }
              cpt::mma_commit_pair(empty + 8 * s, 3);
              if (kb + 1 == end) cpt::mma_commit_pair(acc_full + 8 * b, 3);
            }
            __syncwarp();
            more = 1;
            if (++s == p.stages) {
              s = 0;
              parity ^= 1;
            }
          }
        }
      }
      end_role();
      if (gave_up != 0) {
        int late = 0;
        if (cpt::elect_one()) cpt::mma_commit_pair(drained, 1);
        __syncwarp();
        cpt::mbar_wait(drained, 0, &late);
      }
    } else if (warp == kSumsWarp) {
      // ---------------------------------------------------------- column sums
      if (p.sums.out != nullptr && p.sums.rows != nullptr) {
        for (uint32_t c = blockIdx.x * 32; c < p.sums.n; c += gridDim.x * 32)
          sum_rows(p.sums, c, lane);
      } else if (p.sums.out != nullptr) {
        for (uint32_t c = blockIdx.x * 32 + lane; c < p.sums.n; c += gridDim.x * 32) {
          float sum = 0.0f;
#pragma unroll 8
          for (uint32_t i = 0; i < p.sums.count; ++i)
            sum += p.sums.parts[static_cast<uint64_t>(i) * p.sums.pitch + c];
          if (p.sums.accumulate) sum += load_as_f32(p.sums.out, c, p.sums.dtype);
          store_from_f32(p.sums.out, c, p.sums.dtype, sum);
        }
      }
      end_role();
    } else {
      end_role();
    }
  } else {
    // --------------------------------------------------------------- finish
    if constexpr (kSegments) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFinishRegs));
    const uint32_t mine = warp - kFirstFinish, lanes = (warp & 3) * 32, group = mine >> 2;
    const DropKey key = cpe::drop_key(p.q[0].e.drop);      // (dropout is in the first product alone)
    const uint32_t slots = cpt::smem_addr(tiles) + p.slots_at + mine * p.slots;
    const uint32_t residual_bar = cpt::smem_addr(&residual_bars[mine]);
    uint32_t it = 0;
    Awaited coming;                            // loads of the residual
    bool ok = true;
    for (uint32_t u = pair; u < p.units && ok; u += pairs) {
      const Unit t = unit_of(p, u);
      const PairProduct& q = p.q[t.which];
      const uint32_t blocks = q.bn / 32;
      const uint32_t row0 = t.row0 + half * 128 + lanes;
      const bool raw = q.splits > 1;
      float bias[2] = {};                      // of this lane's columns
      if (q.e.bias != nullptr && !raw) {
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
          const uint32_t c = kGroups * i + group, col = t.col0 + c * 32 + lane;
          if (c < blocks && col < q.e.n) bias[i] = load_as_f32(q.e.bias, col, q.e.bias_dtype);
        }
      }
      uint32_t left = 0;                       // blocks of this warp that have outputs
      if (row0 < q.e.m)
        for (uint32_t c = group; c < blocks && t.col0 + 32 * c < q.e.n; c += kGroups) ++left;
      auto load_residual = [&](uint32_t i, uint32_t count) {   // of blocks i on, slots are free
        if (lane == 0) {
          cpt::stores_read();
          cpt::mbar_expect(residual_bar, count * kSlot);
          for (uint32_t j = 0; j < count; ++j)
            cpt::tma_load(slots + j * kSlot, &p.map_residual[t.which],
                          t.col0 + 32 * (kGroups * (i + j) + group), row0, residual_bar);
        }
        __syncwarp();
        coming.begun();
      };
      const bool two_slots = p.slots > kSlot;
      if (q.tma_residual && left != 0) load_residual(0, two_slots ? left : 1);
      const uint32_t tmem_warp = tmem + (lanes << 16) + 32 * group;
      auto give_back = [&](uint32_t b) {       // the tensor core may have the buffer again
        cpt::tc_fence_before();
        __syncwarp();
        if (lane == 0) cpt::mbar_arrive_cluster(pair_acc_empty + 8 * b);
      };
      auto finish = [&](uint32_t i, float(&v)[32]) {
        const uint32_t col = t.col0 + 32 * (kGroups * i + group);
        if (raw) {
          if (row0 + lane < q.e.m)
            cpe::store32(q.part,
                         (static_cast<uint64_t>(t.split) * q.e.m + row0 + lane) * q.pitch + col,
                         CP_F32, v);
          __syncwarp();
          return;
        }
        const bool fast = q.e.aligned != 0 && col + 32 <= q.e.n;
        cpe::shape_block<kRich>(q.e, key, row0, col, lane, i == 0 ? bias[0] : bias[1], fast, v);
        if (!q.tma_out) {
          cpe::write_block(q.e, row0, col, lane, fast, v);
          return;
        }
        if (q.tma_residual) {
          if (i != 0 && !two_slots) load_residual(i, 1);
          const uint32_t slot = slots + (two_slots ? i * kSlot : 0);
          if (coming.under_way) {
            ok = cpt::mbar_wait(residual_bar, coming.parity, &gave_up);
            coming.waited(ok);
            if (!ok) return;                   // (the slot is still the load's)
          }
          write_slot(slot, lane, q.e.out_dtype, true, v);
          cpt::stores_fence();
          __syncwarp();
          if (lane == 0) cpt::tma_store(&p.map_out[t.which], col, row0, slot);
          __syncwarp();
          return;
        }
        if (q.e.residual != nullptr && row0 + lane < q.e.m) {      // (of 32 bits)
          const uint64_t at = static_cast<uint64_t>(row0 + lane) * q.e.ldr + col;
          if (fast) {
            cpe::add32(v, q.e.residual, at, CP_F32);
          } else {
#pragma unroll
            for (uint32_t j = 0; j < 32; ++j)
              if (col + j < q.e.n) v[j] += static_cast<const float*>(q.e.residual)[at + j];
          }
        }
        // 32 columns of 16 bits at a time, or 16 of 32
        const uint32_t halves = q.e.out_dtype == CP_F32 ? 2 : 1;
        for (uint32_t h = 0; h < halves && col + 16 * h < q.e.n; ++h) {
          if (lane == 0) cpt::stores_read();
          __syncwarp();
          write_slot(slots, lane, q.e.out_dtype, false, v);
          cpt::stores_fence();
          __syncwarp();
          if (lane == 0) cpt::tma_store(&p.map_out[t.which], col + 16 * h, row0, slots);
          __syncwarp();
          if (halves == 2) {
#pragma unroll
            for (uint32_t j = 0; j < 16; ++j) v[j] = v[j + 16];
          }
        }
      };
      if constexpr (kSegments) {
        float acc[64];
#pragma unroll
        for (uint32_t i = 0; i < 64; ++i) acc[i] = 0.0f;
        for (uint32_t kb = t.kb0; kb < t.kb1; kb += kSegment / kStageK >> p.two, ++it) {
          const uint32_t b = it & 1;
          ok = cpt::mbar_wait(acc_full + 8 * b, (it >> 1) & 1, &gave_up);
          if (!ok) break;
          cpt::tc_fence_after();
#pragma unroll
          for (uint32_t i = 0; i < 2; ++i) {
            if (i < left) {
              float v[32];
              cpt::tmem_load32<0>(v, tmem_warp + b * kBuffer + 32 * kGroups * i);
              cpt::tmem_load_wait(v);
#pragma unroll
              for (uint32_t j = 0; j < 32; ++j) acc[32 * i + j] += v[j];
            }
          }
          give_back(b);
        }
        if (!ok) break;
        for (uint32_t i = 0; i < left && ok; ++i) {
          float v[32];
#pragma unroll
          for (uint32_t j = 0; j < 32; ++j) v[j] = acc[j];
#pragma unroll
          for (uint32_t j = 0; j < 32; ++j) acc[j] = acc[j + 32];
          finish(i, v);
        }
      } else {
        const uint32_t b = it & 1;
        ok = cpt::mbar_wait(acc_full + 8 * b, (it >> 1) & 1, &gave_up);
        if (!ok) break;
        cpt::tc_fence_after();
        ++it;
        if (left == 0) give_back(b);
        for (uint32_t i = 0; i < left && ok; ++i) {
          float v[32];
          cpt::tmem_load32<0>(v, tmem_warp + b * kBuffer + 32 * kGroups * i);
          cpt::tmem_load_wait(v);
          if (i + 1 == left) give_back(b);
          finish(i, v);
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&g_linear_gave_up, 1u);
    if (lane == 0) cpt::stores_done();         // before the slots are someone else's
    __syncwarp();
    if (coming.under_way) {
      int late = 0;
      cpt::mbar_wait(residual_bar, coming.parity, &late);
    }
    end_role();
  }
  __syncwarp();
  cpt::cluster_sync();                 // no CTA leaves while the other may use its memory
  if (warp == kMmaWarp) cpt::tmem_free_pair(tmem, 2 * kBuffer);
}

// ------------------------------------------------------------- sums of the splits
//
// Four neighbouring sums a thread: the splits' added in order, then the epilogue.  Also the whole
// of a product whose k is 0 (no splits: sums of nothing).

struct FinishProduct {
  Epilogue e;
  const float* part;
  uint64_t pitch;
  uint32_t splits, quads;              // quads of a row
};
struct FinishParams {
  FinishProduct q[kMostProducts];
  uint64_t first, total;               // quads of the first product, of both
};

constexpr int kFinishThreads = 256;

__global__ void __launch_bounds__(kFinishThreads)
    finish_kernel(const __grid_constant__ FinishParams p) {
  wait_for_previous();
  let_next_start();
  const DropKey key = cpe::drop_key(p.q[0].e.drop);
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * kFinishThreads;
  for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * kFinishThreads + threadIdx.x; u < p.total;
       u += step) {
    const FinishProduct& q = p.q[u < p.first ? 0 : 1];
    const uint64_t at = u < p.first ? u : u - p.first;
    const uint32_t row = (at >> 32) == 0 ? static_cast<uint32_t>(at) / q.quads
                                         : static_cast<uint32_t>(at / q.quads);
    const uint32_t col = static_cast<uint32_t>(at - static_cast<uint64_t>(row) * q.quads) * 4;
    float v[4] = {};
#pragma unroll 4
    for (uint32_t i = 0; i < q.splits; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(
          q.part + (static_cast<uint64_t>(i) * q.e.m + row) * q.pitch + col);
      v[0] += x.x;
      v[1] += x.y;
      v[2] += x.z;
      v[3] += x.w;
    }
    cpe::finish_quad(q.e, key, row, col, v);
  }
}

// ------------------------------------------- few rows of a, many bytes of b: one SM
//
// With at most 128 rows of a the operands change places: 128 rows of b are the tensor core's
// 128 x 16 operand, up to 64 rows of a its N (16, 32, 48 or 64) columns, and the kernel is bound by
// the stream of b (a second tile of rows of a finds it in L2).  Two CTAs share an SM; `splits` CTAs
// of a cluster share a tile's k and add their sums in order through distributed shared memory.
//
// 1 x 4096 x 24576: 32.3 us, 201 MB at 6.2 TB/s; 48 rows of a 34.6, 128 rows 41.2 (the pairs 39.7, 40.7,
// 44.6); 1 x 4096 x 4096 7.8-9.0 (24.8), 128 rows 12.0 (14.1); 1 x 1024 x 1024 4.0, about 4 us being start,
// first loads and exchange.

constexpr int kThinThreads = 256;      // four finishing warps, TMA, MMA, two idle
constexpr uint32_t kThinMaxStages = 6;
constexpr uint32_t kThinSmem = 115200; // dynamic shared memory of a CTA, two to an SM

struct ThinParams {
  Epilogue e;
  uint32_t kblocks, splits, stages, tiles_m, instr;
};

template <uint32_t kN>
__global__ void __launch_bounds__(kThinThreads, 2)
    thin_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ ThinParams p) {
  constexpr uint32_t kStage = kTileA + kN * 128;
  constexpr uint32_t kBufferN = kN == 48 ? 64 : kN;  // of tensor memory: two buffers, a power of two
  constexpr uint32_t kColumns = 2 * kBufferN;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[2 * kThinMaxStages + 5];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t warp = cpt::warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = p.splits == 1 ? 0 : cpt::cluster_rank();
  const uint32_t tile = blockIdx.x / p.splits;       // those of one part of b come together
  const uint32_t row0 = tile / p.tiles_m * 128;
  const uint32_t token0 = tile % p.tiles_m * kN, tokens = min(p.e.m - token0, kN);
  const uint32_t full = cpt::smem_addr(bars), empty = full + 8 * kThinMaxStages;
  const uint32_t acc_full = empty + 8 * kThinMaxStages, acc_empty = acc_full + 16;
  const uint32_t drained = acc_empty + 16;
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < p.stages; ++s) {
      cpt::mbar_init(full + 8 * s, 1);
      cpt::mbar_init(empty + 8 * s, 1);
    }
    for (uint32_t b = 0; b < 2; ++b) {
      cpt::mbar_init(acc_full + 8 * b, 1);
      cpt::mbar_init(acc_empty + 8 * b, 4);
    }
    cpt::mbar_init(drained, 1);
    cpt::mbar_init_fence();
    gave_up = 0;
  }
  if (warp == 5) cpt::tmem_alloc(cpt::smem_addr(&tmem_base), kColumns);
  cpt::tc_fence_before();
  __syncthreads();
  cpt::tc_fence_after();
  wait_for_previous();
  let_next_start();
  const uint32_t tmem = tmem_base;
  const uint32_t kb0 = static_cast<uint32_t>(static_cast<uint64_t>(p.kblocks) * rank / p.splits);
  const uint32_t kb1 =
      static_cast<uint32_t>(static_cast<uint64_t>(p.kblocks) * (rank + 1) / p.splits);
  float* part = reinterpret_cast<float*>(tiles);     // [row of a][row of b], over the stages
  bool ok = true;
  // Every warp comes here when its role ends.  If a wait ran out, whichever warp's, the loads and
  // products in flight then end (their waits have a limit too) before the stages and tensor memory
  // are used for anything else.
  auto end_role = [&] {
    if (!ok && lane == 0) atomicOr(&g_linear_gave_up, 1u);
    __syncwarp();
    cpt::tc_fence_before();
    asm volatile("barrier.sync 1, %0;" ::"n"(kThinThreads) : "memory");
  };

  if (warp == 4) {
    // ------------------------------------------------------------------ loads
    if (cpt::elect_one()) {
      cpt::tma_prefetch_map(&map_a);
      cpt::tma_prefetch_map(&map_b);
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
        cpt::tma_load(dst, &map_b, kb * kStageK, row0, full + 8 * s);
        cpt::tma_load(dst + kTileA, &map_a, kb * kStageK, token0, full + 8 * s);
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
    uint32_t s = 0, round = 0, it = 0;
    for (uint32_t kb = kb0; kb < kb1 && ok; ++it) {
      const uint32_t b = it & 1, end = min(kb + kSegment / kStageK, kb1);
      ok = it < 2 || cpt::mbar_wait(acc_empty + 8 * b, ((it >> 1) - 1) & 1, &gave_up);
      if (!ok) break;
      uint32_t more = 0;
      for (; kb < end; ++kb) {
        ok = cpt::mbar_wait(full + 8 * s, round & 1, &gave_up);
        if (!ok) break;
        cpt::tc_fence_after();
        const uint32_t at = cpt::smem_addr(tiles) + s * kStage;
        const uint64_t db = cpt::operand_desc(at), da = cpt::operand_desc(at + kTileA);
        if (cpt::elect_one()) {
          cpt::mma_half_one(tmem + b * kBufferN, db, da, p.instr, more);
#pragma unroll
          for (uint32_t k = 1; k < 4; ++k)
            cpt::mma_half_one(tmem + b * kBufferN, db + 2 * k, da + 2 * k, p.instr, 1);
          cpt::mma_commit(empty + 8 * s);
          if (kb + 1 == end) cpt::mma_commit(acc_full + 8 * b);
        }
        __syncwarp();
        more = 1;
        if (++s == p.stages) {
          s = 0;
          ++round;
        }
      }
    }
    end_role();
    if (gave_up != 0) {
      int late = 0;
      if (cpt::elect_one()) cpt::mma_commit(drained);
      __syncwarp();
      cpt::mbar_wait(drained, 0, &late);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------------- sums
    float acc[kN];
#pragma unroll
    for (uint32_t i = 0; i < kN; ++i) acc[i] = 0.0f;
    uint32_t it = 0;
    for (uint32_t kb = kb0; kb < kb1; kb += kSegment / kStageK, ++it) {
      const uint32_t b = it & 1;
      ok = cpt::mbar_wait(acc_full + 8 * b, (it >> 1) & 1, &gave_up);
      if (!ok) break;
      cpt::tc_fence_after();
      const uint32_t at = tmem + ((warp * 32) << 16) + b * kBufferN;
#pragma unroll
      for (uint32_t c = 0; c < (kN + 31) / 32; ++c) {
        float x[32] = {};
        const bool part = 32 * c + 32 > kN;
        if (part) cpt::tmem_load16<0>(x, at + 32 * c);
        else cpt::tmem_load32<0>(x, at + 32 * c);
        cpt::tmem_load_wait(x);
#pragma unroll
        for (uint32_t i = 0; i < 32; ++i)
          if (32 * c + i < kN) acc[32 * c + i < kN ? 32 * c + i : 0] += x[i];
      }
      cpt::tc_fence_before();
      __syncwarp();
      if (lane == 0) cpt::mbar_arrive(acc_empty + 8 * b);
    }
    if (ok) {                            // (all products are done: the stages are free)
#pragma unroll
      for (uint32_t i = 0; i < kN; ++i) part[i * 128 + threadIdx.x] = acc[i];
    }
    end_role();
  } else {
    end_role();
  }
  __syncthreads();
  if (p.splits > 1) cpt::cluster_sync();
  const DropKey key = cpe::drop_key(p.e.drop);
  const uint32_t i0 = tokens * 32 * rank / p.splits, i1 = tokens * 32 * (rank + 1) / p.splits;
  for (uint32_t i = i0 + threadIdx.x; i < i1; i += kThinThreads) {
    const uint32_t at = cpt::smem_addr(part + 4 * i);
    float v[4];
    if (p.splits == 1) {
      const float4 x = *reinterpret_cast<const float4*>(part + 4 * i);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
      float4 x[8];
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q)
        if (q < p.splits) x[q] = cpt::load_cluster4(cpt::map_rank(at, q));
      v[0] = x[0].x; v[1] = x[0].y; v[2] = x[0].z; v[3] = x[0].w;
#pragma unroll
      for (uint32_t q = 1; q < 8; ++q) {
        if (q < p.splits) {
          v[0] += x[q].x;
          v[1] += x[q].y;
          v[2] += x[q].z;
          v[3] += x[q].w;
        }
      }
    }
    const uint32_t col = row0 + i % 32 * 4;
    if (col < p.e.n) cpe::finish_quad(p.e, key, token0 + i / 32, col, v);
  }
  if (p.splits > 1) cpt::cluster_sync();  // no CTA leaves while another may read its shared memory
  __syncwarp();
  if (warp == 5) cpt::tmem_free(tmem, kColumns);
}

// ---------------------------------------------------------------------------- host

using PairKernel = void (*)(PairParams);
constexpr PairKernel kPairKernels[4] = {      // 1: rich, 2: segments
    &pairs_kernel<false, false>, &pairs_kernel<true, false>, &pairs_kernel<false, true>,
    &pairs_kernel<true, true>};

// What a launch needs to know of the device, found once.
struct Device {
  std::atomic<int> state{0};           // 1: found
  int pairs = 0;                       // clusters of two CTAs that run at once
};
Device g_devices[64];
std::mutex g_device_lock;

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::atomic<EncodeTiled> g_encode{nullptr};

const Device* device(cudaError_t* err) {
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err == cudaSuccess && dev >= 64) *err = cudaErrorInvalidDevice;
  if (*err != cudaSuccess) return nullptr;
  Device& d = g_devices[dev];
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
  auto allow = [&](const void* kernel, uint32_t bytes) {
    if (*err == cudaSuccess)
      *err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(bytes));
  };
  for (int i = 0; i < 4; ++i) {
    allow(reinterpret_cast<const void*>(kPairKernels[i]), kSmemMost);
    cudaFuncAttributes attrs{};
    if (*err == cudaSuccess)
      *err = cudaFuncGetAttributes(&attrs, reinterpret_cast<const void*>(kPairKernels[i]));
    if (*err == cudaSuccess && i >= 2 && attrs.numRegs != kLaunchRegs)
      *err = cudaErrorInvalidConfiguration;
  }
  allow(reinterpret_cast<const void*>(&thin_kernel<16>), kThinSmem);
  allow(reinterpret_cast<const void*>(&thin_kernel<32>), kThinSmem);
  allow(reinterpret_cast<const void*>(&thin_kernel<48>), kThinSmem);
  allow(reinterpret_cast<const void*>(&thin_kernel<64>), kThinSmem);
  if (*err != cudaSuccess) return nullptr;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(256);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemMost;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int most = 0;
  *err = cudaOccupancyMaxActiveClusters(&most, reinterpret_cast<const void*>(kPairKernels[3]),
                                        &cfg);
  if (*err == cudaSuccess && most < 1) *err = cudaErrorInvalidConfiguration;
  if (*err != cudaSuccess) return nullptr;
  d.pairs = most;
  d.state.store(1, std::memory_order_release);
  return &d;
}

// Boxes of 64 elements of the array's rows by box_rows of them.
bool encode_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t rows, uint64_t ld,
                uint32_t box_rows) {
  const cuuint64_t dims[2] = {inner, rows};
  const cuuint64_t strides[1] = {rows == 1 ? (2 * inner + 15) / 16 * 16 : 2 * ld};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t elem[2] = {1, 1};
  return g_encode.load()(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims,
                         strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 32 rows by 64 bytes of the outputs (or of the residual) as write_slot lays them out.
bool encode_block_map(CUtensorMap* map, const void* base, int dtype, uint64_t n, uint64_t m,
                      uint64_t ld) {
  const uint64_t size = dtype_size(dtype);
  const cuuint64_t dims[2] = {n, m};
  const cuuint64_t strides[1] = {m == 1 ? (size * n + 15) / 16 * 16 : size * ld};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(64 / size), 32};
  const cuuint32_t elem[2] = {1, 1};
  return g_encode.load()(
             map, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
             const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool block_map_ok(const void* p, int dtype, uint64_t m, uint64_t ld) {
  return cpx::aligned(p, 16) && (m == 1 || (ld != 0 && ld * dtype_size(dtype) % 16 == 0));
}
// A store writes whole 16-byte pieces: of a row that ends inside one, what lies behind it too
// (measured).  Loads end with the row's last element.
bool store_map_ok(const void* p, int dtype, uint64_t n, uint64_t m, uint64_t ld) {
  return block_map_ok(p, dtype, m, ld) && n * dtype_size(dtype) % 16 == 0;
}

// Columns of a tile and units that share its k, of each product of a launch.  By shapes alone, for
// the 76 pairs of a whole card, so that a product's sums and its workspace are the same wherever it
// runs.  In nanoseconds, measured at 4096 x 4096 and on a turn of few tiles: 64 of k take 303 at
// 256 columns, 273 at 224, 204 at 128, 144 at 64 and below; a tile besides them 300 + 6.5 a
// column; sharing k 4500 and the sums' way to memory and back.  Units are dealt in turn, so the
// first pair has the most.
constexpr uint32_t kPairs = 76;
Tiling best_splits(uint32_t m, uint32_t n, uint32_t k, uint32_t bn) {
  const uint32_t kblocks = (k + kStageK - 1) / kStageK;
  const uint64_t tiles = (static_cast<uint64_t>(m) + 255) / 256 * ((static_cast<uint64_t>(n) + bn - 1) / bn);
  const double stage = bn <= 80 ? 140.0 : 60.0 + 0.95 * bn;
  const double traffic = 4.0 / 3000.0 * m * n;
  Tiling best{};
  double least = 0.0;
  for (uint32_t s : {1u, 2u, 3u, 4u, 6u, 8u, 12u, 16u, 24u, 32u}) {
    if (s > 1 && (tiles * s > 2 * kPairs || 4 * s > kblocks)) break;
    Tiling t{bn, s, tiles * s, (kblocks + s - 1) / s * stage + 300.0 + 6.5 * bn, 0.0};
    if (s > 1) t.extra = 4500.0 + (s + 1) * traffic;
    const double cost = static_cast<double>((t.units + kPairs - 1) / kPairs) * t.each + t.extra;
    if (s == 1 || cost < least) {
      least = cost;
      best = t;
    }
  }
  return best;
}
uint64_t part_pitch(uint32_t n) { return (static_cast<uint64_t>(n) + 31) / 32 * 32; }

bool rich(const Epilogue& e) {
  return e.act != CP_ACT_NONE || e.drop.mode != 0 || e.pre != nullptr;
}

cp_status too_many_tiles() {
  cpx::set_error("m and n make more than 2^31 tiles");
  return CP_ERR_INVALID_ARG;
}

}  // namespace

namespace cplin {

Tilings tilings(const uint32_t* m, const uint32_t* n, const uint32_t* k, int count) {
  Tilings t{};
  for (int i = 0; i < count; ++i) {
    t.m[i] = m[i];
    t.n[i] = n[i];
    for (uint32_t b = 0; b < kWidths; ++b) t.way[i][b] = best_splits(m[i], n[i], k[i], 256 - 32 * b);
  }
  return t;
}

void choose(const Tilings& t, int first, int count, Tiling* out) {
  const Tiling none{};
  const Tiling *ways = t.way[first], *others = count > 1 ? t.way[first + 1] : &none;
  double least = 1e300;
  for (int a = 0; a < kWidths; ++a) {
    for (int b = 0; b < (count > 1 ? kWidths : 1); ++b) {
      const bool swap = others[b].each > ways[a].each;     // (the longer units go first)
      const Tiling &x = swap ? others[b] : ways[a], &y = swap ? ways[a] : others[b];
      const uint64_t turns = (x.units + kPairs - 1) / kPairs;
      const uint64_t all = (x.units + y.units + kPairs - 1) / kPairs;
      const double even = (x.units * x.each + y.units * y.each) * (1.0 / kPairs);
      const double cost = std::max(turns * x.each + (all - turns) * y.each, even) +
                          std::max(x.extra, y.extra);
      if (cost < least) {
        least = cost;
        out[0] = ways[a];
        if (count > 1) out[1] = others[b];
      }
    }
  }
}

// With dropout a short k's products are done before the finishing warps are.  Up to 128 columns a warp
// has one block of a tile, above two in a row: 128 columns where the last turn then loses clearly less.
// Nanoseconds of a tile's finishing, measured at k = 1024.  Both widths measured at 84 sizes and epilogues
// beyond L2: 0.86 to 1.02 of the time where this takes 128 (8192 x 2048 x 1024 with a residual 43.8 us to
// 37.6, with silu and kept sums too 50.6 to 45.2), 0.96 to 1.05 where it does not.
void choose_dropped(const Tilings& t, Tiling* chosen) {
  const Tiling& narrow = t.way[0][4];                      // 128 columns
  if (chosen->splits != 1 || narrow.splits != 1 || chosen->bn <= narrow.bn) return;
  auto cost = [](const Tiling& x, double finish) {
    return x.each + static_cast<double>((x.units + kPairs - 1) / kPairs) * std::max(x.each, finish);
  };
  if (cost(narrow, 1800.0 + 22.5 * 128) < 0.92 * cost(*chosen, 3800.0 + 19.5 * chosen->bn))
    *chosen = narrow;
}

uint64_t part_floats(const Tilings& t, int first, int count) {
  Tiling chosen[kMostProducts];
  choose(t, first, count, chosen);
  uint64_t floats = 0;
  for (int i = 0; i < count; ++i)
    if (chosen[i].splits > 1)
      floats += static_cast<uint64_t>(chosen[i].splits) * t.m[first + i] * part_pitch(t.n[first + i]);
  return floats;
}

cp_status launch_products(const Product* q, int count, const Tiling* chosen, const ColumnSums& sums,
                          float* part, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const Device* d = device(&e);
  if (d == nullptr) return cpx::cuda_fail(e, "linear device query");
  PairParams p{};
  FinishParams f{};
  bool is_rich = false, segments = false, finish = false;
  uint64_t units[kMostProducts] = {};
  uint32_t ks[kMostProducts] = {};
  int used = 0;
  for (int i = 0; i < count; ++i)
    if (q[i].e.m != 0 && q[i].e.n != 0 && q[i].k != 0) ks[used++] = q[i].k;
  // units are dealt in turn: the longer ones first
  const bool swap = used == 2 && chosen[1].each > chosen[0].each;
  used = 0;
  for (int i = 0; i < count; ++i) {
    const Epilogue& ep = q[i].e;
    if (ep.m == 0 || ep.n == 0) continue;
    const uint64_t quads = (static_cast<uint64_t>(ep.n) + 3) / 4;
    FinishProduct& fp = f.q[i];
    fp.e = ep;
    fp.quads = static_cast<uint32_t>(quads);
    if (q[i].k == 0) {                     // sums of nothing
      finish = true;
      (i == 0 ? f.first : f.total) += quads * ep.m;
      continue;
    }
    const int at = swap ? 1 - used : used;
    PairProduct& x = p.q[at];
    const Tiling& t = chosen[used];
    x.e = ep;
    x.bn = t.bn;
    x.splits = t.splits;
    x.tiles_m = (ep.m + 255) / 256;
    x.tiles_n = (ep.n + t.bn - 1) / t.bn;
    const uint64_t tiles = static_cast<uint64_t>(x.tiles_m) * x.tiles_n;
    units[at] = tiles * t.splits;
    if (units[at] >= (1ull << 31)) return too_many_tiles();
    x.tiles = static_cast<uint32_t>(tiles);
    x.a_across = q[i].a.across;
    x.b_across = q[i].b.across;
    x.b_boxes = x.b_across ? (t.bn / 2 + 63) / 64 : 1;
    x.b_bytes = x.b_across ? x.b_boxes * kBlock : t.bn / 2 * 128;
    x.instr = cpt::half_instr_desc(256, t.bn, q[i].dtype == CP_BF16, x.a_across, x.b_across);
    segments |= q[i].k / t.splits > min(long_sum(ep.out_dtype),
                                        ep.pre != nullptr ? long_sum(ep.pre_dtype) : ~0u);
    if (t.splits > 1) {
      x.pitch = part_pitch(ep.n);
      x.part = part;
      part += static_cast<uint64_t>(t.splits) * ep.m * x.pitch;
      fp.part = x.part;
      fp.pitch = x.pitch;
      fp.splits = t.splits;
      finish = true;
      (i == 0 ? f.first : f.total) += quads * ep.m;
    } else {
      is_rich |= rich(ep);
    }
    const Operand &a = q[i].a, &b = q[i].b;
    const bool ok =
        (a.across ? encode_map(&p.map_a[at], a.p, ep.m, q[i].k, a.ld, kStageK)
                  : encode_map(&p.map_a[at], a.p, q[i].k, ep.m, a.ld, 128)) &&
        (b.across ? encode_map(&p.map_b[at], b.p, ep.n, q[i].k, b.ld, kStageK)
                  : encode_map(&p.map_b[at], b.p, q[i].k, ep.n, b.ld, t.bn / 2));
    if (!ok) {
      cpx::set_error("tensor map refused");
      return CP_ERR_CUDA;
    }
    // Outputs through TMA, where their rows allow it, and the residual too, unless it has 32 bits.
    const bool f32 = ep.out_dtype == CP_F32;
    const bool residual_ok =
        ep.residual == nullptr ||
        (f32 ? ep.aligned != 0 : block_map_ok(ep.residual, ep.out_dtype, ep.m, ep.ldr));
    x.tma_out = t.splits == 1 && residual_ok &&
                store_map_ok(ep.out, ep.out_dtype, ep.n, ep.m, ep.ldo);
    x.tma_residual = x.tma_out && ep.residual != nullptr && !f32;
    if ((x.tma_out &&
         !encode_block_map(&p.map_out[at], ep.out, ep.out_dtype, ep.n, ep.m, ep.ldo)) ||
        (x.tma_residual &&
         !encode_block_map(&p.map_residual[at], ep.residual, ep.out_dtype, ep.n, ep.m, ep.ldr))) {
      cpx::set_error("tensor map refused");
      return CP_ERR_CUDA;
    }
    // (both blocks' residuals ahead where tiles follow one another quickly: 4096 x 4096 x 256 16.7 us
    // against 18.6; a deeper ring of stages where they do not: k = 24576 453 against 500)
    if (x.tma_out)
      p.slots = max(p.slots, x.tma_residual && q[i].k <= kQuickK ? 2 * kSlot : kSlot);
    p.stage_bytes = max(p.stage_bytes, kTileA + x.b_bytes);
    ++used;
  }
  if (units[0] + units[1] >= (1ull << 31)) return too_many_tiles();
  if (used > 0 || (sums.out != nullptr && sums.n != 0)) {
    p.sums = sums;
    p.first_units = static_cast<uint32_t>(units[0]);
    p.units = static_cast<uint32_t>(units[0] + units[1]);
    if (used == 0) p.stage_bytes = kTileA;
    if (used == 1) {                       // (prefetched, not used)
      p.map_a[1] = p.map_a[0];
      p.map_b[1] = p.map_b[0];
    }
    p.two = p.stage_bytes <= kTwoBytes ? 1 : 0;
    p.stage_bytes <<= p.two;
    p.stages = min((kSmemUsed - kSumWarps * p.slots) / p.stage_bytes, kMaxStages);
    p.slots_at = p.stages * p.stage_bytes;
    for (int i = 0; i < used; ++i)
      p.q[swap ? 1 - i : i].kblocks = (ks[i] + (kStageK << p.two) - 1) / (kStageK << p.two);
    uint32_t pairs = p.units;
    if (sums.out != nullptr) pairs = max(pairs, (sums.n + 63) / 64);
    pairs = min(pairs, static_cast<uint32_t>(d->pairs));
    const Launch l{dim3(2 * pairs), kThreads, kSmemMost, s, 2};
    e = launch(l, kPairKernels[(is_rich ? 1 : 0) + (segments ? 2 : 0)], p);
    if (e != cudaSuccess) return cpx::cuda_fail(e, "linear launch");
  }
  if (finish) {
    f.total += f.first;
    const uint64_t ctas = (f.total + kFinishThreads - 1) / kFinishThreads;
    e = launch(Launch{dim3(static_cast<unsigned>(ctas < 1216 ? ctas : 1216)), kFinishThreads, 0, s},
               &finish_kernel, f);
    if (e != cudaSuccess) return cpx::cuda_fail(e, "linear launch");
  }
  return CP_OK;
}

cp_status launch_thin(const Product& q, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (device(&e) == nullptr) return cpx::cuda_fail(e, "linear device query");
  const uint32_t m = q.e.m, n = q.e.n;
  const uint32_t kn = m <= 16 ? 16 : m <= 32 ? 32 : m <= 48 || (m > 64 && m <= 96) ? 48 : 64;
  ThinParams p{};
  p.e = q.e;
  p.kblocks = (q.k + kStageK - 1) / kStageK;
  p.tiles_m = (m + kn - 1) / kn;
  const uint64_t tiles = (static_cast<uint64_t>(n) + 127) / 128 * p.tiles_m;
  // CTAs share a tile until there are enough to keep every SM's loads in flight.
  p.splits = 1;
  while (p.splits < 8 && tiles * p.splits * 2 <= 304 && p.kblocks >= 2 * p.splits) p.splits *= 2;
  if (tiles * p.splits >= (1ull << 31)) return too_many_tiles();
  p.instr = cpt::half_instr_desc(128, kn, q.dtype == CP_BF16, false, false);
  p.stages = min((kThinSmem - 1024) / (kTileA + kn * 128), kThinMaxStages);
  CUtensorMap map_a, map_b;
  if (!encode_map(&map_a, q.a.p, q.k, m, q.a.ld, kn) ||
      !encode_map(&map_b, q.b.p, q.k, n, q.b.ld, 128)) {
    cpx::set_error("tensor map refused");
    return CP_ERR_CUDA;
  }
  const Launch l{dim3(static_cast<unsigned>(tiles * p.splits)), kThinThreads, kThinSmem, s,
                 p.splits};
  e = kn == 16   ? launch(l, &thin_kernel<16>, map_a, map_b, p)
      : kn == 32 ? launch(l, &thin_kernel<32>, map_a, map_b, p)
      : kn == 48 ? launch(l, &thin_kernel<48>, map_a, map_b, p)
                 : launch(l, &thin_kernel<64>, map_a, map_b, p);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "linear launch");
  return CP_OK;
}

}  // namespace cplin

extern "C" cp_status cp_linear_status(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cpx::cuda_fail(e, "linear");
  uint32_t word = 0;
  e = cudaMemcpyFromSymbol(&word, g_linear_gave_up, sizeof(word));
  if (e != cudaSuccess) return cpx::cuda_fail(e, "linear status");
  if (word == 0) return CP_OK;
  const uint32_t zero = 0;
  e = cudaMemcpyToSymbol(g_linear_gave_up, &zero, sizeof(zero));
  if (e != cudaSuccess) return cpx::cuda_fail(e, "linear status");
  cpx::set_error("a wait inside cp_linear or cp_linear_grad ran out of time; its output is not valid");
  return CP_ERR_CUDA;
}

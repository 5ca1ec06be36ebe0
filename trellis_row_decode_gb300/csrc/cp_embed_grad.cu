// cp_embed_grad.cu -- gradient of a table lookup by sorted ids (include/cp.h,
// cp_embed_grad).
//
//   grad[r] = scale * sum of dy[j / group] over the j with ids[j] = r
//
// 1. Sort.  (id, position) pairs are sorted stably by id with a radix sort: a
//    kernel counts digits per tile, the next places every pair (its digit's base,
//    plus the counts of earlier tiles, plus its rank in the tile), and so on for
//    each digit.  Ids outside the table sort behind all rows.  Up to kSmallMax ids
//    are sorted by one CTA in shared memory instead: one launch, no global passes.
// 2. Sum.  Lookups (reads of a dy row) and table rows (writes of a grad row) are
//    merged into one list, each row behind its lookups, and the list is cut into
//    chunks of equal length, one per warp and slab of 256 columns: a warp's share of
//    the traffic is the same whether it meets one hot row or a stretch of rows that
//    no id names.  A cut that falls inside a row moves to the row's end when that is
//    at most 32 lookups away; else the row's parts go to the workspace as fp32 sums.
// 3. Join.  The parts of a row that spans chunks are added in order, and written.
// Every sum's order follows from the ids alone: no floating-point atomics.
//
// Bound by memory: dy read once, grad written once.  196,608 Zipf ids, 1024 columns of bf16 into
// 131,072 rows: the sums take 112 us of the call's 145 (671 MB at 6.0 TB/s), the sort's four
// kernels and the join of the hot rows the rest, which waits for latency, not bandwidth.  4,096
// ids of 4,096 x 256 fp32: 15.2 us, three kernels whose chains of dependent loads are the bound.
#include <cstdint>

#include <cuda_runtime.h>

#include "cp.h"
#include "cp_internal.h"
#include "cp_layer.cuh"
#include "cp_tcgen05.cuh"

namespace {

using namespace cpl;

constexpr uint32_t kFull = 0xFFFFFFFFu;

// ------------------------------------------------------------------------ sort

constexpr int kRounds = 4;                                   // keys per thread and sub-tile
constexpr int kSmallThreads = 1024;
constexpr uint32_t kSmallMax = kSmallThreads * kRounds;      // ids that one CTA sorts
constexpr int kSortThreads = 512;
constexpr uint32_t kSub = kSortThreads * kRounds;            // 2048 keys per sub-tile
constexpr uint32_t kMaxTiles = 512;
constexpr int kMaxBits = 9;                                  // digit width
constexpr int kSmallBits = 8;                                // in one CTA (48 KB of shared memory)
constexpr uint32_t kMaxBins = 1u << kMaxBits;

__device__ __forceinline__ uint32_t key_of(int64_t id, uint32_t n_rows) {
  return static_cast<uint64_t>(id) < n_rows ? static_cast<uint32_t>(id) : n_rows;
}

// Lanes whose digit (of `bits` bits) is the same as this lane's, among those with a key.
__device__ __forceinline__ uint32_t same_digit(uint32_t digit, int bits, bool have) {
  uint32_t peers = __ballot_sync(kFull, have);
  for (int b = 0; b < bits; ++b) {
    const uint32_t set = __ballot_sync(kFull, (digit >> b) & 1);
    peers &= (digit >> b) & 1 ? set : ~set;
  }
  return peers;
}

// Exclusive prefix sums of v[0..bins), bins <= 512, over the CTA (512 threads or more).
__device__ __forceinline__ void exclusive_scan(uint32_t* v, uint32_t bins, uint32_t* warp_sums) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t own = 0, x = 0;
  if (threadIdx.x < kMaxBins) {
    own = x = threadIdx.x < bins ? v[threadIdx.x] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kFull, x, o);
      if (lane >= static_cast<uint32_t>(o)) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
  }
  __syncthreads();
  if (threadIdx.x < kMaxBins) {
    const uint32_t before = __reduce_add_sync(kFull, lane < warp ? warp_sums[lane] : 0);
    if (threadIdx.x < bins) v[threadIdx.x] = before + x - own;
  }
  __syncthreads();
}

// Ranks of a sub-tile's keys among the keys of the same digit, in order.  Warp w owns
// keys [w * 128, w * 128 + 128), 32 a round; `hist` [warp][bin] ends as the count of the
// bin in earlier warps, `total` as the sub-tile's counts.  digit == bins: no key.
struct Ranks {
  uint32_t r[kRounds];
};

template <int kThreads>
__device__ __forceinline__ Ranks rank_digits(const uint32_t (&digit)[kRounds], int bits,
                                             uint16_t* hist, uint32_t* total) {
  constexpr int kWarps = kThreads / 32;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1u << bits;
  uint16_t* mine = hist + warp * bins;
  for (uint32_t b = lane; b < bins; b += 32) mine[b] = 0;
  __syncwarp();
  Ranks out;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const uint32_t d = digit[r];
    const bool have = d < bins;
    const uint32_t peers = same_digit(d, bits, have);
    const uint32_t before = __popc(peers & ((1u << lane) - 1));
    uint32_t prior = 0;
    if (have) prior = mine[d];
    __syncwarp();
    if (have && before == 0) mine[d] = static_cast<uint16_t>(prior + __popc(peers));
    __syncwarp();
    out.r[r] = prior + before;
  }
  __syncthreads();
  for (uint32_t b = threadIdx.x; b < bins; b += kThreads) {
    uint32_t c[kWarps], sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) c[w] = hist[w * bins + b];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      hist[w * bins + b] = static_cast<uint16_t>(sum);
      sum += c[w];
    }
    total[b] = sum;
  }
  __syncthreads();
  return out;
}

// Up to kSmallMax ids in one CTA: all passes in shared memory.
__global__ void __launch_bounds__(kSmallThreads)
    sort_small_kernel(const int64_t* ids, uint32_t n, uint32_t n_rows, int passes,
                      int bits, uint2* pairs_out, uint32_t* status) {
  __shared__ uint32_t key_s[kSmallMax];
  __shared__ uint16_t pos_s[kSmallMax];
  extern __shared__ uint16_t hist[];             // [warps][bins]
  __shared__ uint32_t total[kMaxBins], warp_sums[32];
  wait_for_previous();
  let_next_start();
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t key[kRounds], pos[kRounds];
  bool bad = false;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const uint32_t i = warp * (32 * kRounds) + r * 32 + lane;
    pos[r] = i;
    key[r] = n_rows;
    if (i < n) {
      key[r] = key_of(ids[i], n_rows);
      bad |= key[r] == n_rows;
    }
  }
  if (status != nullptr && bad) atomicOr(status, 1u);
  const uint32_t bins = 1u << bits;
  for (int p = 0; p < passes; ++p) {
    uint32_t digit[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      digit[r] = pos[r] < n ? (key[r] >> (p * bits)) & (bins - 1) : bins;
    const Ranks rk = rank_digits<kSmallThreads>(digit, bits, hist, total);
    exclusive_scan(total, bins, warp_sums);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      if (digit[r] < bins) {
        const uint32_t to = total[digit[r]] + hist[warp * bins + digit[r]] + rk.r[r];
        key_s[to] = key[r];
        pos_s[to] = static_cast<uint16_t>(pos[r]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const uint32_t i = warp * (32 * kRounds) + r * 32 + lane;
      if (i < n) {
        key[r] = key_s[i];
        pos[r] = pos_s[i];
      } else {
        pos[r] = kFull;                          // no key: stays out of every digit
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const uint32_t i = warp * (32 * kRounds) + r * 32 + lane;
    if (i < n) pairs_out[i] = make_uint2(key[r], pos[r]);
  }
}

// Counts are kept at two levels, so that placing a tile reads few of them: a cluster of
// kTileCluster tiles adds up its tiles' counts through distributed shared memory.
constexpr uint32_t kTileCluster = 8;

struct SortPass {
  const int64_t* ids;            // first pass: the ids; else null
  const uint2* pairs;            // later passes: (key, position) of the pass before
  uint2* pairs_out;
  uint32_t* counts;              // [tiles][bins]: keys in the earlier tiles of the tile's cluster
  uint32_t* totals;              // [clusters][bins]: keys of a cluster
  uint32_t n, n_rows, per_tile;  // per_tile: a multiple of kSub
  uint32_t shift;
  int bits;
  uint32_t* status;
};

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortPass p) {
  __shared__ uint32_t hist[kMaxBins];
  const uint32_t bins = 1u << p.bits;
  for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads) hist[b] = 0;
  __syncthreads();
  wait_for_previous();
  let_next_start();
  const uint64_t lo = static_cast<uint64_t>(blockIdx.x) * p.per_tile;
  const uint64_t hi = lo + p.per_tile < p.n ? lo + p.per_tile : p.n;
  bool bad = false;
  for (uint64_t i0 = lo; i0 < hi; i0 += kSub) {
    uint32_t key[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const uint64_t i = i0 + r * kSortThreads + threadIdx.x;
      key[r] = kFull;
      if (i < hi) {
        key[r] = p.ids != nullptr ? key_of(p.ids[i], p.n_rows) : p.pairs[i].x;
        bad |= key[r] == p.n_rows;
      }
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      if (key[r] != kFull) atomicAdd(&hist[(key[r] >> p.shift) & (bins - 1)], 1u);
  }
  if (p.ids != nullptr && p.status != nullptr && bad) atomicOr(p.status, 1u);
  cpt::cluster_sync();
  const uint32_t rank = blockIdx.x % kTileCluster;
  for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads) {
    const uint32_t at = cpt::smem_addr(hist + b);
    uint32_t c[kTileCluster], before = 0, all = 0;
#pragma unroll
    for (uint32_t q = 0; q < kTileCluster; ++q)
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(c[q]) : "r"(cpt::map_rank(at, q)));
#pragma unroll
    for (uint32_t q = 0; q < kTileCluster; ++q) {
      before += q < rank ? c[q] : 0;
      all += c[q];
    }
    p.counts[blockIdx.x * bins + b] = before;
    if (rank == 0) p.totals[blockIdx.x / kTileCluster * bins + b] = all;
  }
  cpt::cluster_sync();               // no CTA leaves while another may read its counts
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortPass p) {
  extern __shared__ uint16_t hist[];             // [warps][bins]
  __shared__ uint32_t total[kMaxBins], warp_sums[32];
  __shared__ uint32_t base[kMaxBins];            // where this tile's next key of a digit goes
  __shared__ uint4 part[kSortThreads], part_all[kSortThreads];
  const uint32_t bins = 1u << p.bits, tile = blockIdx.x;
  const uint32_t clusters = gridDim.x / kTileCluster, cluster = tile / kTileCluster;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_previous();
  let_next_start();
  const uint64_t lo = static_cast<uint64_t>(tile) * p.per_tile;
  const uint64_t hi = lo + p.per_tile < p.n ? lo + p.per_tile : p.n;
  uint2 pair[kRounds];
  auto load_pairs = [&](uint64_t i0) {
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const uint64_t i = i0 + warp * (32 * kRounds) + r * 32 + lane;
      pair[r] = make_uint2(kFull, kFull);
      if (i < hi)
        pair[r] = p.ids != nullptr
                      ? make_uint2(key_of(p.ids[i], p.n_rows), static_cast<uint32_t>(i))
                      : p.pairs[i];
    }
  };
  load_pairs(lo);
  // Counts of each digit in the clusters before this one and in all: bins / 4 threads read a
  // cluster's counts four at a time, and the thread groups share the clusters.
  {
    const uint32_t per = bins / 4, groups = kSortThreads / per;       // bins >= 4
    const uint32_t g = threadIdx.x / per, q = threadIdx.x - g * per;
    uint4 before = make_uint4(0, 0, 0, 0), all = before;
    if (g < groups) {
#pragma unroll 4
      for (uint32_t t = g; t < clusters; t += groups) {
        const uint4 c = *reinterpret_cast<const uint4*>(p.totals + t * bins + 4 * q);
        all.x += c.x;
        all.y += c.y;
        all.z += c.z;
        all.w += c.w;
        if (t < cluster) {
          before.x += c.x;
          before.y += c.y;
          before.z += c.z;
          before.w += c.w;
        }
      }
    }
    part[threadIdx.x] = before;
    part_all[threadIdx.x] = all;
    uint32_t own = 0;
    if (threadIdx.x < bins) own = p.counts[tile * bins + threadIdx.x];
    __syncthreads();
    const uint32_t* parts = reinterpret_cast<const uint32_t*>(part);
    const uint32_t* parts_all = reinterpret_cast<const uint32_t*>(part_all);
    static_assert(kMaxBins <= kSortThreads, "a thread per bin");
    if (threadIdx.x < bins) {
      uint32_t y = 0;
      for (uint32_t k = 0; k < groups; ++k) {
        own += parts[k * bins + threadIdx.x];
        y += parts_all[k * bins + threadIdx.x];
      }
      total[threadIdx.x] = y;
    }
    __syncthreads();
    exclusive_scan(total, bins, warp_sums);
    if (threadIdx.x < bins) base[threadIdx.x] = own + total[threadIdx.x];
    __syncthreads();
  }
  for (uint64_t i0 = lo; i0 < hi; i0 += kSub) {
    if (i0 != lo) load_pairs(i0);
    uint32_t digit[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      digit[r] = pair[r].y != kFull ? (pair[r].x >> p.shift) & (bins - 1) : bins;
    const Ranks rk = rank_digits<kSortThreads>(digit, p.bits, hist, total);
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      if (digit[r] < bins)
        p.pairs_out[base[digit[r]] + hist[warp * bins + digit[r]] + rk.r[r]] = pair[r];
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads) base[b] += total[b];
    __syncthreads();
  }
}

// ------------------------------------------------------------------- sum and join

constexpr int kSumThreads = 256;
constexpr uint32_t kSlab = 256;                  // columns of a warp: an octet per lane
constexpr uint32_t kAhead = 8;                   // dy rows in flight per warp
constexpr uint32_t kBatch = 128;                 // lookups whose ids a warp stages at a time
constexpr uint32_t kWarps = kSumThreads / 32;

// Bytes of a warp's octets of one dy row in the ring, with the word behind them where rows start
// anywhere.
template <typename T, bool VEC>
constexpr uint32_t ring_row() {
  return 32 * 8 * sizeof(T) + (VEC ? 0 : 16);
}

struct SumParams {
  const uint2* pairs;            // (id, position), sorted; id n_rows for those outside the table
  uint32_t n, n_rows, d, slabs, chunks, per_chunk;
  uint32_t lanes_log2;           // a row's octets in a warp, rounded up to a power of two
  uint32_t group;                // lookups that share a row of dy
  const void* dy;
  uint64_t dy_stride;
  float scale;
  void* grad;
  uint64_t grad_stride;
  uint64_t pitch;                // d rounded up to whole octets
  float* head;                   // [chunks][pitch]: a row's last part, where it began earlier
  float* tail;                   // [chunks][pitch]: a row's part, where it goes on
  uint32_t* head_row;            // [chunks]: that row, or kFull
  uint32_t* end_key;             // [chunks]: 2 * (row in progress at the end) + (1: a part is left)
};

// A cut of the merged list: entries before `i` and rows before `r` lie in front of it.
// mid: row r has entries in front of the cut and more than 32 behind it.
struct Cut {
  uint32_t i, r;
  bool mid;
};

// The cut at diagonal `diag` (all lanes of the warp take part).  Overwriting, the list
// holds every row; accumulating, only lookups count and rows are those they name.
template <bool ACC>
__device__ __forceinline__ Cut find_cut(const SumParams& p, uint64_t diag) {
  const uint32_t lane = threadIdx.x & 31;
  Cut c;
  if constexpr (ACC) {
    if (diag >= p.n) return Cut{p.n, p.n_rows, false};
    c.i = static_cast<uint32_t>(diag);
  } else {
    if (diag >= static_cast<uint64_t>(p.n) + p.n_rows) return Cut{p.n, p.n_rows, false};
    // the smallest i in [lo, hi] with i == hi or keys[i] >= diag - i: 33 parts a step
    uint64_t lo = diag > p.n_rows ? diag - p.n_rows : 0;
    uint64_t hi = diag < p.n ? diag : p.n;
    while (lo < hi) {
      const uint64_t step = (hi - lo + 32) / 33;
      const uint64_t at = lo + step * (lane + 1) - 1;        // probes lo+step-1, lo+2step-1, ..
      const bool past = at >= hi || p.pairs[at].x >= diag - at;
      const uint32_t first = __ffs(__ballot_sync(kFull, past));
      if (first == 0) {
        lo = lo + step * 32;
      } else {
        const uint64_t top = lo + step * first - 1;
        lo = lo + step * (first - 1);
        hi = top < hi ? top : hi;
      }
    }
    c.i = static_cast<uint32_t>(lo);
  }
  c.r = ACC ? (c.i < p.n ? p.pairs[c.i].x : p.n_rows) : static_cast<uint32_t>(diag - c.i);
  c.mid = false;
  const uint32_t at = c.i + lane;                // (both loads at once: they only depend on c.i)
  const uint32_t in_front = c.i > 0 ? p.pairs[c.i - 1].x : kFull;
  const uint32_t behind = at < p.n ? p.pairs[at].x : kFull;
  if (c.r < p.n_rows && in_front == c.r) {
    const bool other = behind != c.r;
    const uint32_t first = __ffs(__ballot_sync(kFull, other));
    if (first == 0) {
      c.mid = true;
    } else {
      c.i += first - 1;
      c.r = ACC ? (c.i < p.n ? p.pairs[c.i].x : p.n_rows) : c.r + 1;
    }
  }
  return c;
}

template <typename TG, bool VEC>
__device__ __forceinline__ void clear_row(const SumParams& p, uint32_t row, uint32_t o) {
  store_row_octet<TG, VEC>(static_cast<TG*>(p.grad) + static_cast<uint64_t>(row) * p.grad_stride, o,
                           p.d, zero_octet<TG>());
}

// `count` consecutive elements, by a warp: single ones up to the first 16-byte boundary and behind
// the last one, whole pieces between.
template <typename TG>
__device__ __forceinline__ void clear_span(TG* at, uint64_t count) {
  constexpr uint32_t kPiece = 16 / sizeof(TG);
  const uint32_t lane = threadIdx.x & 31;
  uint32_t head = (kPiece - (reinterpret_cast<uintptr_t>(at) & 15) / sizeof(TG)) % kPiece;
  if (head > count) head = static_cast<uint32_t>(count);
  if (lane < head) at[lane] = from_f32<TG>(0.0f);
  at += head;
  count -= head;
  for (uint64_t i = lane; i < count / kPiece; i += 32)
    reinterpret_cast<uint4*>(at)[i] = make_uint4(0, 0, 0, 0);
  if (lane < count % kPiece) at[count - count % kPiece + lane] = from_f32<TG>(0.0f);
}

template <typename TG, bool VEC, bool ACC>
__device__ __forceinline__ void write_row(const SumParams& p, uint32_t row, uint32_t o,
                                          const float (&acc)[8]) {
  TG* g = static_cast<TG*>(p.grad) + static_cast<uint64_t>(row) * p.grad_stride;
  float v[8];
  if constexpr (ACC) {
    unpack<TG>(load_row_octet<TG, VEC>(g, o, p.d), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf(p.scale, acc[e], v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = p.scale * acc[e];
  }
  store_row_octet<TG, VEC>(g, o, p.d, pack<TG>(v));
}

__device__ __forceinline__ void store_part(float* part, uint32_t o, const float (&acc)[8]) {
  float4* to = reinterpret_cast<float4*>(part + 8 * o);
  to[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  to[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

template <typename TD, typename TG, bool VD, bool VG, bool ACC>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(SumParams p) {
  __shared__ Cut cuts[kWarps + 1];
  __shared__ uint32_t key_s[kWarps][kBatch + kAhead], pos_s[kWarps][kBatch + kAhead];
  extern __shared__ __align__(16) uint8_t ring[];  // [warp][kAhead][lane] octets
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_previous();
  // The CTA's warps find its chunks' cuts side by side: chunk0, chunk0 + 1, ..
  const uint64_t unit0 = static_cast<uint64_t>(blockIdx.x) * kWarps, unit = unit0 + warp;
  const uint32_t chunk0 = static_cast<uint32_t>(unit0 / p.slabs);
  const uint32_t chunk = static_cast<uint32_t>(unit / p.slabs);
  const uint32_t last = static_cast<uint32_t>((unit0 + kWarps - 1) / p.slabs);
  for (uint32_t k = warp; k <= last - chunk0 + 1; k += kWarps) {
    const uint64_t c = static_cast<uint64_t>(chunk0) + k;
    const Cut cut = c >= p.chunks ? Cut{p.n, p.n_rows, false} : find_cut<ACC>(p, c * p.per_chunk);
    if (lane == 0) cuts[k] = cut;
  }
  __syncthreads();
  if (chunk >= p.chunks) return;
  const uint32_t slab = static_cast<uint32_t>(unit - static_cast<uint64_t>(chunk) * p.slabs);
  const uint32_t o = slab * 32 + lane;
  const bool live = 8 * o < p.d;
  const Cut from = cuts[chunk - chunk0], to = cuts[chunk - chunk0 + 1];
  uint32_t cur = from.r;          // the row in progress
  bool begun = from.mid;          // whether it has parts in front of this chunk
  bool any = false;               // whether it has lookups in this chunk
  uint32_t head_row = kFull;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;

  const TD* dy = static_cast<const TD*>(p.dy);
  // Close row `cur` and move to row `next` (the rows between are named by no id).
  auto advance = [&](uint32_t next) {
    if (begun) {
      head_row = cur;
      if (live) store_part(p.head + chunk * p.pitch, o, acc);
    } else if (any) {
      if (live) write_row<TG, VG, ACC>(p, cur, o, acc);
    } else if (!ACC) {
      if (live) clear_row<TG, VG>(p, cur, o);
    }
    if constexpr (!ACC) {
      // (958,530 rows of 25 bf16 with 28,039 lookups: 67 us, 86 with dy loaded to registers, 116
      // with a row at a time by octets; 35,378 x 878 fp32 with 352: 34 against 49)
      TG* grad = static_cast<TG*>(p.grad);
      if (p.slabs == 1 && p.grad_stride == p.d) {
        if (next > cur + 1)
          clear_span<TG>(grad + static_cast<uint64_t>(cur + 1) * p.d,
                         static_cast<uint64_t>(next - cur - 1) * p.d);
      } else if (!VG && p.lanes_log2 == 5) {
        for (uint32_t r = cur + 1; r < next; ++r)
          clear_span<TG>(grad + r * p.grad_stride + slab * kSlab, min(p.d - slab * kSlab, kSlab));
      } else {                   // (narrow rows: a warp clears several at once)
        const uint32_t co = slab * 32 + (lane & ((1u << p.lanes_log2) - 1));
        if (8 * co < p.d)
          for (uint32_t r = cur + 1 + (lane >> p.lanes_log2); r < next; r += 32u >> p.lanes_log2)
            clear_row<TG, VG>(p, r, co);
      }
    }
    cur = next;
    begun = any = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  };

  // Lookups [i, i + batch) at a time: their ids and places go to shared memory, their dy rows
  // through a ring of copies to shared memory, kAhead - 1 in flight (copies complete in order,
  // group by group; register loads would share too few scoreboards to be waited for one by one).
  // A key of n_rows ends the list.
  constexpr uint32_t kOctet = 8 * sizeof(TD);
  constexpr uint32_t kRow = ring_row<TD, VD>();
  const uint8_t* mine = ring + warp * (kAhead * kRow) + lane * kOctet;
  const uint32_t mine_at = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  const bool copies = live || (!VD && o == (p.d + 7) / 8);
  uint32_t* keys = key_s[warp];
  uint32_t* places = pos_s[warp];
  bool done = false;
  for (uint32_t i = from.i; i < to.i && !done; i += kBatch) {
    __syncwarp();
    for (uint32_t k = lane; k < kBatch + kAhead; k += 32) {
      const bool in = k < kBatch && i + k < to.i;
      const uint2 pair = in ? p.pairs[i + k] : make_uint2(kFull, 0);
      keys[k] = pair.x;
      places[k] = p.group == 1 ? pair.y : pair.y / p.group;
    }
    __syncwarp();
    auto fetch = [&](uint32_t k) {
      if (copies && keys[k] < p.n_rows)
        copy_octet<TD, VD>(mine_at + k % kAhead * kRow,
                           dy + static_cast<uint64_t>(places[k]) * p.dy_stride, o, p.d, lane == 31);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (uint32_t u = 0; u < kAhead - 1; ++u) fetch(u);
    for (uint32_t k0 = 0; k0 < kBatch; ++k0) {
      if constexpr (!VD) __syncwarp();  // the neighbour has read what is overwritten now
      fetch(k0 + kAhead - 1);
      const uint32_t k = keys[k0];
      if (k >= p.n_rows) {              // the chunk's end, or an id outside: all that follow too
        done = true;
        break;
      }
      if (k != cur) advance(k);
      any = true;
      // the oldest copy has landed; a lane reads what it copied itself, and the word behind it
      // where rows lie off 16-byte boundaries
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
      if constexpr (!VD) __syncwarp();
      const Packed<TD> r =
          live ? copied_octet<TD, VD>(mine + k0 % kAhead * kRow,
                                      dy + static_cast<uint64_t>(places[k0]) * p.dy_stride)
               : zero_octet<TD>();
      float v[8];
      unpack<TD>(r, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += v[e];
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  let_next_start();        // (early, the next kernel's waiting CTAs would take this one's place)
  if (to.r > cur) advance(to.r);
  const bool left = any || begun;                 // a part of row `cur` that goes on
  if (left && to.mid && live) store_part(p.tail + chunk * p.pitch, o, acc);
  if (slab == 0 && lane == 0) {
    p.head_row[chunk] = head_row;
    p.end_key[chunk] = 2 * to.r + (left && to.mid ? 1u : 0u);
  }
}

constexpr int kJoinThreads = 256;
constexpr uint32_t kJoinChunks = 8;              // chunks that a CTA looks through

// Rows that span chunks: chunk c holds the last part, the chunks in front of it the
// earlier ones, from the one where the row began.  Eight warps take a contiguous share
// of the parts each; their sums are added in order.
template <typename TG, bool VEC, bool ACC>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(SumParams p) {
  __shared__ float part[kJoinThreads / 32][kSlab];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t o = blockIdx.y * 32 + lane;
  const bool live = 8 * o < p.d;
  wait_for_previous();
  {
    const uint32_t c0 = blockIdx.x * kJoinChunks;
    const uint32_t mine =
        lane < kJoinChunks && c0 + lane < p.chunks ? p.head_row[c0 + lane] : kFull;
    uint32_t todo = __ballot_sync(kFull, mine != kFull);
    while (todo != 0) {
      const uint32_t b = __ffs(todo) - 1;
      todo &= todo - 1;
      const uint32_t c = c0 + b, row = __shfl_sync(kFull, mine, b);
      // the first chunk that left a part of this row (end_key never falls), 33 parts a step
      uint32_t lo = 0, hi = c;
      while (lo < hi) {
        const uint32_t step = (hi - lo + 32) / 33;
        const uint32_t at = lo + step * (lane + 1) - 1;
        const bool past = at >= hi || p.end_key[at] >= 2 * row + 1;
        const uint32_t first = __ffs(__ballot_sync(kFull, past));
        if (first == 0) {
          lo += step * 32;
        } else {
          const uint32_t top = lo + step * first - 1;
          lo = lo + step * (first - 1);
          hi = top < hi ? top : hi;
        }
      }
      const uint32_t parts = c - lo;              // tails lo .. c-1, then the head of c
      const uint32_t share = (parts + 7) / 8;
      const uint32_t q0 = lo + (warp * share < parts ? warp * share : parts);
      const uint32_t q1 = lo + ((warp + 1) * share < parts ? (warp + 1) * share : parts);
      float acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
      if (live) {
#pragma unroll 8
        for (uint32_t q = q0; q < q1; ++q) {
          const float4* from = reinterpret_cast<const float4*>(p.tail + q * p.pitch + 8 * o);
          const float4 x = from[0], y = from[1];
          const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += v[e];
        }
      }
      *reinterpret_cast<float4*>(&part[warp][lane * 8]) =
          make_float4(acc[0], acc[1], acc[2], acc[3]);
      *reinterpret_cast<float4*>(&part[warp][lane * 8 + 4]) =
          make_float4(acc[4], acc[5], acc[6], acc[7]);
      __syncthreads();
      if (warp == 0 && live) {
        const float* last = p.head + c * p.pitch + 8 * o;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float s = acc[e];
          for (int w = 1; w < kJoinThreads / 32; ++w) s += part[w][lane * 8 + e];
          acc[e] = s + last[e];
        }
        write_row<TG, VEC, ACC>(p, row, o, acc);
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------------- host

constexpr uint64_t up(uint64_t x, uint64_t m) { return (x + m - 1) / m * m; }

struct Plan {
  int passes, bits;
  uint32_t tiles, per_tile;
  uint32_t chunks, per_chunk;
  uint64_t pairs[2], counts, totals, head, tail, head_row, end_key, total;
};

// Workspace of a call; accumulate or not, the larger list's chunks are planned for.
Plan plan(uint64_t n, uint64_t n_rows, uint32_t d, bool accumulate) {
  Plan w{};
  int nbits = 1;
  while (nbits < 32 && (n_rows >> nbits) != 0) ++nbits;    // n_rows itself is a key
  const int widest = n <= kSmallMax ? kSmallBits : kMaxBits;
  w.passes = (nbits + widest - 1) / widest;
  w.bits = (nbits + w.passes - 1) / w.passes;
  if (w.bits < 2) w.bits = 2;                              // (counts are read four at a time)
  const uint64_t subs = (n + kSub - 1) / kSub;
  const uint64_t per = (subs + kMaxTiles - 1) / kMaxTiles;
  w.per_tile = static_cast<uint32_t>((per == 0 ? 1 : per) * kSub);
  w.tiles = static_cast<uint32_t>(up((n + w.per_tile - 1) / w.per_tile, kTileCluster));
  const uint64_t items = accumulate ? n : n + n_rows;
  // A chunk of 64 items when there are enough of them to fill the warps, down to 4 when
  // there are few and their latency counts (64 lookups of 64 rows: 8.5 us against 10.1 with
  // 16; 4,096 of 4,096 x 256: 15.3 against 16.5; halving further at 196,608 lookups costs,
  // 77 us against 58 at d = 8); more when there are so many that the chunks' parts would
  // pass 268 MB of workspace.
  const uint64_t slabs = (d + kSlab - 1) / kSlab;
  uint64_t per_chunk = 64;
  while (per_chunk > 4 && items / per_chunk * slabs < 4096) per_chunk /= 2;
  while (items / per_chunk * slabs > (1u << 17)) per_chunk *= 2;
  const uint64_t chunks = items == 0 ? 1 : (items + per_chunk - 1) / per_chunk;
  w.per_chunk = static_cast<uint32_t>(per_chunk);
  w.chunks = static_cast<uint32_t>(chunks);
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += up(bytes, 256);
    return here;
  };
  for (int k = 0; k < 2; ++k) w.pairs[k] = take(8 * n);
  w.counts = take(4ull * w.tiles * kMaxBins);
  w.totals = take(4ull * w.tiles / kTileCluster * kMaxBins);
  const uint64_t pitch = up(d, 8);
  w.head = take(4 * chunks * pitch);
  w.tail = take(4 * chunks * pitch);
  w.head_row = take(4 * chunks);
  w.end_key = take(4 * chunks);
  w.total = at;
  return w;
}

template <typename TD, typename TG, bool ACC>
cudaError_t launch_sums(const SumParams& p, bool vd, bool vg, cudaStream_t s) {
  const uint64_t warps = static_cast<uint64_t>(p.chunks) * p.slabs;
  const uint64_t blocks = (warps * 32 + kSumThreads - 1) / kSumThreads;
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  auto* fn = vd ? (vg ? &sum_kernel<TD, TG, true, true, ACC> : &sum_kernel<TD, TG, true, false, ACC>)
                : (vg ? &sum_kernel<TD, TG, false, true, ACC>
                      : &sum_kernel<TD, TG, false, false, ACC>);
  const uint32_t smem = kWarps * kAhead * (vd ? ring_row<TD, true>() : ring_row<TD, false>());
  cudaError_t e = cudaSuccess;
  if (smem > 32768)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(fn),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess)
    e = launch_after(fn, dim3(static_cast<unsigned>(blocks)), kSumThreads, smem, s, p);
  if (e != cudaSuccess) return e;
  if (p.n <= 32) return e;       // a row spans chunks only with a lookup in front of a cut and 32 behind it
  auto* jn = vg ? &join_kernel<TG, true, ACC> : &join_kernel<TG, false, ACC>;
  return launch_after(jn, dim3((p.chunks + kJoinChunks - 1) / kJoinChunks, p.slabs), kJoinThreads, 0,
                      s, p);
}

template <typename TD, typename TG>
cudaError_t launch_sums(const SumParams& p, bool acc, bool vd, bool vg, cudaStream_t s) {
  return acc ? launch_sums<TD, TG, true>(p, vd, vg, s) : launch_sums<TD, TG, false>(p, vd, vg, s);
}

template <typename TD>
cudaError_t launch_sums(const SumParams& p, int grad_dtype, bool acc, bool vd, bool vg,
                        cudaStream_t s) {
  if (grad_dtype == CP_F32) return launch_sums<TD, float>(p, acc, vd, vg, s);
  if (grad_dtype == CP_F16) return launch_sums<TD, __half>(p, acc, vd, vg, s);
  return launch_sums<TD, __nv_bfloat16>(p, acc, vd, vg, s);
}

bool sizes_ok(uint64_t n, uint64_t n_rows, uint32_t d) {
  return d != 0 && d <= (1u << 20) && n < (1ull << 31) && n_rows < (1ull << 31);
}

}  // namespace

extern "C" uint64_t cp_embed_grad_workspace_bytes(uint64_t n, uint64_t n_rows, uint32_t d) {
  if (!sizes_ok(n, n_rows, d)) return 0;
  const uint64_t a = plan(n, n_rows, d, false).total, b = plan(n, n_rows, d, true).total;
  return a > b ? a : b;
}

extern "C" cp_status cp_embed_grad(const void* dy, int dy_dtype, uint64_t dy_stride,
                                   const int64_t* ids, uint64_t n, uint32_t group, uint64_t n_rows,
                                   uint32_t d, float scale, int accumulate, void* grad, int grad_dtype,
                                   uint64_t grad_stride, uint32_t* status, void* workspace,
                                   uint64_t workspace_bytes, void* stream) {
  if (!dtype_ok(dy_dtype) || !dtype_ok(grad_dtype) || !sizes_ok(n, n_rows, d) ||
      (dy_stride < d && dy_stride != 0) || grad_stride < d || (accumulate != 0 && accumulate != 1) ||
      group == 0 || n % group != 0) {
    cpx::set_error("bad dtype, n, group, n_rows, d, row stride or accumulate");
    return CP_ERR_INVALID_ARG;
  }
  if (n_rows == 0 && n == 0) return CP_OK;
  if (accumulate && n == 0) return CP_OK;
  const uint64_t ed = dtype_size(dy_dtype), eg = dtype_size(grad_dtype);
  if ((n != 0 && (dy == nullptr || ids == nullptr)) || (grad == nullptr && n_rows != 0) ||
      !cpx::aligned(dy, ed) || !cpx::aligned(grad, eg) || !cpx::aligned(ids, 8) ||
      !cpx::aligned(status, 4)) {
    cpx::set_error("null or misaligned dy, ids, grad or status");
    return CP_ERR_INVALID_ARG;
  }
  const Plan w = plan(n, n_rows, d, accumulate != 0);
  if (workspace == nullptr || !cpx::aligned(workspace, 16) || workspace_bytes < w.total) {
    cpx::set_error("workspace must be 16-byte aligned and hold cp_embed_grad_workspace_bytes bytes");
    return CP_ERR_INVALID_ARG;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto pairs = [&](uint64_t off) { return reinterpret_cast<uint2*>(ws + off); };
  auto words = [&](uint64_t off) { return reinterpret_cast<uint32_t*>(ws + off); };
  int last = 0;
  cudaError_t e = cudaSuccess;
  if (n != 0 && n <= kSmallMax) {
    e = launch(Launch{dim3(1), kSmallThreads, static_cast<size_t>(kSmallThreads / 32 << w.bits) * 2, s},
               &sort_small_kernel, ids, static_cast<uint32_t>(n), static_cast<uint32_t>(n_rows),
               w.passes, w.bits, pairs(w.pairs[0]), status);
  } else if (n != 0) {
    for (int pass = 0; pass < w.passes && e == cudaSuccess; ++pass) {
      SortPass p;
      p.ids = pass == 0 ? ids : nullptr;
      p.pairs = pairs(w.pairs[(pass + 1) & 1]);
      p.pairs_out = pairs(w.pairs[pass & 1]);
      p.counts = words(w.counts);
      p.totals = words(w.totals);
      p.n = static_cast<uint32_t>(n);
      p.n_rows = static_cast<uint32_t>(n_rows);
      p.per_tile = w.per_tile;
      p.shift = static_cast<uint32_t>(pass * w.bits);
      p.bits = w.bits;
      p.status = status;
      e = launch_after(&sort_count_kernel, dim3(w.tiles), kSortThreads, 0, s, p, kTileCluster);
      if (e == cudaSuccess)
        e = launch_after(&sort_place_kernel, dim3(w.tiles), kSortThreads,
                         (kSortThreads / 32 << w.bits) * 2, s, p);
      last = pass & 1;
    }
  }
  if (e != cudaSuccess) return cpx::cuda_fail(e, "embed gradient sort");
  if (n_rows == 0) return CP_OK;
  SumParams q{};
  q.pairs = pairs(w.pairs[last]);
  q.n = static_cast<uint32_t>(n);
  q.n_rows = static_cast<uint32_t>(n_rows);
  q.d = d;
  q.slabs = (d + kSlab - 1) / kSlab;
  while (q.lanes_log2 < 5 && (8u << q.lanes_log2) < d) ++q.lanes_log2;
  q.chunks = w.chunks;
  q.per_chunk = w.per_chunk;
  q.group = group;
  q.dy = dy;
  q.dy_stride = dy_stride;
  q.scale = scale;
  q.grad = grad;
  q.grad_stride = grad_stride;
  q.pitch = up(d, 8);
  q.head = reinterpret_cast<float*>(ws + w.head);
  q.tail = reinterpret_cast<float*>(ws + w.tail);
  q.head_row = words(w.head_row);
  q.end_key = words(w.end_key);
  const bool vd = octets_ok(dy, dy_stride, d, ed), vg = octets_ok(grad, grad_stride, d, eg);
  const bool acc = accumulate != 0;
  if (dy_dtype == CP_F32) e = launch_sums<float>(q, grad_dtype, acc, vd, vg, s);
  else if (dy_dtype == CP_F16) e = launch_sums<__half>(q, grad_dtype, acc, vd, vg, s);
  else e = launch_sums<__nv_bfloat16>(q, grad_dtype, acc, vd, vg, s);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "embed gradient sums");
  return CP_OK;
}

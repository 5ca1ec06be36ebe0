// cp_embed_grad.cu -- gradient of a table lookup by sorted ids (include/cp.h,
// cp_embed_grad).
//
//   grad[r] = scale * sum of dy[j] over the j with ids[j] = r
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
// Bound by memory: dy read once, grad written once.
#include <cstdint>

#include <cuda_runtime.h>

#include "cp.h"
#include "cp_internal.h"
#include "cp_layer.cuh"

namespace {

using namespace cpl;

constexpr uint32_t kFull = 0xFFFFFFFFu;

// ------------------------------------------------------------------------ sort

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kRounds = 4;                                   // keys per thread and sub-tile
constexpr uint32_t kSub = kSortThreads * kRounds;            // 4096 keys per sub-tile
constexpr uint32_t kMaxTiles = 512;
constexpr uint32_t kSmallMax = kSub;                         // one CTA's keys
constexpr int kMaxBits = 9;                                  // digit width
constexpr int kSmallBits = 8;                                // in one CTA (48 KB of shared memory)
constexpr uint32_t kMaxBins = 1u << kMaxBits;

__device__ __forceinline__ uint32_t key_of(int64_t id, uint32_t n_rows) {
  return static_cast<uint64_t>(id) < n_rows ? static_cast<uint32_t>(id) : n_rows;
}

// Ranks of a sub-tile's keys among the keys of the same digit, in order.  Warp w owns
// keys [w * 128, w * 128 + 128), 32 a round; `hist` [warp][bin] ends as the count of the
// bin in earlier warps, `total` as the sub-tile's counts.
struct Ranks {
  uint32_t r[kRounds];
};

__device__ __forceinline__ Ranks rank_digits(const uint32_t (&digit)[kRounds], uint32_t bins,
                                             uint16_t* hist, uint32_t* total) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint16_t* mine = hist + warp * bins;
  for (uint32_t b = lane; b < bins; b += 32) mine[b] = 0;
  __syncwarp();
  Ranks out;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const uint32_t d = digit[r];                 // bins: no key here
    const uint32_t peers = __match_any_sync(kFull, d);
    const uint32_t before = __popc(peers & ((1u << lane) - 1));
    uint32_t prior = 0;
    if (d < bins) prior = mine[d];
    __syncwarp();
    if (d < bins && before == 0) mine[d] = static_cast<uint16_t>(prior + __popc(peers));
    __syncwarp();
    out.r[r] = prior + before;
  }
  __syncthreads();
  for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads) {
    uint32_t sum = 0;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = hist[w * bins + b];
      hist[w * bins + b] = static_cast<uint16_t>(sum);
      sum += c;
    }
    total[b] = sum;
  }
  __syncthreads();
  return out;
}

// Exclusive prefix sums of v[0..bins), bins <= 512, by warp 0; all threads sync.
__device__ __forceinline__ void exclusive_scan(uint32_t* v, uint32_t bins) {
  if (threadIdx.x < 32) {
    const uint32_t lane = threadIdx.x;
    uint32_t carry = 0;
    for (uint32_t b = 0; b < bins; b += 32) {
      uint32_t x = b + lane < bins ? v[b + lane] : 0;
      const uint32_t own = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kFull, x, o);
        if (lane >= static_cast<uint32_t>(o)) x += y;
      }
      if (b + lane < bins) v[b + lane] = carry + x - own;
      carry += __shfl_sync(kFull, x, 31);
    }
  }
  __syncthreads();
}

// Up to kSmallMax ids in one CTA: all passes in shared memory.
__global__ void __launch_bounds__(kSortThreads)
    sort_small_kernel(const int64_t* __restrict__ ids, uint32_t n, uint32_t n_rows, int passes,
                      int bits, uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out,
                      uint32_t* status) {
  __shared__ uint32_t key_s[kSub];
  __shared__ uint16_t pos_s[kSub];
  extern __shared__ uint16_t hist[];             // [warps][bins]
  __shared__ uint32_t total[kMaxBins];
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
    const Ranks rk = rank_digits(digit, bins, hist, total);
    exclusive_scan(total, bins);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      if (digit[r] < bins) {
        const uint32_t to = total[digit[r]] + hist[warp * bins + digit[r]] + rk.r[r];
        if (p + 1 == passes) {
          keys_out[to] = key[r];
          pos_out[to] = pos[r];
        } else {
          key_s[to] = key[r];
          pos_s[to] = static_cast<uint16_t>(pos[r]);
        }
      }
    }
    __syncthreads();
    if (p + 1 < passes) {
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const uint32_t i = warp * (32 * kRounds) + r * 32 + lane;
        if (i < n) {
          key[r] = key_s[i];
          pos[r] = pos_s[i];
        } else {
          pos[r] = kFull;                        // no key: stays out of every digit
        }
      }
    }
    __syncthreads();
  }
}

struct SortPass {
  const int64_t* ids;            // first pass: the ids; else null
  const uint32_t* keys;          // later passes: pairs of the pass before
  const uint32_t* pos;
  uint32_t* keys_out;
  uint32_t* pos_out;
  uint32_t* counts;              // [tiles][bins]
  uint32_t n, n_rows, per_tile;  // per_tile: a multiple of kSub
  uint32_t shift, bits;
  uint32_t* status;
};

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortPass p) {
  __shared__ uint32_t hist[kMaxBins];
  const uint32_t bins = 1u << p.bits;
  for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads) hist[b] = 0;
  __syncthreads();
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
        key[r] = p.ids != nullptr ? key_of(p.ids[i], p.n_rows) : p.keys[i];
        bad |= key[r] == p.n_rows;
      }
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const bool have = key[r] != kFull;
      const uint32_t d = have ? (key[r] >> p.shift) & (bins - 1) : bins;
      const uint32_t peers = __match_any_sync(kFull, d);
      if (have && (peers & ((1u << (threadIdx.x & 31)) - 1)) == 0)
        atomicAdd(&hist[d], static_cast<uint32_t>(__popc(peers)));
    }
  }
  if (p.ids != nullptr && p.status != nullptr && bad) atomicOr(p.status, 1u);
  __syncthreads();
  for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads)
    p.counts[blockIdx.x * bins + b] = hist[b];
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortPass p) {
  extern __shared__ uint16_t hist[];             // [warps][bins]
  __shared__ uint32_t total[kMaxBins];
  __shared__ uint32_t base[kMaxBins];            // where this tile's next key of a digit goes
  __shared__ uint32_t part[kSortThreads], part_all[kSortThreads];
  const uint32_t bins = 1u << p.bits, tiles = gridDim.x, tile = blockIdx.x;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // counts of each digit before this tile and in all tiles: thread groups of `bins`
  // threads share the tiles, reading whole rows of counts
  {
    const uint32_t groups = kSortThreads / bins;           // bins <= 512: at least 2
    const uint32_t g = threadIdx.x / bins, b = threadIdx.x - g * bins;
    uint32_t before = 0, all = 0;
    if (g < groups) {
#pragma unroll 8
      for (uint32_t t = g; t < tiles; t += groups) {
        const uint32_t c = p.counts[t * bins + b];
        all += c;
        before += t < tile ? c : 0;
      }
    }
    part[threadIdx.x] = before;
    part_all[threadIdx.x] = all;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < bins; i += kSortThreads) {
      uint32_t x = 0, y = 0;
      for (uint32_t k = 0; k < groups; ++k) {
        x += part[k * bins + i];
        y += part_all[k * bins + i];
      }
      base[i] = x;
      total[i] = y;
    }
    __syncthreads();
    exclusive_scan(total, bins);
    for (uint32_t i = threadIdx.x; i < bins; i += kSortThreads) base[i] += total[i];
    __syncthreads();
  }
  const uint64_t lo = static_cast<uint64_t>(tile) * p.per_tile;
  const uint64_t hi = lo + p.per_tile < p.n ? lo + p.per_tile : p.n;
  for (uint64_t i0 = lo; i0 < hi; i0 += kSub) {
    uint32_t key[kRounds], pos[kRounds], digit[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const uint64_t i = i0 + warp * (32 * kRounds) + r * 32 + lane;
      digit[r] = bins;
      if (i < hi) {
        key[r] = p.ids != nullptr ? key_of(p.ids[i], p.n_rows) : p.keys[i];
        pos[r] = p.ids != nullptr ? static_cast<uint32_t>(i) : p.pos[i];
        digit[r] = (key[r] >> p.shift) & (bins - 1);
      }
    }
    const Ranks rk = rank_digits(digit, bins, hist, total);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      if (digit[r] < bins) {
        const uint32_t to = base[digit[r]] + hist[warp * bins + digit[r]] + rk.r[r];
        p.keys_out[to] = key[r];
        p.pos_out[to] = pos[r];
      }
    }
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads) base[b] += total[b];
    __syncthreads();
  }
}

// ------------------------------------------------------------------- sum and join

constexpr int kSumThreads = 256;
constexpr uint32_t kSlab = 256;                  // columns of a warp: an octet per lane
constexpr uint32_t kAhead = 8;                   // dy rows in flight per warp

struct SumParams {
  const uint32_t* keys;          // sorted; n_rows for ids outside the table
  const uint32_t* pos;
  uint32_t n, n_rows, d, slabs, chunks, per_chunk;
  const void* dy;
  uint64_t dy_stride;
  float scale;
  void* grad;
  uint64_t grad_stride;
  float* head;                   // [chunks][d]: a row's last part, where it began earlier
  float* tail;                   // [chunks][d]: a row's part, where it goes on
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
      const bool past = at >= hi || p.keys[at] >= diag - at;
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
  c.r = ACC ? (c.i < p.n ? p.keys[c.i] : p.n_rows) : static_cast<uint32_t>(diag - c.i);
  c.mid = false;
  if (c.r < p.n_rows && c.i > 0 && p.keys[c.i - 1] == c.r) {
    const uint32_t at = c.i + lane;
    const bool other = at >= p.n || p.keys[at] != c.r;
    const uint32_t first = __ffs(__ballot_sync(kFull, other));
    if (first == 0) {
      c.mid = true;
    } else {
      c.i += first - 1;
      c.r = ACC ? (c.i < p.n ? p.keys[c.i] : p.n_rows) : c.r + 1;
    }
  }
  return c;
}

template <typename TG, bool VEC>
__device__ __forceinline__ void clear_row(const SumParams& p, uint32_t row, uint32_t o) {
  store_row_octet<TG, VEC>(static_cast<TG*>(p.grad) + static_cast<uint64_t>(row) * p.grad_stride, o,
                           p.d, zero_octet<TG>());
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

__device__ __forceinline__ void store_part(float* part, uint32_t o, uint32_t d,
                                           const float (&acc)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (8 * o + e < d) part[8 * o + e] = acc[e];
}

template <typename TD, typename TG, bool VD, bool VG, bool ACC>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(SumParams p) {
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t unit = (static_cast<uint64_t>(blockIdx.x) * kSumThreads + threadIdx.x) >> 5;
  const uint32_t chunk = static_cast<uint32_t>(unit / p.slabs);
  if (chunk >= p.chunks) return;
  const uint32_t slab = static_cast<uint32_t>(unit - static_cast<uint64_t>(chunk) * p.slabs);
  const uint32_t o = slab * 32 + lane;
  const bool live = 8 * o < p.d;
  const Cut from = find_cut<ACC>(p, static_cast<uint64_t>(chunk) * p.per_chunk);
  const Cut to = chunk + 1 == p.chunks
                     ? Cut{p.n, p.n_rows, false}
                     : find_cut<ACC>(p, static_cast<uint64_t>(chunk + 1) * p.per_chunk);
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
      if (live) store_part(p.head + static_cast<uint64_t>(chunk) * p.d, o, p.d, acc);
    } else if (any) {
      if (live) write_row<TG, VG, ACC>(p, cur, o, acc);
    } else if (!ACC) {
      if (live) clear_row<TG, VG>(p, cur, o);
    }
    if constexpr (!ACC) {
      if (live)
        for (uint32_t r = cur + 1; r < next; ++r) clear_row<TG, VG>(p, r, o);
    }
    cur = next;
    begun = any = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  };

  uint32_t i = from.i;
  bool done = false;
  while (i < to.i && !done) {
    const uint32_t batch = to.i - i < 32 ? to.i - i : 32;
    uint32_t kk = p.n_rows, pp = 0;
    if (lane < batch) {
      kk = p.keys[i + lane];
      pp = p.pos[i + lane];
    }
    for (uint32_t t = 0; t < batch && !done; t += kAhead) {
      Packed<TD> r[kAhead];
#pragma unroll
      for (uint32_t u = 0; u < kAhead; ++u) {
        const uint32_t k = __shfl_sync(kFull, kk, t + u);
        const uint32_t j = __shfl_sync(kFull, pp, t + u);
        r[u] = live && k < p.n_rows
                   ? load_row_octet<TD, VD>(dy + static_cast<uint64_t>(j) * p.dy_stride, o, p.d)
                   : zero_octet<TD>();
      }
#pragma unroll
      for (uint32_t u = 0; u < kAhead; ++u) {
        const uint32_t k = __shfl_sync(kFull, kk, t + u);
        if (k >= p.n_rows) {      // past the batch, or an id outside the table: all that follow too
          if (t + u < batch) done = true;
        } else {
          if (k != cur) advance(k);
          any = true;
          float v[8];
          unpack<TD>(r[u], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += v[e];
        }
      }
    }
    i += batch;
  }
  if (to.r > cur) advance(to.r);
  const bool left = any || begun;                 // a part of row `cur` that goes on
  if (left && to.mid && live) store_part(p.tail + static_cast<uint64_t>(chunk) * p.d, o, p.d, acc);
  if (slab == 0 && lane == 0) {
    p.head_row[chunk] = head_row;
    p.end_key[chunk] = 2 * to.r + (left && to.mid ? 1u : 0u);
  }
}

constexpr int kJoinThreads = 256;
constexpr uint32_t kJoinChunks = 64;             // chunks that a CTA looks through

// Rows that span chunks: chunk c holds the last part, the chunks in front of it the
// earlier ones, from the one where the row began.  Eight warps take a contiguous share
// of the parts each; their sums are added in order.
template <typename TG, bool VEC, bool ACC>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(SumParams p) {
  __shared__ float part[kJoinThreads / 32][kSlab];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t o = blockIdx.y * 32 + lane;
  for (uint32_t k = 0; k < kJoinChunks; k += 32) {
    const uint32_t c0 = blockIdx.x * kJoinChunks + k;
    const uint32_t mine = c0 + lane < p.chunks ? p.head_row[c0 + lane] : kFull;
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
#pragma unroll 4
      for (uint32_t q = q0; q < q1; ++q) {
        const float* t = p.tail + static_cast<uint64_t>(q) * p.d;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (8 * o + e < p.d) acc[e] += t[8 * o + e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) part[warp][lane * 8 + e] = acc[e];
      __syncthreads();
      if (warp == 0 && 8 * o < p.d) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float s = acc[e];
          for (int w = 1; w < kJoinThreads / 32; ++w) s += part[w][lane * 8 + e];
          if (8 * o + e < p.d) s += p.head[static_cast<uint64_t>(c) * p.d + 8 * o + e];
          acc[e] = s;
        }
        write_row<TG, VEC, ACC>(p, row, o, acc);
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------------- host

uint64_t up(uint64_t x, uint64_t m) { return (x + m - 1) / m * m; }

struct Plan {
  int passes, bits;
  uint32_t tiles, per_tile;
  uint32_t chunks, per_chunk;
  uint64_t keys[2], pos[2], counts, head, tail, head_row, end_key, total;
};

// Workspace of a call; accumulate or not, the larger list's chunks are planned for.
Plan plan(uint64_t n, uint64_t n_rows, uint32_t d, bool accumulate) {
  Plan w{};
  int nbits = 1;
  while (nbits < 32 && (n_rows >> nbits) != 0) ++nbits;    // n_rows itself is a key
  const int widest = n <= kSmallMax ? kSmallBits : kMaxBits;
  w.passes = (nbits + widest - 1) / widest;
  w.bits = (nbits + w.passes - 1) / w.passes;
  const uint64_t subs = (n + kSub - 1) / kSub;
  const uint64_t per = (subs + kMaxTiles - 1) / kMaxTiles;
  w.per_tile = static_cast<uint32_t>((per == 0 ? 1 : per) * kSub);
  w.tiles = static_cast<uint32_t>((n + w.per_tile - 1) / w.per_tile);
  const uint64_t items = accumulate ? n : n + n_rows;
  // A chunk of 64 items when there are enough of them to fill the warps, down to 16
  // when there are few (their latency counts); more when there are so many that the
  // chunks' parts would pass 268 MB of workspace.
  const uint64_t slabs = (d + kSlab - 1) / kSlab;
  uint64_t per_chunk = 64;
  while (per_chunk > 16 && items / per_chunk * slabs < 4096) per_chunk /= 2;
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
  for (int k = 0; k < 2; ++k) {
    w.keys[k] = take(4 * n);
    w.pos[k] = take(4 * n);
  }
  w.counts = take(4ull * w.tiles * kMaxBins);
  w.head = take(4ull * chunks * d);
  w.tail = take(4ull * chunks * d);
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
  fn<<<static_cast<unsigned>(blocks), kSumThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  auto* jn = vg ? &join_kernel<TG, true, ACC> : &join_kernel<TG, false, ACC>;
  jn<<<dim3((p.chunks + kJoinChunks - 1) / kJoinChunks, p.slabs), kJoinThreads, 0, s>>>(p);
  return cudaGetLastError();
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
                                   const int64_t* ids, uint64_t n, uint64_t n_rows, uint32_t d,
                                   float scale, int accumulate, void* grad, int grad_dtype,
                                   uint64_t grad_stride, uint32_t* status, void* workspace,
                                   uint64_t workspace_bytes, void* stream) {
  if (!dtype_ok(dy_dtype) || !dtype_ok(grad_dtype) || !sizes_ok(n, n_rows, d) ||
      (dy_stride < d && dy_stride != 0) || grad_stride < d || (accumulate != 0 && accumulate != 1)) {
    cpx::set_error("bad dtype, n, n_rows, d, row stride or accumulate");
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
  auto words = [&](uint64_t off) { return reinterpret_cast<uint32_t*>(ws + off); };
  int last = 0;
  cudaError_t e = cudaSuccess;
  const size_t hist_bytes = (static_cast<size_t>(kSortWarps) << w.bits) * 2;
  if (n != 0 && n <= kSmallMax) {
    sort_small_kernel<<<1, kSortThreads, hist_bytes, s>>>(
        ids, static_cast<uint32_t>(n), static_cast<uint32_t>(n_rows), w.passes, w.bits,
        words(w.keys[0]), words(w.pos[0]), status);
    e = cudaGetLastError();
  } else if (n != 0) {
    for (int pass = 0; pass < w.passes && e == cudaSuccess; ++pass) {
      SortPass p;
      p.ids = pass == 0 ? ids : nullptr;
      p.keys = words(w.keys[(pass + 1) & 1]);
      p.pos = words(w.pos[(pass + 1) & 1]);
      p.keys_out = words(w.keys[pass & 1]);
      p.pos_out = words(w.pos[pass & 1]);
      p.counts = words(w.counts);
      p.n = static_cast<uint32_t>(n);
      p.n_rows = static_cast<uint32_t>(n_rows);
      p.per_tile = w.per_tile;
      p.shift = static_cast<uint32_t>(pass * w.bits);
      p.bits = static_cast<uint32_t>(w.bits);
      p.status = status;
      sort_count_kernel<<<w.tiles, kSortThreads, 0, s>>>(p);
      sort_place_kernel<<<w.tiles, kSortThreads, hist_bytes, s>>>(p);
      e = cudaGetLastError();
      last = pass & 1;
    }
  }
  if (e != cudaSuccess) return cpx::cuda_fail(e, "embed gradient sort");
  if (n_rows == 0) return CP_OK;
  SumParams q{};
  q.keys = words(w.keys[last]);
  q.pos = words(w.pos[last]);
  q.n = static_cast<uint32_t>(n);
  q.n_rows = static_cast<uint32_t>(n_rows);
  q.d = d;
  q.slabs = (d + kSlab - 1) / kSlab;
  q.chunks = w.chunks;
  q.per_chunk = w.per_chunk;
  q.dy = dy;
  q.dy_stride = dy_stride;
  q.scale = scale;
  q.grad = grad;
  q.grad_stride = grad_stride;
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

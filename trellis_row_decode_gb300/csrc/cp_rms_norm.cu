// cp_rms_norm.cu -- root-mean-square norm with the residual's addition, in the
// input's type or in 8 bits with scales, and its gradients (include/cp.h).
//
//   s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//   scales = amax |y| / 448 over 128 columns,  q = e4m3(y / scales)
//   dx = dres + r (t - n mean(t n)),  dw = sum over rows of dy n,  n = s r, t = dy w
//
// One pass: a row's octets stay in registers between the sum of squares and the
// scaling, so every array is read and written once and the kernels are bound by
// memory.  A team of 4 to 1024 threads (a few lanes of a warp, or a whole CTA) holds a
// row, up to kOct octets a thread; 16 neighbouring lanes hold one group of 128 columns,
// whose largest magnitude takes four shuffles.  A team walks over the rows: its part of
// the weight is loaded once, and a row's loads are issued before the row in front of it
// is summed, so the memory system is busy through the reductions.  Rows too wide for
// registers are read twice, the second time from the cache.
//
// 4096 x 4096 bf16: x and residual to h and e4m3 in 20.0 us (118 MB at 5.9 TB/s), the gradient in
// 28.3 us (134 MB at 4.7 TB/s, of it 3 us for the 5 MB of the CTAs' sums for dw).  One row of 1024:
// 2.2 us, a launch and two dependent trips to memory.
#include <cstdint>

#include <cuda_runtime.h>

#include "cp.h"
#include "cp_internal.h"
#include "cp_layer.cuh"

namespace {

using namespace cpl;

constexpr uint32_t kMaxD = 49152;      // the weight gradient's sums of one CTA: 192 KB

struct NormParams {
  const void* x;
  const void* residual;        // or null
  const void* weight;
  void* y;                     // null: the 8-bit output
  void* h;                     // with the residual
  uint8_t* q;
  float* scales;
  uint64_t x_stride, residual_stride;
  uint32_t rows, d;
  int weight_dtype;
  float eps;
};

// Sums `a` and `b` over the team's threads, in the same order on every thread.  Teams of more
// than a warp are whole CTAs; `red` alternates between two halves from row to row, so one
// barrier a row is enough.
template <int THREADS>
__device__ __forceinline__ void team_sum(float& a, float& b, float2* red) {
#pragma unroll
  for (int m = THREADS < 32 ? THREADS / 2 : 16; m > 0; m >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, m);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, m);
  }
  if constexpr (THREADS > 32) {
    constexpr int W = THREADS / 32;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 v = red[w];
      a += v.x;
      b += v.y;
    }
  }
}

// Eight weights of octet o (zeros past d).
template <bool VEC>
__device__ __forceinline__ void load_weight(const void* w, int dtype, uint32_t o, uint32_t d,
                                            float (&v)[8]) {
  if constexpr (VEC) {
    if (dtype == CP_F32)
      unpack<float>(load_octet(static_cast<const float*>(w) + 8ull * o), v);
    else if (dtype == CP_F16)
      unpack<__half>(load_octet(static_cast<const __half*>(w) + 8ull * o), v);
    else
      unpack<__nv_bfloat16>(load_octet(static_cast<const __nv_bfloat16*>(w) + 8ull * o), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 8 * o + e < d ? load_as_f32(w, 8 * o + e, dtype) : 0.0f;
  }
}

// One octet of s = x + residual.
template <typename T, bool VEC>
__device__ __forceinline__ void load_sum(const NormParams& p, const T* x, const T* res, uint32_t o,
                                         float (&v)[8]) {
  unpack<T>(load_row_octet<T, VEC>(x, o, p.d), v);
  if (res != nullptr) {
    float u[8];
    unpack<T>(load_row_octet<T, VEC>(res, o, p.d), u);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += u[e];
  }
}

// The octet's part of the output.  All lanes of the warp take part (the group's largest
// magnitude is shuffled among kGroup lanes: 16, or all of a team of fewer); `live`: the octet
// lies in a row.
template <typename T, bool VEC, bool Q, int kGroup = 16>
__device__ __forceinline__ void emit(const NormParams& p, uint64_t row, uint32_t o, bool live,
                                     float r, const float (&s)[8], const float (&w)[8]) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = s[e] * r * w[e];
  if (live && p.residual != nullptr)
    store_row_octet<T, VEC>(static_cast<T*>(p.h) + row * p.d, o, p.d, pack<T>(s));
  if constexpr (!Q) {
    if (live) store_row_octet<T, VEC>(static_cast<T*>(p.y) + row * p.d, o, p.d, pack<T>(y));
  } else {
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (live && (VEC || 8 * o + e < p.d)) amax = max(amax, mag_bits(y[e]));
#pragma unroll
    for (int m = kGroup / 2; m > 0; m >>= 1)
      amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, m));
    const float scale = scale_of(amax);
    if (live) {
      store_q_octet<VEC>(p.q + row * p.d, o, p.d, quantize_octet(y, __frcp_rn(scale)));
      if ((o & 15) == 0) p.scales[row * ((p.d + 127) / 128) + o / 16] = scale;
    }
  }
}

// Threads of a CTA of teams of `threads`, and CTAs that share an SM.
constexpr int cta_threads(int threads) { return threads <= 32 ? 256 : threads; }
constexpr int ctas_of(int sm_threads, int threads) {
  return sm_threads / cta_threads(threads) > 1 ? sm_threads / cta_threads(threads) : 1;
}
constexpr int norm_ctas(int threads) { return ctas_of(768, threads); }
constexpr int grad_ctas_per_sm(int threads) { return ctas_of(512, threads); }
constexpr bool norm_ring(int threads) { return threads == 1024 || threads <= 16; }

// Rows on octet boundaries travel through shared memory: a thread copies its own octets of the
// coming rows there (asynchronously, up to 216 KB an SM in all) and reads them back itself, so it
// waits for nobody and no registers hold what is under way.  Bytes of one row's octets of
// `arrays` arrays, and the rows that fit; one row or less: they wait in registers instead.
// Measured, 4096 x 4096 bf16: the gradient takes 28.4 us with three rows under way, 29.8 with
// four, 32.0 from registers; the forward, with fewer values to hold, 20.6 us from registers and
// 22.6 through shared memory, except in teams of 1024 (64 registers a thread; 1024 x 16384: 25.1
// against 28.4) and of a few lanes (100000 x 128: 17.0 against 18.3).
// Rows on other boundaries travel as the aligned 16-byte words that hold their bytes, one word more
// for each team or warp, and are shifted into place on the way back.  1707 x 4626 bf16: the
// gradient takes 30.1 us (64.8 with loads to registers), the forward 21.3; 19011 x 812: forward 36.2
// (51.9), gradient 38.8; 4096 x 4095 fp32: gradient 81 (116).
constexpr int lanes_of(int threads) { return threads < 32 ? threads : 32; }
template <typename T, bool VEC, int THREADS>
constexpr int array_bytes() {          // one array's octets, one of each thread of the CTA
  return cta_threads(THREADS) * 8 * static_cast<int>(sizeof(T)) +
         (VEC ? 0 : cta_threads(THREADS) / lanes_of(THREADS) * 16);
}
template <typename T, bool VEC, int THREADS>
constexpr int stage_bytes(int arrays, int oct) {
  return arrays * oct * array_bytes<T, VEC, THREADS>();
}
constexpr int kRingBytes = 216 << 10;    // of an SM
constexpr int stages_of(int ctas, int stage) {
  return kRingBytes / (ctas * stage) >= 3 ? 3 : kRingBytes / (ctas * stage);
}

// Where a thread's octets lie in an array of a stage.
template <typename T, bool VEC, int THREADS>
__device__ __forceinline__ uint32_t slot_of() {
  constexpr uint32_t kLanes = lanes_of(THREADS);
  return threadIdx.x * 8 * static_cast<uint32_t>(sizeof(T)) + (VEC ? 0 : threadIdx.x / kLanes * 16);
}

template <typename T, bool VEC, bool Q, int THREADS, int kOct>
__global__ void __launch_bounds__(cta_threads(THREADS), norm_ctas(THREADS)) norm_kernel(NormParams p) {
  constexpr int kTeams = cta_threads(THREADS) / THREADS;
  __shared__ float2 red[2][THREADS <= 32 ? 1 : THREADS / 32];
  const uint32_t tid = threadIdx.x % THREADS;
  const uint32_t octets = (p.d + 7) / 8;
  wait_for_previous();
  float w[kOct][8];
#pragma unroll
  for (int i = 0; i < kOct; ++i) {
    const uint32_t o = tid + i * THREADS;
    if (o < octets) {
      load_weight<VEC>(p.weight, p.weight_dtype, o, p.d, w[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = 0.0f;
    }
  }
  constexpr int kStage = stage_bytes<T, VEC, THREADS>(2, kOct);
  constexpr int kStages =
      !VEC || norm_ring(THREADS) ? stages_of(norm_ctas(THREADS), kStage) : 1;
  constexpr bool kRing = kStages >= 2;
  constexpr uint32_t kArray = array_bytes<T, VEC, THREADS>();
  const bool last = threadIdx.x % lanes_of(THREADS) == lanes_of(THREADS) - 1;
  extern __shared__ __align__(16) uint8_t ring[];
  uint8_t* mine_ring = ring + slot_of<T, VEC, THREADS>();
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(mine_ring));
  Packed<T> xn[kOct], rn[kOct];        // the next row (or, with the ring, this one)
  auto fetch = [&](uint64_t row, int stage) {
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
    const T* res = static_cast<const T*>(p.residual) + row * p.residual_stride;
#pragma unroll
    for (int i = 0; i < kOct; ++i) {
      const uint32_t o = tid + i * THREADS;
      const bool in = row < p.rows && o < octets;
      if constexpr (kRing) {
        const uint32_t at = ring_at + stage * kStage + 2 * i * kArray;
        if (in || (!VEC && row < p.rows && o == octets)) {
          copy_octet<T, VEC>(at, x, o, p.d, last);
          if (p.residual != nullptr) copy_octet<T, VEC>(at + kArray, res, o, p.d, last);
        }
      } else {
        xn[i] = in ? load_row_octet<T, VEC>(x, o, p.d) : zero_octet<T>();
        rn[i] = in && p.residual != nullptr ? load_row_octet<T, VEC>(res, o, p.d) : zero_octet<T>();
      }
    }
    if constexpr (kRing) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // (teams within a warp take their turns together: the shuffles are the warp's)
  const uint64_t lead = static_cast<uint64_t>(blockIdx.x) * kTeams +
                        (THREADS < 32 ? threadIdx.x / 32 * (32 / THREADS) : threadIdx.x / THREADS);
  const uint64_t mine = THREADS < 32 ? (threadIdx.x & 31) / THREADS : 0;
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * kTeams;
#pragma unroll
  for (int k = 0; k < (kRing ? kStages - 1 : 1); ++k) fetch(lead + mine + k * step, k);
  int turn = 0, stage = 0;
  for (uint64_t at = lead; at < p.rows; at += step, turn ^= 1) {
    const uint64_t row = at + mine;
    if constexpr (kRing) {
      if constexpr (!VEC) __syncwarp();        // the neighbour has read what is overwritten now
      fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      if constexpr (!VEC) __syncwarp();        // (a word behind an octet is the neighbour's copy)
      const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
      const T* res = static_cast<const T*>(p.residual) + row * p.residual_stride;
#pragma unroll
      for (int i = 0; i < kOct; ++i) {
        const bool in = row < p.rows && tid + i * THREADS < octets;
        const uint8_t* from = mine_ring + stage * kStage + 2 * i * kArray;
        xn[i] = in ? copied_octet<T, VEC>(from, x) : zero_octet<T>();
        rn[i] = in && p.residual != nullptr ? copied_octet<T, VEC>(from + kArray, res)
                                            : zero_octet<T>();
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    float s[kOct][8];
    float sq = 0.0f, unused = 0.0f;
#pragma unroll
    for (int i = 0; i < kOct; ++i) {
      unpack<T>(xn[i], s[i]);
      if (p.residual != nullptr) {
        float u[8];
        unpack<T>(rn[i], u);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[i][e] += u[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(s[i][e], s[i][e], sq);
    }
    if constexpr (!kRing) fetch(row + step, 0);
    team_sum<THREADS>(sq, unused, red[turn]);
    const float r = 1.0f / sqrtf(sq / static_cast<float>(p.d) + p.eps);
#pragma unroll
    for (int i = 0; i < kOct; ++i) {
      const uint32_t o = tid + i * THREADS;
      emit<T, VEC, Q, THREADS < 16 ? THREADS : 16>(p, row, o, row < p.rows && o < octets, r, s[i],
                                                   w[i]);
    }
  }
}

// Rows of any width: the second reading comes from the cache.
template <typename T, bool VEC, bool Q>
__global__ void __launch_bounds__(1024) norm_wide_kernel(NormParams p) {
  __shared__ float2 red[32];
  const uint64_t row = blockIdx.x;
  const uint32_t octets = (p.d + 7) / 8;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const T* res = p.residual != nullptr
                     ? static_cast<const T*>(p.residual) + row * p.residual_stride
                     : nullptr;
  float sq = 0.0f, unused = 0.0f;
  for (uint32_t o = threadIdx.x; o < octets; o += 1024) {
    float s[8];
    load_sum<T, VEC>(p, x, res, o, s);
#pragma unroll
    for (int e = 0; e < 8; ++e) sq = fmaf(s[e], s[e], sq);
  }
  team_sum<1024>(sq, unused, red);
  const float r = 1.0f / sqrtf(sq / static_cast<float>(p.d) + p.eps);
  for (uint32_t o0 = 0; o0 < octets; o0 += 1024) {
    const uint32_t o = o0 + threadIdx.x;
    float s[8] = {}, w[8] = {};
    if (o < octets) {
      load_sum<T, VEC>(p, x, res, o, s);
      load_weight<VEC>(p.weight, p.weight_dtype, o, p.d, w);
    }
    emit<T, VEC, Q>(p, row, o, o < octets, r, s, w);
  }
}

// ------------------------------------------------------------------------ gradient

struct GradParams {
  const void* dy;
  const void* h;
  const void* dres;            // or null
  const void* weight;
  void* dx;
  void* dw;
  float* parts;                // [gridDim.x][d]: each CTA's sums for dw
  uint64_t dy_stride, h_stride, dres_stride;
  uint32_t rows, d, ctas;
  int weight_dtype;
  float eps;
};

// dx = dres + r (t - n c), c = mean(t n).  (n = h r stays near one where r^2 would overflow: rows
// of a mean square below 2.9e-39, with eps as small.)
template <typename T, bool VEC>
__device__ __forceinline__ void emit_dx(const GradParams& p, uint64_t row, uint32_t o, float r,
                                        float c, const float (&t)[8], const float (&n)[8],
                                        const Packed<T>& res) {
  float dx[8];
  unpack<T>(res, dx);
#pragma unroll
  for (int e = 0; e < 8; ++e) dx[e] += r * (t[e] - n[e] * c);
  store_row_octet<T, VEC>(static_cast<T*>(p.dx) + row * p.d, o, p.d, pack<T>(dx));
}

// Teams walk over the rows; a thread's columns are the same in every row, so it sums its part
// of dw in registers, and the CTA's teams add theirs in order behind the last row.
template <typename T, bool VEC, int THREADS, int kOct>
__global__ void __launch_bounds__(cta_threads(THREADS), grad_ctas_per_sm(THREADS))
    norm_grad_kernel(GradParams p) {
  constexpr int kTeams = cta_threads(THREADS) / THREADS;
  __shared__ float2 red[2][THREADS <= 32 ? 1 : THREADS / 32];
  __shared__ float sums[kTeams == 1 ? 1 : THREADS * kOct * 8];
  const uint32_t tid = threadIdx.x % THREADS;
  const uint32_t octets = (p.d + 7) / 8;
  wait_for_previous();
  float w[kOct][8], dw[kOct][8];
#pragma unroll
  for (int i = 0; i < kOct; ++i) {
    const uint32_t o = tid + i * THREADS;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[i][e] = dw[i][e] = 0.0f;
    if (o < octets) load_weight<VEC>(p.weight, p.weight_dtype, o, p.d, w[i]);
  }
  constexpr int kStage = stage_bytes<T, VEC, THREADS>(3, kOct);
  constexpr int kStages = stages_of(grad_ctas_per_sm(THREADS), kStage);
  constexpr bool kRing = kStages >= 2;
  constexpr uint32_t kArray = array_bytes<T, VEC, THREADS>();
  const bool last = threadIdx.x % lanes_of(THREADS) == lanes_of(THREADS) - 1;
  extern __shared__ __align__(16) uint8_t ring[];
  uint8_t* mine_ring = ring + slot_of<T, VEC, THREADS>();
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(mine_ring));
  Packed<T> hn[kOct], gn[kOct], rn[kOct];          // the next row (or, with the ring, this one)
  auto fetch = [&](uint64_t row, int stage) {
    const T* h = static_cast<const T*>(p.h) + row * p.h_stride;
    const T* dy = static_cast<const T*>(p.dy) + row * p.dy_stride;
    const T* res = static_cast<const T*>(p.dres) + row * p.dres_stride;
#pragma unroll
    for (int i = 0; i < kOct; ++i) {
      const uint32_t o = tid + i * THREADS;
      const bool in = row < p.rows && o < octets;
      if constexpr (kRing) {
        const uint32_t at = ring_at + stage * kStage + 3 * i * kArray;
        if (in || (!VEC && row < p.rows && o == octets)) {
          copy_octet<T, VEC>(at, h, o, p.d, last);
          copy_octet<T, VEC>(at + kArray, dy, o, p.d, last);
          if (p.dres != nullptr) copy_octet<T, VEC>(at + 2 * kArray, res, o, p.d, last);
        }
      } else {
        hn[i] = in ? load_row_octet<T, VEC>(h, o, p.d) : zero_octet<T>();
        gn[i] = in ? load_row_octet<T, VEC>(dy, o, p.d) : zero_octet<T>();
      }
    }
    if constexpr (kRing) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto fetch_res = [&](uint64_t row) {
    const T* res = static_cast<const T*>(p.dres) + row * p.dres_stride;
#pragma unroll
    for (int i = 0; i < kOct; ++i) {
      const uint32_t o = tid + i * THREADS;
      rn[i] = row < p.rows && o < octets && p.dres != nullptr ? load_row_octet<T, VEC>(res, o, p.d)
                                                               : zero_octet<T>();
    }
  };
  const uint64_t lead = static_cast<uint64_t>(blockIdx.x) * kTeams +
                        (THREADS < 32 ? threadIdx.x / 32 * (32 / THREADS) : threadIdx.x / THREADS);
  const uint64_t mine = THREADS < 32 ? (threadIdx.x & 31) / THREADS : 0;
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * kTeams;
#pragma unroll
  for (int k = 0; k < (kRing ? kStages - 1 : 1); ++k) fetch(lead + mine + k * step, k);
  if constexpr (!kRing) fetch_res(lead + mine);
  int turn = 0, stage = 0;
  for (uint64_t at = lead; at < p.rows; at += step, turn ^= 1) {
    const uint64_t row = at + mine;
    if constexpr (kRing) {
      if constexpr (!VEC) __syncwarp();        // the neighbour has read what is overwritten now
      fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      if constexpr (!VEC) __syncwarp();        // (a word behind an octet is the neighbour's copy)
      const T* hr = static_cast<const T*>(p.h) + row * p.h_stride;
      const T* dyr = static_cast<const T*>(p.dy) + row * p.dy_stride;
      const T* res = static_cast<const T*>(p.dres) + row * p.dres_stride;
#pragma unroll
      for (int i = 0; i < kOct; ++i) {
        const bool in = row < p.rows && tid + i * THREADS < octets;
        const uint8_t* from = mine_ring + stage * kStage + 3 * i * kArray;
        hn[i] = in ? copied_octet<T, VEC>(from, hr) : zero_octet<T>();
        gn[i] = in ? copied_octet<T, VEC>(from + kArray, dyr) : zero_octet<T>();
        rn[i] = in && p.dres != nullptr ? copied_octet<T, VEC>(from + 2 * kArray, res)
                                        : zero_octet<T>();
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    float h[kOct][8], t[kOct][8];
    float sq = 0.0f, th = 0.0f;
#pragma unroll
    for (int i = 0; i < kOct; ++i) {
      unpack<T>(hn[i], h[i]);
      unpack<T>(gn[i], t[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sq = fmaf(h[i][e], h[i][e], sq);
        th = fmaf(t[i][e] * w[i][e], h[i][e], th);
      }
    }
    if constexpr (!kRing) fetch(row + step, 0);
    team_sum<THREADS>(sq, th, red[turn]);
    const float inv_d = 1.0f / static_cast<float>(p.d);
    const float r = 1.0f / sqrtf(sq * inv_d + p.eps);
    const float c = r * (th * inv_d);              // mean(t n) = r mean(t h)
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < kOct; ++i) {
        const uint32_t o = tid + i * THREADS;
        if (o < octets) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            h[i][e] *= r;                          // n
            dw[i][e] = fmaf(t[i][e], h[i][e], dw[i][e]);
            t[i][e] *= w[i][e];
          }
          emit_dx<T, VEC>(p, row, o, r, c, t[i], h[i], rn[i]);
        }
      }
    }
    if constexpr (!kRing) fetch_res(row + step);
  }
  let_next_start();
  float* part = p.parts + static_cast<uint64_t>(blockIdx.x) * p.d;
  if constexpr (kTeams == 1) {
#pragma unroll
    for (int i = 0; i < kOct; ++i) {
      const uint32_t o = tid + i * THREADS;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * o + e < p.d) part[8 * o + e] = dw[i][e];
    }
  } else {
    // columns lie by element first, so that neighbouring lanes have neighbouring words
    for (uint32_t team = 0; team < kTeams; ++team) {
      if (threadIdx.x / THREADS == team) {
#pragma unroll
        for (int i = 0; i < kOct; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float& s = sums[(i * 8 + e) * THREADS + tid];
            s = team == 0 ? dw[i][e] : s + dw[i][e];
          }
      }
      __syncthreads();
    }
    for (uint32_t c = threadIdx.x; c < p.d; c += cta_threads(THREADS)) {
      const uint32_t o = c / 8;
      part[c] = sums[(o / THREADS * 8 + c % 8) * THREADS + o % THREADS];
    }
  }
}

// Rows wider than the registers: read twice, dw summed in shared memory (each thread
// its own columns).
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) norm_grad_wide_kernel(GradParams p) {
  __shared__ float2 red[2][32];
  extern __shared__ float dw[];
  const uint32_t octets = (p.d + 7) / 8;
  for (uint32_t o = threadIdx.x; o < octets; o += 1024)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e * octets + o] = 0.0f;
  int turn = 0;
  for (uint64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const T* dyr = static_cast<const T*>(p.dy) + row * p.dy_stride;
    const T* hr = static_cast<const T*>(p.h) + row * p.h_stride;
    float sq = 0.0f, th = 0.0f;
    for (uint32_t o = threadIdx.x; o < octets; o += 1024) {
      float h[8], t[8], w[8];
      unpack<T>(load_row_octet<T, VEC>(hr, o, p.d), h);
      unpack<T>(load_row_octet<T, VEC>(dyr, o, p.d), t);
      load_weight<VEC>(p.weight, p.weight_dtype, o, p.d, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sq = fmaf(h[e], h[e], sq);
        th = fmaf(t[e] * w[e], h[e], th);
      }
    }
    team_sum<1024>(sq, th, red[turn]);
    const float inv_d = 1.0f / static_cast<float>(p.d);
    const float r = 1.0f / sqrtf(sq * inv_d + p.eps);
    const float c = r * (th * inv_d);              // mean(t n) = r mean(t h)
    for (uint32_t o = threadIdx.x; o < octets; o += 1024) {
      float h[8], t[8], w[8];
      unpack<T>(load_row_octet<T, VEC>(hr, o, p.d), h);
      unpack<T>(load_row_octet<T, VEC>(dyr, o, p.d), t);
      load_weight<VEC>(p.weight, p.weight_dtype, o, p.d, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[e] *= r;                                 // n
        dw[e * octets + o] = fmaf(t[e], h[e], dw[e * octets + o]);
        t[e] *= w[e];
      }
      emit_dx<T, VEC>(p, row, o, r, c, t, h,
                      p.dres != nullptr
                          ? load_row_octet<T, VEC>(
                                static_cast<const T*>(p.dres) + row * p.dres_stride, o, p.d)
                          : zero_octet<T>());
    }
  }
  let_next_start();
  float* part = p.parts + static_cast<uint64_t>(blockIdx.x) * p.d;
  for (uint32_t o = threadIdx.x; o < octets; o += 1024)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (8 * o + e < p.d) part[8 * o + e] = dw[e * octets + o];
}

constexpr int kDwThreads = 1024;

// dw[c] = sum of the CTAs' parts in order: 32 columns a CTA, 32 warps a contiguous share
// of the parts each.
__global__ void __launch_bounds__(kDwThreads) norm_dw_kernel(GradParams p) {
  __shared__ float sums[32][33];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t col = blockIdx.x * 32 + lane;
  const uint32_t share = (p.ctas + 31) / 32;
  const uint32_t lo = warp * share, hi = min(lo + share, p.ctas);
  float s = 0.0f;
  wait_for_previous();
  if (col < p.d) {
#pragma unroll 8
    for (uint32_t k = lo; k < hi; ++k) s += p.parts[static_cast<uint64_t>(k) * p.d + col];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < p.d) {
    for (int w = 1; w < 32; ++w) s += sums[w][lane];
    store_from_f32(p.dw, col, p.weight_dtype, s);
  }
}

// -------------------------------------------------------------------------- host

constexpr uint64_t kSms = 152;

// Dynamic shared memory of the ring, allowed for the kernel where it needs to be.
template <typename K>
cudaError_t allow_ring(K* kernel, int bytes) {
  return bytes <= 32768 ? cudaSuccess
                        : cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, bool VEC, bool Q, int THREADS, int kOct>
cudaError_t launch_teams(const NormParams& p, cudaStream_t s) {
  constexpr int kTeams = cta_threads(THREADS) / THREADS;
  constexpr int kStage = stage_bytes<T, VEC, THREADS>(2, kOct);
  constexpr int kStages =
      !VEC || norm_ring(THREADS) ? stages_of(norm_ctas(THREADS), kStage) : 1;
  constexpr int kBytes = kStages >= 2 ? kStages * kStage : 0;
  auto* kernel = &norm_kernel<T, VEC, Q, THREADS, kOct>;
  const cudaError_t e = allow_ring(kernel, kBytes);
  if (e != cudaSuccess) return e;
  const uint64_t ctas = (static_cast<uint64_t>(p.rows) + kTeams - 1) / kTeams;
  const uint64_t most = kSms * norm_ctas(THREADS);
  return launch_after(kernel, dim3(static_cast<unsigned>(ctas < most ? ctas : most)),
                      cta_threads(THREADS), kBytes, s, p);
}

// Teams just wide enough: 96, 192 and 384 threads between the powers of two keep more rows under
// way (bf16, 10900 x 1536: 19.8 us against 21.7; 6500 x 2560: 20.8 against 24.4; 2700 x 6144: 20.2
// against 25.5).
template <typename T, bool VEC, bool Q>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  const uint32_t octets = (p.d + 7) / 8;
  if (octets <= 4) return launch_teams<T, VEC, Q, 4, 1>(p, s);
  if (octets <= 8) return launch_teams<T, VEC, Q, 8, 1>(p, s);
  if (octets <= 16) return launch_teams<T, VEC, Q, 16, 1>(p, s);
  if (octets <= 32) return launch_teams<T, VEC, Q, 32, 1>(p, s);
  if (octets <= 64) return launch_teams<T, VEC, Q, 32, 2>(p, s);
  if (octets <= 128) return launch_teams<T, VEC, Q, 64, 2>(p, s);
  if (octets <= 192) return launch_teams<T, VEC, Q, 96, 2>(p, s);
  if (octets <= 256) return launch_teams<T, VEC, Q, 128, 2>(p, s);
  if (octets <= 384) return launch_teams<T, VEC, Q, 192, 2>(p, s);
  if (octets <= 512) return launch_teams<T, VEC, Q, 256, 2>(p, s);
  if (octets <= 768) return launch_teams<T, VEC, Q, 384, 2>(p, s);
  if (octets <= 1024) return launch_teams<T, VEC, Q, 512, 2>(p, s);
  if (octets <= 2048) return launch_teams<T, VEC, Q, 1024, 2>(p, s);
  norm_wide_kernel<T, VEC, Q><<<p.rows, 1024, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_norm(const NormParams& p, bool vec, cudaStream_t s) {
  if (p.y == nullptr)
    return vec ? launch_norm<T, true, true>(p, s) : launch_norm<T, false, true>(p, s);
  return vec ? launch_norm<T, true, false>(p, s) : launch_norm<T, false, false>(p, s);
}

template <typename T, bool VEC, int THREADS, int kOct>
cudaError_t launch_grad_teams(const GradParams& p, cudaStream_t s) {
  constexpr int kStage = stage_bytes<T, VEC, THREADS>(3, kOct);
  constexpr int kStages = stages_of(grad_ctas_per_sm(THREADS), kStage);
  constexpr int kBytes = kStages >= 2 ? kStages * kStage : 0;
  auto* kernel = &norm_grad_kernel<T, VEC, THREADS, kOct>;
  const cudaError_t e = allow_ring(kernel, kBytes);
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3(p.ctas), cta_threads(THREADS), kBytes, s, p);
}

template <typename T, bool VEC>
cudaError_t launch_rows(const GradParams& p, cudaStream_t s) {
  const uint32_t octets = (p.d + 7) / 8;
  if (octets <= 4) return launch_grad_teams<T, VEC, 4, 1>(p, s);
  if (octets <= 8) return launch_grad_teams<T, VEC, 8, 1>(p, s);
  if (octets <= 16) return launch_grad_teams<T, VEC, 16, 1>(p, s);
  if (octets <= 32) return launch_grad_teams<T, VEC, 32, 1>(p, s);
  if (octets <= 64) return launch_grad_teams<T, VEC, 32, 2>(p, s);
  if (octets <= 128) return launch_grad_teams<T, VEC, 64, 2>(p, s);
  if (octets <= 256) return launch_grad_teams<T, VEC, 128, 2>(p, s);
  if (octets <= 512) return launch_grad_teams<T, VEC, 256, 2>(p, s);
  if (octets <= 1024) return launch_grad_teams<T, VEC, 512, 2>(p, s);
  const int smem = static_cast<int>(octets * 32);
  auto* fn = &norm_grad_wide_kernel<T, VEC>;
  const cudaError_t e = allow_ring(fn, smem);
  if (e != cudaSuccess) return e;
  fn<<<p.ctas, 1024, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t launch_grad(const GradParams& p, cudaStream_t s) {
  const cudaError_t e = launch_rows<T, VEC>(p, s);
  if (e != cudaSuccess) return e;
  return launch_after(&norm_dw_kernel, dim3((p.d + 31) / 32), kDwThreads, 0, s, p);
}

// CTAs of a gradient call, each with its own sums for dw: those that fit on the card at once.
uint32_t grad_ctas(uint64_t rows, uint32_t d) {
  const uint32_t octets = (d + 7) / 8;
  uint32_t team = 4;
  while (team < 32 && team < octets) team *= 2;
  if (octets > 64) team = octets <= 128 ? 64 : octets <= 256 ? 128 : octets <= 512 ? 256 : octets <= 1024 ? 512 : 1024;
  const int threads = static_cast<int>(team);
  const uint64_t teams = cta_threads(threads) / threads;
  const uint64_t ctas = (rows + teams - 1) / teams, most = kSms * grad_ctas_per_sm(threads);
  return static_cast<uint32_t>(ctas < most ? ctas : most);
}

// Checks shared by the norms; writes whether whole octets can be moved.
cp_status norm_args(NormParams* p, const void* x, uint64_t x_stride, const void* residual,
                    uint64_t residual_stride, int dtype, const void* weight, int weight_dtype,
                    uint64_t rows, uint32_t d, float eps, const void* out, uint64_t out_align,
                    uint64_t out_vec, void* h, bool* vec) {
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype) || d == 0 || d > kMaxD || rows >= (1ull << 31) ||
      (x_stride < d && x_stride != 0) || !(eps >= 0.0f) ||
      (residual != nullptr && residual_stride < d && residual_stride != 0)) {
    cpx::set_error("bad dtype, rows, d, row stride or eps");
    return CP_ERR_INVALID_ARG;
  }
  if ((residual == nullptr) != (h == nullptr)) {
    cpx::set_error("residual and h go together");
    return CP_ERR_INVALID_ARG;
  }
  const uint64_t elt = dtype_size(dtype), welt = dtype_size(weight_dtype);
  if (rows != 0 && (x == nullptr || weight == nullptr || out == nullptr || !cpx::aligned(x, elt) ||
                    !cpx::aligned(residual, elt) || !cpx::aligned(h, elt) ||
                    !cpx::aligned(weight, welt) || !cpx::aligned(out, out_align))) {
    cpx::set_error("null or misaligned x, residual, weight or output");
    return CP_ERR_INVALID_ARG;
  }
  p->x = x;
  p->residual = residual;
  p->weight = weight;
  p->h = h;
  p->x_stride = x_stride;
  p->residual_stride = residual_stride;
  p->rows = static_cast<uint32_t>(rows);
  p->d = d;
  p->weight_dtype = weight_dtype;
  p->eps = eps;
  *vec = octets_ok(x, x_stride, d, elt) && octets_ok(weight, 0, d, welt) &&
         cpx::aligned(out, out_vec) &&
         (residual == nullptr ||
          (octets_ok(residual, residual_stride, d, elt) && octets_ok(h, d, d, elt)));
  return CP_OK;
}

cp_status run_norm(const NormParams& p, int dtype, bool vec, cudaStream_t s) {
  if (p.rows == 0) return CP_OK;
  cudaError_t e;
  if (dtype == CP_F32) e = launch_norm<float>(p, vec, s);
  else if (dtype == CP_F16) e = launch_norm<__half>(p, vec, s);
  else e = launch_norm<__nv_bfloat16>(p, vec, s);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "rms norm launch");
  return CP_OK;
}

}  // namespace

extern "C" cp_status cp_rms_norm(const void* x, uint64_t x_stride, const void* residual,
                                 uint64_t residual_stride, int dtype, const void* weight,
                                 int weight_dtype, uint64_t rows, uint32_t d, float eps, void* y,
                                 void* h, void* stream) {
  NormParams p{};
  bool vec = false;
  const uint64_t elt = dtype_ok(dtype) ? dtype_size(dtype) : 4;
  const cp_status st = norm_args(&p, x, x_stride, residual, residual_stride, dtype, weight,
                                 weight_dtype, rows, d, eps, y, elt, 8 * elt, h, &vec);
  if (st != CP_OK) return st;
  p.y = y;
  return run_norm(p, dtype, vec, static_cast<cudaStream_t>(stream));
}

extern "C" cp_status cp_rms_norm_fp8(const void* x, uint64_t x_stride, const void* residual,
                                     uint64_t residual_stride, int dtype, const void* weight,
                                     int weight_dtype, uint64_t rows, uint32_t d, float eps,
                                     uint8_t* q, float* scales, void* h, void* stream) {
  NormParams p{};
  bool vec = false;
  const cp_status st = norm_args(&p, x, x_stride, residual, residual_stride, dtype, weight,
                                 weight_dtype, rows, d, eps, q, 1, 8, h, &vec);
  if (st != CP_OK) return st;
  if (rows != 0 && (scales == nullptr || !cpx::aligned(scales, 4))) {
    cpx::set_error("null or misaligned scales");
    return CP_ERR_INVALID_ARG;
  }
  p.q = q;
  p.scales = scales;
  return run_norm(p, dtype, vec, static_cast<cudaStream_t>(stream));
}

extern "C" uint64_t cp_rms_norm_grad_workspace_bytes(uint64_t rows, uint32_t d) {
  if (d == 0 || d > kMaxD || rows >= (1ull << 31)) return 0;
  const uint64_t bytes = 4ull * grad_ctas(rows, d) * d;
  return bytes == 0 ? 16 : bytes;
}

extern "C" cp_status cp_rms_norm_grad(const void* dy, uint64_t dy_stride, const void* h,
                                      uint64_t h_stride, const void* dres, uint64_t dres_stride,
                                      int dtype, const void* weight, int weight_dtype,
                                      uint64_t rows, uint32_t d, float eps, void* dx, void* dw,
                                      void* workspace, uint64_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype) || d == 0 || d > kMaxD || rows >= (1ull << 31) ||
      (dy_stride < d && dy_stride != 0) || (h_stride < d && h_stride != 0) ||
      (dres != nullptr && dres_stride < d && dres_stride != 0) || !(eps >= 0.0f)) {
    cpx::set_error("bad dtype, rows, d, row stride or eps");
    return CP_ERR_INVALID_ARG;
  }
  const uint64_t elt = dtype_size(dtype), welt = dtype_size(weight_dtype);
  if (dw == nullptr || !cpx::aligned(dw, welt) ||
      (rows != 0 && (dy == nullptr || h == nullptr || weight == nullptr || dx == nullptr ||
                     !cpx::aligned(dy, elt) || !cpx::aligned(h, elt) || !cpx::aligned(dres, elt) ||
                     !cpx::aligned(dx, elt) || !cpx::aligned(weight, welt)))) {
    cpx::set_error("null or misaligned dy, h, dres, weight, dx or dw");
    return CP_ERR_INVALID_ARG;
  }
  if (workspace == nullptr || !cpx::aligned(workspace, 16) ||
      workspace_bytes < cp_rms_norm_grad_workspace_bytes(rows, d)) {
    cpx::set_error(
        "workspace must be 16-byte aligned and hold cp_rms_norm_grad_workspace_bytes bytes");
    return CP_ERR_INVALID_ARG;
  }
  GradParams p{};
  p.dy = dy;
  p.h = h;
  p.dres = dres;
  p.weight = weight;
  p.dx = dx;
  p.dw = dw;
  p.parts = static_cast<float*>(workspace);
  p.dy_stride = dy_stride;
  p.h_stride = h_stride;
  p.dres_stride = dres_stride;
  p.rows = static_cast<uint32_t>(rows);
  p.d = d;
  p.ctas = grad_ctas(rows, d);
  p.weight_dtype = weight_dtype;
  p.eps = eps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (rows == 0) {
    norm_dw_kernel<<<(d + 31) / 32, kDwThreads, 0, s>>>(p);      // no parts: zeros
    e = cudaGetLastError();
  } else {
    const bool vec = octets_ok(dy, dy_stride, d, elt) && octets_ok(h, h_stride, d, elt) &&
                     octets_ok(dx, d, d, elt) && octets_ok(weight, 0, d, welt) &&
                     (dres == nullptr || octets_ok(dres, dres_stride, d, elt));
    if (dtype == CP_F32)
      e = vec ? launch_grad<float, true>(p, s) : launch_grad<float, false>(p, s);
    else if (dtype == CP_F16)
      e = vec ? launch_grad<__half, true>(p, s) : launch_grad<__half, false>(p, s);
    else
      e = vec ? launch_grad<__nv_bfloat16, true>(p, s) : launch_grad<__nv_bfloat16, false>(p, s);
  }
  if (e != cudaSuccess) return cpx::cuda_fail(e, "rms norm gradient launch");
  return CP_OK;
}

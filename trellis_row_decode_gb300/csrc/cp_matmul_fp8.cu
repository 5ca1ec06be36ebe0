// cp_matmul_fp8.cu -- product of e4m3 matrices with a scale for each block of 128
// (include/cp.h, cp_matmul_fp8).
//
//   out[i][j] = sum over g of sa[i][g] sw[j / 128][g] * (a[i] . w[j] over group g)
//
// The products of a group are exact in the tensor core's fp32 sums; a group's sum is
// scaled and added to the running fp32 sum before the next group begins.
#include <cstdint>

#include <cuda_runtime.h>

#include "cp.h"
#include "cp_internal.h"
#include "cp_layer.cuh"

namespace {

using namespace cpl;

struct MatmulParams {
  const uint8_t* a;
  const float* sa;
  const uint8_t* w;
  const float* sw;
  void* out;
  uint64_t lda, ldw, ldo;
  uint32_t m, n, k, groups;
  int out_dtype;
};

// ---------------------------------------------------- rows on any byte boundary

constexpr int kTile = 64;              // rows of a and of w per CTA
constexpr int kPitch = 144;            // shared row pitch: fragment reads without conflicts
constexpr int kAnyThreads = 128;
constexpr int kWords = kTile * 32 / kAnyThreads;   // 4-byte words a thread stages per operand

// d = a (16 x 32) * b (32 x 8) + d on the tensor core, e4m3 operands.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// This thread's words of rows [row0, row0 + 64), columns [k0, k0 + 128); zeros outside
// the matrix.  ALIGNED: rows on 4-byte boundaries.
template <bool ALIGNED>
__device__ __forceinline__ void stage_load(uint32_t (&v)[kWords], const uint8_t* base, uint64_t ld,
                                           uint32_t row0, uint32_t rows, uint32_t k0, uint32_t k) {
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    const uint32_t idx = threadIdx.x + i * kAnyThreads;
    const uint32_t row = row0 + idx / 32, col = k0 + (idx % 32) * 4;
    uint32_t x = 0;
    if (row < rows && col < k) {
      const uint8_t* p = base + row * ld + col;
      if (ALIGNED && col + 4 <= k) {
        x = *reinterpret_cast<const uint32_t*>(p);
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (col + b < k) x |= static_cast<uint32_t>(p[b]) << (8 * b);
      }
    }
    v[i] = x;
  }
}

__device__ __forceinline__ void stage_store(uint8_t* tile, const uint32_t (&v)[kWords]) {
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    const uint32_t idx = threadIdx.x + i * kAnyThreads;
    *reinterpret_cast<uint32_t*>(tile + (idx / 32) * kPitch + (idx % 32) * 4) = v[i];
  }
}

// 64 x 64 outputs per CTA, four warps of 32 x 32; the next group's words are loaded
// into registers while the tensor core works on this one's.
template <bool ALIGNED>
__global__ void __launch_bounds__(kAnyThreads) matmul_any_kernel(MatmulParams p) {
  __shared__ __align__(16) uint8_t ta[kTile * kPitch];
  __shared__ __align__(16) uint8_t tw[kTile * kPitch];
  const uint32_t tiles_n = (p.n + kTile - 1) / kTile;
  const uint32_t row0 = blockIdx.x / tiles_n * kTile, col0 = blockIdx.x % tiles_n * kTile;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t wr = (warp >> 1) * 32, wc = (warp & 1) * 32;
  const uint32_t g = lane >> 2, t = lane & 3;
  float acc[2][4][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
  uint32_t va[kWords], vw[kWords];
  stage_load<ALIGNED>(va, p.a, p.lda, row0, p.m, 0, p.k);
  stage_load<ALIGNED>(vw, p.w, p.ldw, col0, p.n, 0, p.k);
  const float* sw = p.sw + static_cast<uint64_t>(col0 / 128) * p.groups;
  for (uint32_t kb = 0; kb < p.groups; ++kb) {
    __syncthreads();
    stage_store(ta, va);
    stage_store(tw, vw);
    __syncthreads();
    if (kb + 1 < p.groups) {
      stage_load<ALIGNED>(va, p.a, p.lda, row0, p.m, (kb + 1) * 128, p.k);
      stage_load<ALIGNED>(vw, p.w, p.ldw, col0, p.n, (kb + 1) * 128, p.k);
    }
    float c[2][4][4] = {};
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t fa[2][4], fb[4][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* q = ta + (wr + 16 * i + g) * kPitch + ks * 32 + t * 4;
        fa[i][0] = *reinterpret_cast<const uint32_t*>(q);
        fa[i][1] = *reinterpret_cast<const uint32_t*>(q + 8 * kPitch);
        fa[i][2] = *reinterpret_cast<const uint32_t*>(q + 16);
        fa[i][3] = *reinterpret_cast<const uint32_t*>(q + 8 * kPitch + 16);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* q = tw + (wc + 8 * j + g) * kPitch + ks * 32 + t * 4;
        fb[j][0] = *reinterpret_cast<const uint32_t*>(q);
        fb[j][1] = *reinterpret_cast<const uint32_t*>(q + 16);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_e4m3(c[i][j], fa[i], fb[j][0], fb[j][1]);
    }
    const float scale_w = __ldg(sw + kb);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t row = row0 + wr + 16 * i + 8 * half + g;
        const float f =
            row < p.m ? __ldg(p.sa + static_cast<uint64_t>(row) * p.groups + kb) * scale_w : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            acc[i][j][2 * half + e] = fmaf(f, c[i][j][2 * half + e], acc[i][j][2 * half + e]);
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t row = row0 + wr + 16 * i + 8 * (e >> 1) + g;
        const uint32_t col = col0 + wc + 8 * j + 2 * t + (e & 1);
        if (row < p.m && col < p.n)
          store_from_f32(p.out, row * p.ldo + col, p.out_dtype, acc[i][j][e]);
      }
}

}  // namespace

extern "C" cp_status cp_matmul_fp8(const uint8_t* a, uint64_t a_stride, const float* a_scales,
                                   const uint8_t* w, uint64_t w_stride, const float* w_scales,
                                   uint64_t m, uint64_t n, uint64_t k, void* out, int out_dtype,
                                   uint64_t out_stride, void* stream) {
  constexpr uint64_t kMost = 1ull << 31;
  if (!dtype_ok(out_dtype) || m >= kMost || n >= kMost || k >= kMost - 128 || out_stride < n ||
      (a_stride < k && a_stride != 0) || (w_stride < k && w_stride != 0)) {
    cpx::set_error("bad out_dtype, m, n, k or row stride");
    return CP_ERR_INVALID_ARG;
  }
  if (m == 0 || n == 0) return CP_OK;
  if (out == nullptr || !cpx::aligned(out, dtype_size(out_dtype)) ||
      (k != 0 && (a == nullptr || w == nullptr || a_scales == nullptr || w_scales == nullptr ||
                  !cpx::aligned(a_scales, 4) || !cpx::aligned(w_scales, 4)))) {
    cpx::set_error("null or misaligned a, w, scales or out");
    return CP_ERR_INVALID_ARG;
  }
  MatmulParams p{a,
                 a_scales,
                 w,
                 w_scales,
                 out,
                 a_stride,
                 w_stride,
                 out_stride,
                 static_cast<uint32_t>(m),
                 static_cast<uint32_t>(n),
                 static_cast<uint32_t>(k),
                 static_cast<uint32_t>((k + 127) / 128),
                 out_dtype};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint64_t tiles = ((m + kTile - 1) / kTile) * ((n + kTile - 1) / kTile);
  if (tiles >= kMost) {
    cpx::set_error("m and n make more than 2^31 tiles");
    return CP_ERR_INVALID_ARG;
  }
  const bool words = cpx::aligned(a, 4) && cpx::aligned(w, 4) && a_stride % 4 == 0 &&
                     w_stride % 4 == 0;
  auto* fn = words ? &matmul_any_kernel<true> : &matmul_any_kernel<false>;
  fn<<<static_cast<unsigned>(tiles), kAnyThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul launch");
  return CP_OK;
}

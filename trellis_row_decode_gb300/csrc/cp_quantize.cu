// cp_quantize.cu -- values to e4m3 with a scale for each block (include/cp.h,
// cp_quantize_fp8).
//
//   scale = max(amax |x|, 1e-30) / 448 over a block,  q = e4m3(x * (1 / scale))
//
// Read once, written once: a block's values stay in registers between its largest
// magnitude and the conversion.  Blocks of one row: 16 lanes hold a group of 128
// columns, a half warp takes four groups at a time so that four loads are in flight.
// Blocks of 128 rows: one CTA holds the 128 x 128 block, eight octets a thread.  Four such CTAs
// an SM for 16-bit inputs (64 registers): 4096 x 24576 bf16 takes 47 us (6.4 TB/s), against 60 us
// with three; with five the registers spill (56 us).
#include <cstdint>

#include <cuda_runtime.h>

#include "cp.h"
#include "cp_internal.h"
#include "cp_layer.cuh"

namespace {

using namespace cpl;

constexpr int kThreads = 256;
constexpr int kGroups = 4;         // groups of a half warp

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    quantize_rows_kernel(const T* x, uint64_t stride, uint32_t d, uint32_t per_row,
                         uint32_t groups, uint8_t* q, float* scales) {
  const uint32_t sub = threadIdx.x & 15;
  // (below 2^29: at most 2^31 groups; the thread's own index would pass 32 bits)
  const uint32_t half = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
  wait_for_previous();
  Packed<T> r[kGroups];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const uint32_t g = half * kGroups + i;
    const uint32_t row = g / per_row, o = (g - row * per_row) * 16 + sub;
    r[i] = g < groups && 8 * o < d ? load_row_octet<T, VEC>(x + row * stride, o, d)
                                   : zero_octet<T>();
  }
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const uint32_t g = half * kGroups + i;
    const uint32_t row = g / per_row, o = (g - row * per_row) * 16 + sub;
    float v[8];
    unpack<T>(r[i], v);
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max(amax, mag_bits(v[e]));
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, m));
    const float scale = scale_of(amax);
    if (g < groups) {
      if (8 * o < d)
        store_q_octet<VEC>(q + static_cast<uint64_t>(row) * d, o, d,
                           quantize_octet(v, __frcp_rn(scale)));
      if (sub == 0) scales[g] = scale;
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
    quantize_block_kernel(const T* x, uint64_t stride, uint64_t rows, uint32_t d,
                          uint32_t per_row, uint8_t* q, float* scales) {
  __shared__ uint32_t red[kThreads / 32];
  const uint32_t bi = blockIdx.x / per_row, bj = blockIdx.x - bi * per_row;
  const uint32_t o = bj * 16 + (threadIdx.x & 15);
  const uint64_t row0 = 128ull * bi + (threadIdx.x >> 4);
  wait_for_previous();
  Packed<T> r[8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t row = row0 + 16 * i;
    r[i] = row < rows && 8 * o < d ? load_row_octet<T, VEC>(x + row * stride, o, d)
                                   : zero_octet<T>();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack<T>(r[i], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max(amax, mag_bits(v[e]));
  }
  amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = max(amax, red[w]);
  const float scale = scale_of(amax), inv = __frcp_rn(scale);
  if (threadIdx.x == 0) scales[blockIdx.x] = scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t row = row0 + 16 * i;
    if (row < rows && 8 * o < d) {
      float v[8];
      unpack<T>(r[i], v);
      store_q_octet<VEC>(q + row * d, o, d, quantize_octet(v, inv));
    }
  }
}

template <typename T>
cudaError_t launch_quantize(const void* x, uint64_t stride, uint64_t rows, uint32_t d, uint32_t block_rows,
                   uint8_t* q, float* scales, cudaStream_t s) {
  const uint32_t per_row = static_cast<uint32_t>((static_cast<uint64_t>(d) + 127) / 128);
  const uint32_t blocks = static_cast<uint32_t>((rows + block_rows - 1) / block_rows) * per_row;
  const bool vec = octets_ok(x, stride, d, sizeof(T)) && cpx::aligned(q, 8);
  const T* p = static_cast<const T*>(x);
  if (block_rows == 1) {
    const uint32_t per_cta = kThreads / 16 * kGroups;
    auto* fn = vec ? &quantize_rows_kernel<T, true> : &quantize_rows_kernel<T, false>;
    return launch(Launch{dim3((blocks - 1) / per_cta + 1), kThreads, 0, s}, fn, p, stride, d,
                  per_row, blocks, q, scales);
  }
  auto* fn = vec ? &quantize_block_kernel<T, true> : &quantize_block_kernel<T, false>;
  return launch(Launch{dim3(blocks), kThreads, 0, s}, fn, p, stride, rows, d, per_row, q, scales);
}

}  // namespace

extern "C" cp_status cp_quantize_fp8(const void* x, uint64_t x_stride, int dtype, uint64_t rows,
                                     uint32_t d, uint32_t block_rows, uint8_t* q, float* scales,
                                     void* stream) {
  const uint64_t per_row = (static_cast<uint64_t>(d) + 127) / 128;
  if (!dtype_ok(dtype) || (block_rows != 1 && block_rows != 128) ||
      (x_stride < d && x_stride != 0) || rows >= (1ull << 40) ||
      (rows + block_rows - 1) / block_rows * per_row >= (1ull << 31)) {
    cpx::set_error("bad dtype, block_rows, row stride or more than 2^31 blocks");
    return CP_ERR_INVALID_ARG;
  }
  if (rows == 0 || d == 0) return CP_OK;
  if (x == nullptr || q == nullptr || scales == nullptr || !cpx::aligned(x, dtype_size(dtype)) ||
      !cpx::aligned(scales, 4)) {
    cpx::set_error("null or misaligned x, q or scales");
    return CP_ERR_INVALID_ARG;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == CP_F32) e = launch_quantize<float>(x, x_stride, rows, d, block_rows, q, scales, s);
  else if (dtype == CP_F16) e = launch_quantize<__half>(x, x_stride, rows, d, block_rows, q, scales, s);
  else e = launch_quantize<__nv_bfloat16>(x, x_stride, rows, d, block_rows, q, scales, s);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "quantize launch");
  return CP_OK;
}

// cp_dropout.cu -- dropout from a counter-based generator, with the residual's addition
// (include/cp.h, cp_dropout).
//
//   out[i][j] = rn(residual[i][j] + D(x)[i][j])
//
// An octet a thread: two calls of the generator.  Bound by memory (x and the residual read, out
// written).
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "cp.h"
#include "cp_epilogue.cuh"
#include "cp_internal.h"
#include "cp_layer.cuh"

namespace {

using namespace cpl;
using cpe::DropKey;

constexpr int kThreads = 256;
constexpr int kAhead = 2;                  // octets whose loads a thread has in flight
constexpr uint64_t kMostCtas = 152 * 8;

struct DropoutParams {
  const void* x;
  const void* residual;
  void* out;
  uint64_t ldx, ldr, ldo, rows;
  uint32_t d, octets;                      // octets of a row
  uint32_t step_rows, step_octets;         // what one step of the grid comes to
  cpe::DropParams drop;
};

template <typename T, bool VEC, bool kResidual>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutParams p) {
  wait_for_previous();
  let_next_start();
  const DropKey key = cpe::drop_key(p.drop);
  const cpe::RoundKeys keys = cpe::round_keys(key);
  // (row, octet) moves on by the grid's step without a division
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  uint64_t row = first / p.octets;
  uint32_t o = static_cast<uint32_t>(first - row * p.octets);
  while (row < p.rows) {
    Packed<T> x[kAhead], r[kAhead];
    uint64_t at[kAhead];
    uint32_t col[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      at[i] = row;
      col[i] = o;
      if (row < p.rows) {
        x[i] = load_row_octet<T, VEC>(static_cast<const T*>(p.x) + row * p.ldx, o, p.d);
        if constexpr (kResidual)
          r[i] = load_row_octet<T, VEC>(static_cast<const T*>(p.residual) + row * p.ldr, o, p.d);
      }
      o += p.step_octets;
      row += p.step_rows;
      if (o >= p.octets) {
        o -= p.octets;
        ++row;
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (at[i] < p.rows) {
        float v[8];
        unpack(x[i], v);
        if (p.drop.mode != 0) {
          const uint32_t line = static_cast<uint32_t>(at[i]);
          cpe::drop_quad(p.drop, key, keys, 2 * col[i], line, v);
          cpe::drop_quad(p.drop, key, keys, 2 * col[i] + 1, line, v + 4);
        }
        if constexpr (kResidual) {
          float w[8];
          unpack(r[i], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += w[e];
        }
        store_row_octet<T, VEC>(static_cast<T*>(p.out) + at[i] * p.ldo, col[i], p.d, pack<T>(v));
      }
    }
  }
}

template <typename T>
cudaError_t launch_dropout(DropoutParams p, bool vec, cudaStream_t s) {
  // (rows and octets of a row lie below 2^32 and 2^29: the product does not wrap)
  const uint64_t units = p.rows * p.octets;
  const uint64_t ctas = std::min((units + kThreads - 1) / kThreads, kMostCtas);
  const uint64_t step = ctas * kThreads;
  p.step_rows = static_cast<uint32_t>(step / p.octets);
  p.step_octets = static_cast<uint32_t>(step % p.octets);
  const Launch l{dim3(static_cast<unsigned>(ctas)), kThreads, 0, s};
  if (p.residual != nullptr)
    return vec ? launch(l, &dropout_kernel<T, true, true>, p)
               : launch(l, &dropout_kernel<T, false, true>, p);
  return vec ? launch(l, &dropout_kernel<T, true, false>, p)
             : launch(l, &dropout_kernel<T, false, false>, p);
}

}  // namespace

extern "C" cp_status cp_dropout(const void* x, uint64_t x_stride, const void* residual,
                                uint64_t residual_stride, int dtype, uint64_t rows, uint32_t d,
                                double p, uint64_t seed, uint64_t offset, const uint64_t* rng,
                                void* out, uint64_t out_stride, void* stream) {
  DropoutParams q{};
  if (!dtype_ok(dtype) || rows >= (1ull << 32) || (x_stride < d && x_stride != 0) ||
      (residual != nullptr && residual_stride < d && residual_stride != 0) || out_stride < d) {
    cpx::set_error("bad dtype, rows or row stride");
    return CP_ERR_INVALID_ARG;
  }
  if (!cpe::drop_params(&q.drop, p, seed, offset, rng) || !cpx::aligned(rng, 8)) {
    cpx::set_error("p must lie in 0 to 1, rng on 8 bytes");
    return CP_ERR_INVALID_ARG;
  }
  if (rows == 0 || d == 0) return CP_OK;
  const uint64_t elt = dtype_size(dtype);
  if (x == nullptr || out == nullptr || !cpx::aligned(x, elt) || !cpx::aligned(out, elt) ||
      !cpx::aligned(residual, elt)) {
    cpx::set_error("null or misaligned x, residual or out");
    return CP_ERR_INVALID_ARG;
  }
  q.x = x;
  q.residual = residual;
  q.out = out;
  q.ldx = x_stride;
  q.ldr = residual_stride;
  q.ldo = out_stride;
  q.rows = rows;
  q.d = d;
  q.octets = static_cast<uint32_t>((static_cast<uint64_t>(d) + 7) / 8);
  const bool vec = octets_ok(x, x_stride, d, elt) && octets_ok(out, out_stride, d, elt) &&
                   (residual == nullptr || octets_ok(residual, residual_stride, d, elt));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == CP_F32   ? launch_dropout<float>(q, vec, s)
                        : dtype == CP_F16 ? launch_dropout<__half>(q, vec, s)
                                          : launch_dropout<__nv_bfloat16>(q, vec, s);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "dropout launch");
  return CP_OK;
}

// cp_dropout.cu -- dropout from a counter-based generator, with the residual's addition
// (include/cp.h, cp_dropout).
//
//   out[i][j] = rn(residual[i][j] + D(x)[i][j])
//
// An octet a thread: two calls of the generator.  In fp32, and in 16 bits with a residual, bound by
// memory (65,536 x 1024 fp32 80 us, 6.7 TB/s; 196,608 x 1024 bf16 with a residual 186, 6.5 TB/s); in 16 bits
// without one by the generator's 32 x 32 -> 64 bit products (158 us at 76 % of their pipe, where the copy
// takes 119): so nothing else is left on that pipe (scales two at a time, values widened by byte
// moves, flat addresses by addition).
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "cp.h"
#include "cp_epilogue.cuh"
#include "cp_internal.h"
#include "cp_layer.cuh"

namespace {

using namespace cpl;
using cpe::DropKey;

constexpr int kThreads = 256;

// x * scale of two elements, by one instruction; and an octet's bits widened by byte moves: the
// generator's products fill the pipe that multiplications and shifts by multiplication share.
__device__ __forceinline__ void scale_pair(float& a, float& b, float scale) {
  asm("{\n"
      ".reg .b64 v, s;\n"
      "mov.b64 v, {%0, %1};\n"
      "mov.b64 s, {%2, %2};\n"
      "mul.rn.f32x2 v, v, s;\n"
      "mov.b64 {%0, %1}, v;\n"
      "}\n"
      : "+f"(a), "+f"(b)
      : "f"(scale));
}
template <typename T>
__device__ __forceinline__ void widen(const Packed<T>& r, float (&v)[8]) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(__byte_perm(r.w[i], 0, 0x1044));
      v[2 * i + 1] = __uint_as_float(__byte_perm(r.w[i], 0, 0x3244));
    }
  } else {
    unpack(r, v);
  }
}

struct DropoutParams {
  const void* x;
  const void* residual;
  void* out;
  uint64_t ldx, ldr, ldo;                  // flat: all d, d a multiple of 8
  uint32_t rows, d, octets;                // octets of a row
  uint32_t step_rows, step_octets;         // what kThreads octets come to
  uint32_t per;                            // octets of a thread
  cpe::DropParams drop;
};

// How rows lie: one behind the other in whole octets; apart, in whole octets; anywhere.  The first
// needs no position of a row (a product of 64 bits each, on the generator's pipe).
enum { kFlat, kRows, kAny };

// Octets whose loads a thread has in flight, and CTAs of an SM, by registers.  Rows anywhere take more
// warps instead, which hides their chains of shifts better (100,000 x 1023 bf16 with a residual 165 us
// against 186 as the others, 9001 x 813 fp32 16.4 against 17.5).
template <int kLayout>
constexpr int kAhead = kLayout == kAny ? 1 : 2;
template <typename T, int kLayout, bool kResidual>
constexpr int kCtas = kLayout == kAny ? (sizeof(T) == 4 ? 6 : 8) : sizeof(T) == 4 ? 4 : kResidual ? 5 : 6;

template <typename T, int kLayout, bool kResidual>
__global__ void __launch_bounds__(kThreads, (kCtas<T, kLayout, kResidual>))
    dropout_kernel(const __grid_constant__ DropoutParams p) {
  constexpr bool VEC = kLayout != kAny;
  constexpr int kAt = kAhead<kLayout>;
  wait_for_previous();
  let_next_start();
  const DropKey key = cpe::drop_key(p.drop);
  const cpe::RoundKeys keys = cpe::round_keys(key);
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * (kThreads * p.per) + threadIdx.x;
  uint32_t row = static_cast<uint32_t>(first / p.octets);
  uint32_t o = static_cast<uint32_t>(first - static_cast<uint64_t>(row) * p.octets);
  const T* px = static_cast<const T*>(p.x) + 8 * first;          // (of kFlat)
  const T* pr = static_cast<const T*>(p.residual) + 8 * first;
  T* po = static_cast<T*>(p.out) + 8 * first;
#pragma unroll 1
  for (uint32_t n = 0; n < p.per && row < p.rows; n += kAt) {
    Packed<T> x[kAt], r[kAt];
    uint32_t at[kAt], col[kAt];
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      at[i] = row;
      col[i] = o;
      if (row < p.rows) {
        if constexpr (kLayout == kFlat) {
          x[i] = load_octet(px + 8 * kThreads * i);
          if constexpr (kResidual) r[i] = load_octet(pr + 8 * kThreads * i);
        } else {
          x[i] = load_row_octet<T, VEC>(static_cast<const T*>(p.x) + row * p.ldx, o, p.d);
          if constexpr (kResidual)
            r[i] = load_row_octet<T, VEC>(static_cast<const T*>(p.residual) + row * p.ldr, o, p.d);
        }
      }
      o += p.step_octets;
      row += p.step_rows;
      if (o >= p.octets) {
        o -= p.octets;
        ++row;
      }
    }
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      if (at[i] < p.rows) {
        float v[8];
        widen(x[i], v);
        if (p.drop.mode == 1) {
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {
            const uint4 w = cpe::philox(2 * col[i] + h, at[i], key, keys);
            float* u = v + 4 * h;
            scale_pair(u[0], u[1], p.drop.scale);
            scale_pair(u[2], u[3], p.drop.scale);
            u[0] = w.x <= p.drop.last ? u[0] : 0.0f;
            u[1] = w.y <= p.drop.last ? u[1] : 0.0f;
            u[2] = w.z <= p.drop.last ? u[2] : 0.0f;
            u[3] = w.w <= p.drop.last ? u[3] : 0.0f;
          }
        } else if (p.drop.mode == 2) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = 0.0f;
        }
        if constexpr (kResidual) {
          float w[8];
          widen(r[i], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += w[e];
        }
        if constexpr (kLayout == kFlat)
          store_octet(po + 8 * kThreads * i, pack<T>(v));
        else
          store_row_octet<T, VEC>(static_cast<T*>(p.out) + at[i] * p.ldo, col[i], p.d, pack<T>(v));
      }
    }
    px += 8 * kThreads * kAt;
    pr += 8 * kThreads * kAt;
    po += 8 * kThreads * kAt;
  }
}

// Rows one behind the other on any boundary.  A lane makes the mask of an octet, eight bits; the
// elements go to the lanes one by one, 32 neighbours an access, and each takes its place and its bit
// from the lane that has its octet.  For fp32 with a residual, where it is the stores of shifted
// octets that take the time (an array of its own as the residual, here / by octets: 90010 x 813 144.6 /
// 145.9 us, 100000 x 1023 200 / 206, 1000 x 4097 14.2 / 19.2, 40000 x 25 6.8 / 8.0, 48 x 1023 3.0 / 3.6).
// Without a residual or in 16 bits the exchange costs more than it saves (90010 x 813 without one 124 us
// against 115; 100000 x 1023 bf16 176 against 125).
__global__ void __launch_bounds__(kThreads, 5)
    dropout_elements_kernel(const __grid_constant__ DropoutParams p) {
  wait_for_previous();
  let_next_start();
  const DropKey key = cpe::drop_key(p.drop);
  const cpe::RoundKeys keys = cpe::round_keys(key);
  const uint32_t lane = threadIdx.x & 31, e = lane & 7;
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * (kThreads * p.per) + threadIdx.x;
  uint32_t row = static_cast<uint32_t>(first / p.octets);
  uint32_t o = static_cast<uint32_t>(first - static_cast<uint64_t>(row) * p.octets);
#pragma unroll 1
  for (uint32_t n = 0; n < p.per; ++n) {
    const bool in = row < p.rows;
    if (!__any_sync(0xFFFFFFFFu, in)) break;
    // how many elements the octet has (bits 0 to 3), how far it lies from the warp's first
    const uint64_t start = static_cast<uint64_t>(row) * p.d + 8 * o;
    const uint64_t base = __shfl_sync(0xFFFFFFFFu, start, 0);
    const uint32_t place =
        in ? min(p.d - 8 * o, 8u) | static_cast<uint32_t>(start - base) << 4 : 0u;
    const float* px = static_cast<const float*>(p.x) + base + e;
    const float* pr = static_cast<const float*>(p.residual) + base + e;
    float* po = static_cast<float*>(p.out) + base + e;
    uint32_t at[8];
    float x[8], r[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      at[i] = __shfl_sync(0xFFFFFFFFu, place, static_cast<int>(4 * i + (lane >> 3)));
      if (e < (at[i] & 15)) {
        x[i] = px[at[i] >> 4];
        r[i] = pr[at[i] >> 4];
      }
    }
    uint32_t kept = 0;               // the octet's, while the elements come
    if (p.drop.mode == 1) {
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) {
        const uint4 w = cpe::philox(2 * o + h, row, key, keys);
        kept |= w.x <= p.drop.last ? 1u << (4 * h) : 0u;
        kept |= w.y <= p.drop.last ? 2u << (4 * h) : 0u;
        kept |= w.z <= p.drop.last ? 4u << (4 * h) : 0u;
        kept |= w.w <= p.drop.last ? 8u << (4 * h) : 0u;
      }
    }
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const uint32_t bits = __shfl_sync(0xFFFFFFFFu, kept, static_cast<int>(4 * i + (lane >> 3)));
      if (e < (at[i] & 15)) {
        float v = x[i];
        if (p.drop.mode != 0) v = bits >> e & 1 ? v * p.drop.scale : 0.0f;
        po[at[i] >> 4] = v + r[i];
      }
    }
    __syncwarp();
    o += p.step_octets;
    row += p.step_rows;
    if (o >= p.octets) {
      o -= p.octets;
      ++row;
    }
  }
}

template <typename T, bool kResidual>
cudaError_t launch_dropout(DropoutParams p, bool vec, uint64_t ctas, cudaStream_t s) {
  const Launch l{dim3(static_cast<unsigned>(ctas)), kThreads, 0, s};
  const bool flat = p.ldx == p.d && p.ldo == p.d && (!kResidual || p.ldr == p.d);
  if (vec)
    return flat ? launch(l, &dropout_kernel<T, kFlat, kResidual>, p)
                : launch(l, &dropout_kernel<T, kRows, kResidual>, p);
  if (sizeof(T) == 4 && kResidual && flat) return launch(l, &dropout_elements_kernel, p);
  return launch(l, &dropout_kernel<T, kAny, kResidual>, p);
}
template <typename T>
cudaError_t launch_dropout(const DropoutParams& p, bool vec, uint64_t ctas, cudaStream_t s) {
  return p.residual != nullptr ? launch_dropout<T, true>(p, vec, ctas, s)
                               : launch_dropout<T, false>(p, vec, ctas, s);
}

}  // namespace

extern "C" cp_status cp_dropout(const void* x, uint64_t x_stride, const void* residual,
                                uint64_t residual_stride, int dtype, uint64_t rows, uint32_t d,
                                double p, uint64_t seed, uint64_t offset, const uint64_t* rng,
                                void* out, uint64_t out_stride, void* stream) {
  DropoutParams q{};
  if (!dtype_ok(dtype) || rows >= (1ull << 31) || (x_stride < d && x_stride != 0) ||
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
  const cpx::RowBytes to{out, out_stride * elt, d * elt, rows};
  if (cpx::rows_clash(to, {x, x_stride * elt, d * elt, rows}) ||
      cpx::rows_clash(to, {residual, residual_stride * elt, d * elt, rows})) {
    cpx::set_error("out lies on part of x or of the residual");
    return CP_ERR_INVALID_ARG;
  }
  q.x = x;
  q.residual = residual;
  q.out = out;
  q.ldx = x_stride;
  q.ldr = residual_stride;
  q.ldo = out_stride;
  q.rows = static_cast<uint32_t>(rows);
  q.d = d;
  q.octets = static_cast<uint32_t>((static_cast<uint64_t>(d) + 7) / 8);
  const bool vec = octets_ok(x, x_stride, d, elt) && octets_ok(out, out_stride, d, elt) &&
                   (residual == nullptr || octets_ok(residual, residual_stride, d, elt));
  q.step_rows = kThreads / q.octets;
  q.step_octets = kThreads % q.octets;
  const uint64_t units = rows * q.octets;
  // CTAs short enough to even out, and as many as run at once where there is little (bf16, 48 x 1024:
  // 2.1 us with two octets a thread, 4.5 with eight; 4096 x 4096: 16.6 with four, 18.4; 196,608 x 1024:
  // 159 with eight, 165 with four).
  q.per = units < (1u << 17) ? 2 : units < (1u << 22) ? 4 : 8;
  const uint64_t ctas = (units + kThreads * q.per - 1) / (kThreads * q.per);
  if (ctas >= (1ull << 31)) {
    cpx::set_error("rows of d make more than 2^42 octets");
    return CP_ERR_INVALID_ARG;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == CP_F32   ? launch_dropout<float>(q, vec, ctas, s)
                        : dtype == CP_F16 ? launch_dropout<__half>(q, vec, ctas, s)
                                          : launch_dropout<__nv_bfloat16>(q, vec, ctas, s);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "dropout launch");
  return CP_OK;
}

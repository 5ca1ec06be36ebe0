// cp_epilogue.cuh -- what follows a projection's sums (include/cp.h, cp_linear): bias,
// activation, dropout, the residual's addition; and what its gradient undoes.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "cp.h"
#include "cp_layer.cuh"

namespace cpe {

using namespace cpl;

// --------------------------------------------------------------------- dropout
//
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// 2011): ten rounds of two 32 x 32 -> 64 bit products on a counter, the key stepped between them.
// Element [i][j] takes word j mod 4 of counter (j / 4, i, offset) under the key `seed`, so four
// neighbouring columns share a call, any kernel can make any part of the mask, and nothing of
// it is stored.

struct DropParams {
  const uint64_t* rng;   // seed and offset on the device, or null
  uint64_t seed, offset; // offset is added to rng[1]
  uint32_t last;         // the largest word that keeps its element
  float scale;           // 1 / (1 - p)
  int mode;              // 0: nothing is dropped, 1: by the words, 2: everything
};

struct DropKey {
  uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ DropKey drop_key(const DropParams& p) {
  uint64_t seed = p.seed, offset = p.offset;
  if (p.mode == 1 && p.rng != nullptr) {
    seed = p.rng[0];
    offset += p.rng[1];
  }
  return DropKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32),
                 static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32)};
}

// The key of each round, for kernels that make many calls and have the registers.
struct RoundKeys {
  uint32_t k0[10], k1[10];
};
__device__ __forceinline__ RoundKeys round_keys(const DropKey& key) {
  RoundKeys r;
#pragma unroll
  for (uint32_t i = 0; i < 10; ++i) {
    r.k0[i] = key.k0 + i * 0x9E3779B9u;
    r.k1[i] = key.k1 + i * 0xBB67AE85u;
  }
  return r;
}

__device__ __forceinline__ uint4 philox(uint32_t quad, uint32_t row, const DropKey& key,
                                        const RoundKeys& k) {
  uint32_t c0 = quad, c1 = row, c2 = key.o0, c3 = key.o1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k.k0[r];
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k.k1[r];
    c3 = static_cast<uint32_t>(a);
  }
  return make_uint4(c0, c1, c2, c3);
}

// Four columns of a row, 4 * quad on.  A dropped element is zero whatever it was.
__device__ __forceinline__ void drop_quad(const DropParams& p, const DropKey& key,
                                          const RoundKeys& k, uint32_t quad, uint32_t row,
                                          float* v) {
  if (p.mode == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 0.0f;
    return;
  }
  const uint4 w = philox(quad, row, key, k);
  v[0] = w.x <= p.last ? v[0] * p.scale : 0.0f;
  v[1] = w.y <= p.last ? v[1] * p.scale : 0.0f;
  v[2] = w.z <= p.last ? v[2] * p.scale : 0.0f;
  v[3] = w.w <= p.last ? v[3] * p.scale : 0.0f;
}
__device__ __forceinline__ void drop_quad(const DropParams& p, const DropKey& key, uint32_t quad,
                                          uint32_t row, float* v) {
  drop_quad(p, key, round_keys(key), quad, row, v);
}

// 4 * kQuads columns, 4 * quad on, of kRows rows, row_step apart: all calls of the generator side by
// side, so that its chains of products overlap and a round's key is made once for all.
template <uint32_t kQuads, uint32_t kRows>
__device__ __forceinline__ void drop_block(const DropParams& p, const DropKey& key, uint32_t quad,
                                           uint32_t row, uint32_t row_step, float* v) {
  constexpr uint32_t kCalls = kQuads * kRows;
  if (p.mode == 2) {
#pragma unroll
    for (uint32_t i = 0; i < 4 * kCalls; ++i) v[i] = 0.0f;
    return;
  }
  uint32_t c0[kCalls], c1[kCalls], c2[kCalls], c3[kCalls], k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (uint32_t q = 0; q < kCalls; ++q) {
    c0[q] = quad + q % kQuads;
    c1[q] = row + q / kQuads * row_step;
    c2[q] = key.o0;
    c3[q] = key.o1;
  }
#pragma unroll
  for (int r = 0; r < 10; ++r) {
#pragma unroll
    for (uint32_t q = 0; q < kCalls; ++q) {
      const uint64_t a = static_cast<uint64_t>(c0[q]) * 0xD2511F53u;
      const uint64_t b = static_cast<uint64_t>(c2[q]) * 0xCD9E8D57u;
      c0[q] = static_cast<uint32_t>(b >> 32) ^ c1[q] ^ k0;
      c1[q] = static_cast<uint32_t>(b);
      c2[q] = static_cast<uint32_t>(a >> 32) ^ c3[q] ^ k1;
      c3[q] = static_cast<uint32_t>(a);
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
#pragma unroll
  for (uint32_t q = 0; q < kCalls; ++q) {
    v[4 * q] = c0[q] <= p.last ? v[4 * q] * p.scale : 0.0f;
    v[4 * q + 1] = c1[q] <= p.last ? v[4 * q + 1] * p.scale : 0.0f;
    v[4 * q + 2] = c2[q] <= p.last ? v[4 * q + 2] * p.scale : 0.0f;
    v[4 * q + 3] = c3[q] <= p.last ? v[4 * q + 3] * p.scale : 0.0f;
  }
}

// What a call's p, seed and offset say; false where p is no probability.
inline bool drop_params(DropParams* d, double p, uint64_t seed, uint64_t offset,
                        const uint64_t* rng) {
  if (!(p >= 0.0 && p <= 1.0)) return false;
  const uint64_t kept = static_cast<uint64_t>((1.0 - p) * 4294967296.0 + 0.5);
  d->rng = rng;
  d->seed = seed;
  d->offset = offset;
  d->mode = p == 0.0 ? 0 : kept == 0 ? 2 : 1;
  d->last = static_cast<uint32_t>(kept == 0 ? 0 : kept - 1);
  d->scale = kept == 0 ? 0.0f : static_cast<float>(1.0 / (1.0 - p));
  return true;
}

// ------------------------------------------------------------------ activations
//
// In fp32.  sigmoid(t) = 1 / (1 + 2^(-t log2 e)), by the approximate exponential and reciprocal: an
// error of the exponent's argument, |t| 2^-24 relative, reaches the sigmoid times 1 - sigmoid, and is
// below 2^-25 for every t > -20 or so and relative to a value below 2^-28 beyond; with the two
// instructions' own errors 2^-22.  The tanh form of gelu is z sigmoid(2 u),
// u = sqrt(2 / pi) (z + 0.044715 z^3), since (1 + tanh u) / 2 = sigmoid(2 u).

constexpr float kTanhScale = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;
constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sigmoid(float t) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp2_approx(-kLog2E * t)));
  return r;
}

// Two values side by side in one instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void pair_to(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, float c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(pair_of(c, c)));
  return r;
}

// Phi(z), the normal distribution, of two values, and `bell`, e^(-z^2 / 2).  Phi(-|z|) = t P(t) bell with
// t = 1 / (1 + 0.3 |z|): the quotient of the two is smooth, falls as 1 / |z| and so is a polynomial in t
// almost to the last place, P of degree 7 fitted to it for the least relative error (1.8e-7 up to
// |z| = 13.5, where the bell ends).  So the lower tail is accurate relative to its own value, up to what
// the bell takes from its argument's roundings: 2^-24 (20 + 1.25 z^2) in all.  Both values of a pair in
// one instruction where there is one: it is issue that bounds the epilogue.
__device__ __forceinline__ void normal_cdf(float za, float zb, float& cdf_a, float& cdf_b,
                                           float& bell_a, float& bell_b) {
  float ta, tb, ea, eb, la, lb;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ta) : "f"(fmaf(0.3f, fabsf(za), 1.0f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(tb) : "f"(fmaf(0.3f, fabsf(zb), 1.0f)));
  const uint64_t z = pair_of(za, zb), t = pair_of(ta, tb);
  pair_to(pair_mul(pair_mul(z, z), pair_of(-0.5f * kLog2E, -0.5f * kLog2E)), ea, eb);
  bell_a = exp2_approx(ea);
  bell_b = exp2_approx(eb);
  uint64_t p = pair_of(0.0359262377f, 0.0359262377f);
  p = pair_fma(p, t, -0.158232927f);
  p = pair_fma(p, t, 0.208094433f);
  p = pair_fma(p, t, -0.0552531257f);
  p = pair_fma(p, t, 0.129374236f);
  p = pair_fma(p, t, 0.0996722728f);
  p = pair_fma(p, t, 0.120791957f);
  p = pair_fma(p, t, 0.11962685f);
  pair_to(pair_mul(pair_mul(t, p), pair_of(bell_a, bell_b)), la, lb);
  cdf_a = za < 0.0f ? la : 1.0f - la;
  cdf_b = zb < 0.0f ? lb : 1.0f - lb;
}

template <int kAct>
__device__ __forceinline__ float act(float z) {
  if constexpr (kAct == CP_ACT_RELU) return z < 0.0f ? 0.0f : z;
  if constexpr (kAct == CP_ACT_SILU) return z * sigmoid(z);
  if constexpr (kAct == CP_ACT_GELU_TANH)
    return z * sigmoid(kTanhScale * (z + kTanhCube * z * z * z));
  return z;
}
// Of an even number of values, in place.
template <int kAct, int kCount>
__device__ __forceinline__ void act_all(float (&v)[kCount]) {
  static_assert(kCount % 2 == 0, "pairs");
#pragma unroll
  for (int i = 0; i < kCount; i += 2) {
    if constexpr (kAct == CP_ACT_GELU) {
      float a, b, bell_a, bell_b;
      normal_cdf(v[i], v[i + 1], a, b, bell_a, bell_b);
      v[i] *= a;
      v[i + 1] *= b;
    } else {
      v[i] = act<kAct>(v[i]);
      v[i + 1] = act<kAct>(v[i + 1]);
    }
  }
}

// Its derivative.
template <int kAct>
__device__ __forceinline__ float slope(float z) {
  if constexpr (kAct == CP_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (kAct == CP_ACT_SILU) {
    const float s = sigmoid(z);
    return s * (1.0f + z * (1.0f - s));
  }
  if constexpr (kAct == CP_ACT_GELU_TANH) {
    const float s = sigmoid(kTanhScale * (z + kTanhCube * z * z * z));
    const float bend = s * (1.0f - s);                 // 0 far out, where z^2 may overflow
    return bend == 0.0f ? s : s + z * bend * kTanhScale * (1.0f + 3.0f * kTanhCube * z * z);
  }
  return 1.0f;
}
// v times the derivative at z, of an even number of values.
template <int kAct, int kCount>
__device__ __forceinline__ void slope_all(const float (&z)[kCount], float (&v)[kCount]) {
  static_assert(kCount % 2 == 0, "pairs");
#pragma unroll
  for (int i = 0; i < kCount; i += 2) {
    if constexpr (kAct == CP_ACT_GELU) {
      float a, b, bell_a, bell_b;
      normal_cdf(z[i], z[i + 1], a, b, bell_a, bell_b);
      v[i] *= a + z[i] * 0.39894228040143268f * bell_a;
      v[i + 1] *= b + z[i + 1] * 0.39894228040143268f * bell_b;
    } else {
      v[i] *= slope<kAct>(z[i]);
      v[i + 1] *= slope<kAct>(z[i + 1]);
    }
  }
}

// f(std::integral_constant-like tag) for the call's activation: the choice is made once for a
// set of values, the same for every thread.
template <int kAct>
struct ActTag {
  static constexpr int value = kAct;
};
template <typename F>
__device__ __forceinline__ void with_act(int which, F&& f) {
  if (which == CP_ACT_RELU) f(ActTag<CP_ACT_RELU>{});
  else if (which == CP_ACT_SILU) f(ActTag<CP_ACT_SILU>{});
  else if (which == CP_ACT_GELU) f(ActTag<CP_ACT_GELU>{});
  else if (which == CP_ACT_GELU_TANH) f(ActTag<CP_ACT_GELU_TANH>{});
}

inline bool act_ok(int a) { return a >= CP_ACT_NONE && a <= CP_ACT_GELU_TANH; }

// --------------------------------------------------------------------- epilogue

struct Epilogue {
  const void* bias;        // [n], or null
  const void* residual;    // [m][n] of out's type, or null
  void* out;
  void* pre;               // the sums in front of the activation, in the operands' type, or null
  uint64_t ldr, ldo, ldp;
  uint32_t m, n;
  int bias_dtype, out_dtype, pre_dtype, act;
  uint32_t aligned;        // rows of out, residual and pre all lie on 32-byte boundaries
  DropParams drop;
};

// Four neighbouring elements of a row, those before n; whole where `vec` (rows on 16 bytes).
__device__ __forceinline__ void load_quad(const void* p, uint64_t at, uint32_t left, int dtype,
                                          bool vec, float (&v)[4]) {
  if (vec && left >= 4) {
    if (dtype == CP_F32) {
      const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
      const uint32_t w[2] = {x.x, x.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t u = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
        v[i] = dtype == CP_F16 ? __half2float(__ushort_as_half(u))
                               : __bfloat162float(__ushort_as_bfloat16(u));
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = static_cast<uint32_t>(i) < left ? load_as_f32(p, at + i, dtype) : 0.0f;
}
__device__ __forceinline__ void store_quad(void* p, uint64_t at, uint32_t left, int dtype, bool vec,
                                           const float (&v)[4]) {
  if (vec && left >= 4) {
    if (dtype == CP_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = dtype == CP_F16 ? __half_as_ushort(__float2half_rn(v[i]))
                               : __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) =
          make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (static_cast<uint32_t>(i) < left) store_from_f32(p, at + i, dtype, v[i]);
}

// The whole epilogue of four neighbouring sums, col a multiple of 4.
__device__ __forceinline__ void finish_quad(const Epilogue& e, const DropKey& key, uint32_t row,
                                            uint32_t col, float (&v)[4]) {
  const uint32_t left = e.n - col;
  const bool vec = e.aligned != 0;
  float r[4] = {};
  if (e.residual != nullptr)
    load_quad(e.residual, static_cast<uint64_t>(row) * e.ldr + col, left, e.out_dtype, vec, r);
  if (e.bias != nullptr) {
    float b[4];
    load_quad(e.bias, col, left, e.bias_dtype, false, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += b[i];
  }
  if (e.pre != nullptr)
    store_quad(e.pre, static_cast<uint64_t>(row) * e.ldp + col, left, e.pre_dtype, vec, v);
  with_act(e.act, [&](auto tag) { act_all<decltype(tag)::value>(v); });
  if (e.drop.mode != 0) drop_quad(e.drop, key, col / 4, row, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] += r[i];
  store_quad(e.out, static_cast<uint64_t>(row) * e.ldo + col, left, e.out_dtype, vec, v);
}

// Sixteen outputs of a row on a 32-byte boundary, whole sectors of L2.
template <typename T>
__device__ __forceinline__ void store16(T* to, const float* v) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Packed<float> r;
#pragma unroll
      for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[8 * h + i]);
      store_octet(reinterpret_cast<float*>(to) + 8 * h, r);
    }
  } else {
    Packed<float> r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = v[8 * h + i];
      const Packed<T> x = pack<T>(u);
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[4 * h + i] = x.w[i];
    }
    store_octet(reinterpret_cast<float*>(to), r);
  }
}
__device__ __forceinline__ void store32(void* p, uint64_t at, int dtype, const float (&v)[32]) {
  if (dtype == CP_F32) {
    store16(static_cast<float*>(p) + at, v);
    store16(static_cast<float*>(p) + at + 16, v + 16);
  } else if (dtype == CP_F16) {
    store16(static_cast<__half*>(p) + at, v);
    store16(static_cast<__half*>(p) + at + 16, v + 16);
  } else {
    store16(static_cast<__nv_bfloat16*>(p) + at, v);
    store16(static_cast<__nv_bfloat16*>(p) + at + 16, v + 16);
  }
}
// v += 32 elements on a 32-byte boundary.
__device__ __forceinline__ void add_pair(float& lo, float& hi, uint32_t w, int dtype) {
  if (dtype == CP_F16) {
    lo += __half2float(__ushort_as_half(static_cast<uint16_t>(w)));
    hi += __half2float(__ushort_as_half(static_cast<uint16_t>(w >> 16)));
  } else {
    lo += __uint_as_float(w << 16);
    hi += __uint_as_float(w & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void add32(float (&v)[32], const void* p, uint64_t at, int dtype) {
  if (dtype == CP_F32) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const Packed<float> r = load_octet(static_cast<const float*>(p) + at + 8 * h);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * h + i] += __uint_as_float(r.w[i]);
    }
  } else {
    Packed<float> r[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      r[h] = load_octet(reinterpret_cast<const float*>(static_cast<const uint16_t*>(p) + at + 16 * h));
#pragma unroll
    for (int i = 0; i < 16; ++i) add_pair(v[2 * i], v[2 * i + 1], r[i / 8].w[i % 8], dtype);
  }
}

// x[i] of lane t becomes x[t] of lane i: five exchanges between lanes.
__device__ __forceinline__ void transpose32(float (&x)[32], uint32_t lane) {
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
}

// A column of up to 32 rows, ld elements apart: written, or added to v.  (One test of the type, not one
// a row.)
template <typename T>
__device__ __forceinline__ void store_column_of(T* to, uint64_t ld, uint32_t rows,
                                                const float (&v)[32]) {
#pragma unroll
  for (uint32_t r = 0; r < 32; ++r, to += ld)
    if (r < rows) *to = from_f32<T>(v[r]);
}
__device__ __forceinline__ void store_column(void* p, uint64_t at, uint64_t ld, uint32_t rows,
                                             int dtype, const float (&v)[32]) {
  if (dtype == CP_F32) store_column_of(static_cast<float*>(p) + at, ld, rows, v);
  else if (dtype == CP_F16) store_column_of(static_cast<__half*>(p) + at, ld, rows, v);
  else store_column_of(static_cast<__nv_bfloat16*>(p) + at, ld, rows, v);
}
template <typename T>
__device__ __forceinline__ void add_column_of(const T* from, uint64_t ld, uint32_t rows,
                                              float (&v)[32]) {
#pragma unroll
  for (uint32_t r = 0; r < 32; ++r, from += ld)
    if (r < rows) v[r] += to_f32(*from);
}
__device__ __forceinline__ void add_column(float (&v)[32], const void* p, uint64_t at, uint64_t ld,
                                           uint32_t rows, int dtype) {
  if (dtype == CP_F32) add_column_of(static_cast<const float*>(p) + at, ld, rows, v);
  else if (dtype == CP_F16) add_column_of(static_cast<const __half*>(p) + at, ld, rows, v);
  else add_column_of(static_cast<const __nv_bfloat16*>(p) + at, ld, rows, v);
}

// The epilogue of a warp's 32 rows (row0 on, one a lane) by 32 columns (col on, a multiple of 32)
// of sums, in two steps.  The first: bias, kept sums, activation, dropout.  `bias`: a lane has that
// of column col + lane.  fast: rows on 32-byte boundaries and columns all there, so a lane reads
// and writes its own row, whole sectors; else the block is transposed, so that each access is of
// 32 neighbours of one row.
template <bool kRich>
__device__ __forceinline__ void shape_block(const Epilogue& e, const DropKey& key, uint32_t row0,
                                            uint32_t col, uint32_t lane, float bias,
                                            bool fast, float (&v)[32]) {
  const uint32_t row = row0 + lane;
  if (e.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xFFFFFFFFu, bias, i);
  }
  if constexpr (kRich) {
    if (e.pre != nullptr) {
      if (fast) {
        if (row < e.m) store32(e.pre, static_cast<uint64_t>(row) * e.ldp + col, e.pre_dtype, v);
      } else {
        float u[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] = v[i];
        transpose32(u, lane);
        if (col + lane < e.n)
          store_column(e.pre, static_cast<uint64_t>(row0) * e.ldp + col + lane, e.ldp,
                       min(32u, e.m - row0), e.pre_dtype, u);
        __syncwarp();
      }
    }
    with_act(e.act, [&](auto tag) { act_all<decltype(tag)::value>(v); });
    if (e.drop.mode != 0) {
      drop_block<4, 1>(e.drop, key, col / 4, row, 0, v);
      drop_block<4, 1>(e.drop, key, col / 4 + 4, row, 0, v + 16);
    }
  }
}

// The second: the residual's addition and the outputs.
__device__ __forceinline__ void write_block(const Epilogue& e, uint32_t row0, uint32_t col,
                                            uint32_t lane, bool fast, float (&v)[32]) {
  const uint32_t row = row0 + lane;
  if (fast) {
    if (row < e.m) {
      if (e.residual != nullptr)
        add32(v, e.residual, static_cast<uint64_t>(row) * e.ldr + col, e.out_dtype);
      store32(e.out, static_cast<uint64_t>(row) * e.ldo + col, e.out_dtype, v);
    }
    __syncwarp();
    return;
  }
  const uint32_t rows = min(32u, e.m - row0);
  transpose32(v, lane);
  if (col + lane < e.n) {
    if (e.residual != nullptr)
      add_column(v, e.residual, static_cast<uint64_t>(row0) * e.ldr + col + lane, e.ldr, rows,
                 e.out_dtype);
    store_column(e.out, static_cast<uint64_t>(row0) * e.ldo + col + lane, e.ldo, rows, e.out_dtype,
                 v);
  }
  __syncwarp();
}

}  // namespace cpe

// cp_layer.cuh -- helpers shared by the memory layer's kernels (embed, RMS norm,
// 8-bit quantiser, 8-bit product): element types, octets of eight elements (the
// unit that one lane loads and stores), reductions, e4m3 groups.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "cp.h"

namespace cpl {

// ---------------------------------------------------------------- element types

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// One value of an array whose type is known at run time (CP_F32, CP_F16, CP_BF16);
// the branch is the same for every thread.
__device__ __forceinline__ float load_as_f32(const void* p, uint64_t i, int dtype) {
  if (dtype == CP_F32) return static_cast<const float*>(p)[i];
  if (dtype == CP_F16) return to_f32(static_cast<const __half*>(p)[i]);
  return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_from_f32(void* p, uint64_t i, int dtype, float x) {
  if (dtype == CP_F32) static_cast<float*>(p)[i] = x;
  else if (dtype == CP_F16) static_cast<__half*>(p)[i] = from_f32<__half>(x);
  else static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(x);
}

// ---------------------------------------------------------------------- octets
//
// An octet is eight consecutive elements.  Packed<T> holds one as loaded, 16 bytes
// (16-bit types: one 128-bit access) or 32 bytes (fp32: one 256-bit access), so a
// kernel can keep several in flight before it converts them.

template <typename T>
struct Packed {
  static constexpr int kWords = sizeof(T) * 2;
  uint32_t w[kWords];
};

template <typename T>
__device__ __forceinline__ Packed<T> load_octet(const T* p) {
  Packed<T> r;
  if constexpr (sizeof(T) == 2) {
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(p));
  } else {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                   "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
                 : "l"(p));
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void store_octet(T* p, const Packed<T>& r) {
  if constexpr (sizeof(T) == 2) {
    asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]),
                 "r"(r.w[2]), "r"(r.w[3])
                 : "memory");
  } else {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0]),
                 "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]),
                 "r"(r.w[7])
                 : "memory");
  }
}

template <typename T>
__device__ __forceinline__ void unpack(const Packed<T>& r, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t lo = static_cast<uint16_t>(r.w[i]), hi = static_cast<uint16_t>(r.w[i] >> 16);
      if constexpr (sizeof(T) == 2) {
        T a, b;
        memcpy(&a, &lo, 2);
        memcpy(&b, &hi, 2);
        v[2 * i] = to_f32(a);
        v[2 * i + 1] = to_f32(b);
      }
    }
  }
}

// Two values to 16 bits, the first in the low half: one conversion for both (the single ones run on
// the pipe of the special functions, an eighth as wide).
template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  uint32_t w;
  if constexpr (std::is_same_v<T, __half>)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

template <typename T>
__device__ __forceinline__ Packed<T> pack(const float (&v)[8]) {
  Packed<T> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = pack_pair<T>(v[2 * i], v[2 * i + 1]);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ Packed<T> zero_octet() {
  Packed<T> r;
#pragma unroll
  for (int i = 0; i < Packed<T>::kWords; ++i) r.w[i] = 0;
  return r;
}

// The octet that starts `skew` bytes into the words x.
template <typename T>
__device__ __forceinline__ Packed<T> shift_octet(uint32_t (&x)[Packed<T>::kWords + 4], uint32_t skew) {
  if (skew & 8) {
#pragma unroll
    for (int i = 0; i < Packed<T>::kWords + 2; ++i) x[i] = x[i + 2];
  }
  if (skew & 4) {
#pragma unroll
    for (int i = 0; i < Packed<T>::kWords + 1; ++i) x[i] = x[i + 1];
  }
  Packed<T> r;
#pragma unroll
  for (int i = 0; i < Packed<T>::kWords; ++i)
    r.w[i] = sizeof(T) == 4 ? x[i] : __funnelshift_r(x[i], x[i + 1], 8 * (skew & 2));
  return r;
}

// Octet `o` of a row of d elements at p.  VEC: rows whose every octet is whole and aligned to its
// own size.  Otherwise rows start anywhere and the last octet may be part full (the rest reads
// as zero and is not written): an octet is shifted out of the aligned 16-byte words that hold
// it, where they lie within the row, and read by single elements at the row's ends; it is
// written in the widest pieces that its address allows.
template <typename T>
__device__ __forceinline__ Packed<T> load_skewed_octet(const T* row, uint32_t o, uint32_t d) {
  constexpr int kQuads = Packed<T>::kWords / 4;
  const uintptr_t first = reinterpret_cast<uintptr_t>(row), at = first + 8ull * sizeof(T) * o;
  const uint32_t skew = static_cast<uint32_t>(at & 15);
  const uintptr_t from = at - skew, to = from + 16 * kQuads + (skew != 0 ? 16 : 0);
  Packed<T> r = zero_octet<T>();
  if (from >= first && to <= first + static_cast<uint64_t>(d) * sizeof(T)) {
    uint32_t x[4 * kQuads + 4];
#pragma unroll
    for (int q = 0; q < kQuads + 1; ++q) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (q < kQuads || skew != 0)
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(from + 16 * q));
      x[4 * q] = v.x;
      x[4 * q + 1] = v.y;
      x[4 * q + 2] = v.z;
      x[4 * q + 3] = v.w;
    }
    r = shift_octet<T>(x, skew);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = 8 * o + i;
      if (c < d) {
        if constexpr (sizeof(T) == 4) {
          r.w[i] = reinterpret_cast<const uint32_t*>(row)[c];
        } else {
          const uint32_t u = reinterpret_cast<const uint16_t*>(row)[c];
          r.w[i / 2] |= u << (16 * (i & 1));
        }
      }
    }
  }
  return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ Packed<T> load_row_octet(const T* row, uint32_t o, uint32_t d) {
  if constexpr (VEC) return load_octet(row + 8ull * o);
  else return load_skewed_octet(row, o, d);
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_row_octet(T* row, uint32_t o, uint32_t d,
                                                const Packed<T>& r) {
  if constexpr (VEC) {
    store_octet(row + 8ull * o, r);
    return;
  }
  T* to = row + 8ull * o;
  const uint32_t skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(to) & 15);
  if (o >= d / 8) {                      // (8 o + 8 wraps in rows of almost 2^32 columns)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (8 * o + i < d) {
        if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(to)[i] = r.w[i];
        else reinterpret_cast<uint16_t*>(to)[i] = static_cast<uint16_t>(r.w[i / 2] >> (16 * (i & 1)));
      }
    }
  } else if (skew == 0) {
#pragma unroll
    for (int q = 0; q < Packed<T>::kWords / 4; ++q)
      reinterpret_cast<uint4*>(to)[q] =
          make_uint4(r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]);
  } else if (skew == 8) {
#pragma unroll
    for (int q = 0; q < Packed<T>::kWords / 2; ++q)
      reinterpret_cast<uint2*>(to)[q] = make_uint2(r.w[2 * q], r.w[2 * q + 1]);
  } else if ((skew & 3) == 0) {
#pragma unroll
    for (int q = 0; q < Packed<T>::kWords; ++q) reinterpret_cast<uint32_t*>(to)[q] = r.w[q];
  } else if constexpr (sizeof(T) == 2) {
    uint16_t* h = reinterpret_cast<uint16_t*>(to);
    h[0] = static_cast<uint16_t>(r.w[0]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
      reinterpret_cast<uint32_t*>(h + 1)[q] = __funnelshift_r(r.w[q], r.w[q + 1], 16);
    h[7] = static_cast<uint16_t>(r.w[3] >> 16);
  }
}

// Octet `o` of a row of d elements to shared memory, asynchronously, and back from there by the
// thread that copied it.  A row that starts off a 16-byte boundary: the first word
// reaches up to 14 bytes in front of it, which are dropped (they lie in the row's allocation:
// allocations start on 256-byte boundaries); behind the row's end nothing is read, zeros stand
// there.  `last`: the lane that also copies the word behind its octet, the others find it at
// their neighbour's.
template <typename T, bool VEC>
__device__ __forceinline__ void copy_octet(uint32_t to, const T* row, uint32_t o, uint32_t d,
                                           bool last) {
  if constexpr (VEC) {
    const uint8_t* from = reinterpret_cast<const uint8_t*>(row + 8ull * o);
#pragma unroll
    for (uint32_t b = 0; b < 8 * sizeof(T); b += 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + b), "l"(from + b)
                   : "memory");
  } else {
    const uint32_t skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15);
    const uintptr_t first = reinterpret_cast<uintptr_t>(row) - skew;
    const uint32_t end = skew + d * static_cast<uint32_t>(sizeof(T));     // of the row, from `first`
#pragma unroll
    for (uint32_t b = 0; b < 8 * sizeof(T) + 16; b += 16) {
      const uint32_t at = 8 * static_cast<uint32_t>(sizeof(T)) * o + b;
      const uint32_t bytes = end <= at ? 0 : min(end - at, 16u);
      // (a word without a byte of the row is not read: its address is the row's own)
      if (b < 8 * sizeof(T) || last)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + b),
                     "l"(first + (bytes == 0 ? 0 : at)), "r"(bytes)
                     : "memory");
    }
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ Packed<T> copied_octet(const uint8_t* at, const T* row) {
  uint32_t x[Packed<T>::kWords + 4];
#pragma unroll
  for (int q = 0; q < Packed<T>::kWords / 4 + (VEC ? 0 : 1); ++q) {
    const uint4 v = reinterpret_cast<const uint4*>(at)[q];
    x[4 * q] = v.x;
    x[4 * q + 1] = v.y;
    x[4 * q + 2] = v.z;
    x[4 * q + 3] = v.w;
  }
  if constexpr (!VEC)
    return shift_octet<T>(x, static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15));
  Packed<T> r;
#pragma unroll
  for (int i = 0; i < Packed<T>::kWords; ++i) r.w[i] = x[i];
  return r;
}

// Whether rows at p, `stride` elements apart and d long, may be read by whole octets.
inline bool octets_ok(const void* p, uint64_t stride, uint32_t d, uint64_t elt) {
  return reinterpret_cast<uintptr_t>(p) % (8 * elt) == 0 && stride % 8 == 0 && d % 8 == 0;
}

inline uint64_t dtype_size(int dtype) { return dtype == CP_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == CP_F32 || dtype == CP_F16 || dtype == CP_BF16; }

// ------------------------------------------------------------------- reductions

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// Largest magnitude as the bits of |x|: ordered like the magnitudes themselves, with
// infinity above every number and NaN above infinity, so a NaN is never lost.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// ---------------------------------------------------------------- e4m3 and scales
//
// A group's scale is amax / 448, 448 the largest e4m3 value; amax below 1e-30 counts
// as 1e-30, so the scale and its reciprocal stay normal numbers and a group of zeros
// gives zeros.  Values are multiplied by the reciprocal of the rounded scale, at most
// 448 (1 + 2^-22), and the conversion saturates: no finite value of a finite group
// becomes NaN.  A NaN or an infinity in the group makes its scale NaN or infinite,
// and the values that carry it NaN: y / scale, as the formula says.
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
  float amax = __uint_as_float(amax_bits);
  if (amax < 1e-30f) amax = 1e-30f;
  return __fdiv_rn(amax, 448.0f);
}

__device__ __forceinline__ uint2 quantize_octet(const float (&v)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(v[4 * i] * inv, v[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

// VEC: q rows 8-byte aligned with whole octets.  8 o < d < 2^32.
template <bool VEC>
__device__ __forceinline__ void store_q_octet(uint8_t* row, uint32_t o, uint32_t d, uint2 q) {
  uint8_t* to = row + 8ull * o;
  if constexpr (VEC) {
    *reinterpret_cast<uint2*>(to) = q;
    return;
  }
  if (d - 8 * o < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * o + i < d) to[i] = static_cast<uint8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
    return;
  }
  // bytes up to the first 4-byte boundary, the word there, the bytes behind it
  const uint32_t head = static_cast<uint32_t>(-reinterpret_cast<uintptr_t>(to)) & 3;
  if (head == 0) {
    reinterpret_cast<uint32_t*>(to)[0] = q.x;
    reinterpret_cast<uint32_t*>(to)[1] = q.y;
  } else {
    if (head & 1) to[0] = static_cast<uint8_t>(q.x);
    if (head & 2)
      *reinterpret_cast<uint16_t*>(to + (head & 1)) =
          static_cast<uint16_t>(q.x >> (8 * (head & 1)));
    *reinterpret_cast<uint32_t*>(to + head) = __funnelshift_r(q.x, q.y, 8 * head);
    // 4 - head bytes are left behind the word: 3, 2 or 1
    if (head != 3)
      *reinterpret_cast<uint16_t*>(to + head + 4) = static_cast<uint16_t>(q.y >> (8 * head));
    if (head & 1) to[7] = static_cast<uint8_t>(q.y >> 24);
  }
}

// ------------------------------------------------------------ one kernel after another
//
// Kernels of one call run in order; each is launched while the one before it still runs
// (programmatic dependent launch) and waits, in hardware, for its results here.  What the kernel
// before may have written is therefore not constant for this kernel's life: no load of these
// kernels takes the read-only path (__ldg, const __restrict__), which the wait does not order.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launches a kernel that may start while the one before it on the stream still runs, its CTAs in
// clusters of `cluster`.  The kernel waits (wait_for_previous) before it touches memory.
struct Launch {
  dim3 grid;
  int threads;
  size_t smem = 0;
  cudaStream_t stream = nullptr;
  uint32_t cluster = 1;
};

template <typename... P>
inline cudaError_t launch(const Launch& l, void (*fn)(P...), P... args) {
  cudaLaunchAttribute attr[2];
  int n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n++].val.programmaticStreamSerializationAllowed = 1;
  if (l.cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = l.cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = l.grid;
  cfg.blockDim = dim3(l.threads);
  cfg.dynamicSmemBytes = l.smem;
  cfg.stream = l.stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}
template <typename P>
inline cudaError_t launch_after(void (*fn)(P), dim3 grid, int threads, size_t smem, cudaStream_t s,
                                const P& p, uint32_t cluster = 1) {
  return launch(Launch{grid, threads, smem, s, cluster}, fn, P(p));
}

}  // namespace cpl

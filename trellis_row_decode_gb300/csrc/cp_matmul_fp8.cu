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
#include "cp_matmul_fp8.h"
#include "cp_tcgen05.cuh"

namespace {

using namespace cpl;
using cpm::MatmulParams;

// ---------------------------------------------------- rows on any byte boundary
//
// 128 x 64 outputs per CTA, eight warps of 32 x 32.  A group's bytes are loaded as aligned words
// and shifted into place, widened to fp16 (exact) once on their way to shared memory, and
// multiplied by the warp-level fp16 product with fp32 sums: widening in front of every e4m3
// product instead, as the warp-level e4m3 instruction does, took 46 us on 3000 x 700 x 900.
// The next group's words are in flight while the tensor core works on this one's.

constexpr int kTileRows = 128, kTileCols = 64;           // rows of a and of w per CTA
constexpr int kAnyThreads = 256;
constexpr int kPitch = 128 * 2 + 16;                     // shared row pitch: no bank conflicts
constexpr int kPieces = (kTileRows + kTileCols) * 8 / kAnyThreads;   // 16-byte pieces of a thread
constexpr int kAnySmem = (kTileRows + kTileCols) * kPitch;

// d = a (16 x 32) * b (32 x 8) + d on the tensor core, e4m3 operands.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d = a (16 x 16) * b (16 x 8) + d, fp16 operands.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Sixteen bytes from row + col on, zeros behind the row's k bytes.  Words that reach outside
// the row are read byte by byte.
__device__ __forceinline__ uint4 load_any_piece(const uint8_t* row, uint32_t col, uint32_t k) {
  uint32_t w[4] = {};
  const uint8_t* p = row + col;
  const uint32_t skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3);
  if (col >= skew && static_cast<uint64_t>(col) + (skew != 0 ? 20 - skew : 16) <= k) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p - skew);
    uint32_t x[5];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __ldg(q + i);
    x[4] = skew != 0 ? __ldg(q + 4) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(x[i], x[i + 1], 8 * skew);
  } else {
#pragma unroll
    for (int b = 0; b < 16; ++b)
      if (static_cast<uint64_t>(col) + b < k) w[b / 4] |= static_cast<uint32_t>(p[b]) << (8 * (b & 3));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four e4m3 bytes as fp16.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
  const __half2_raw hi =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
  return make_uint2(lo.x | static_cast<uint32_t>(lo.y) << 16,
                    hi.x | static_cast<uint32_t>(hi.y) << 16);
}

__global__ void __launch_bounds__(kAnyThreads, 2) matmul_any_kernel(MatmulParams p) {
  extern __shared__ __align__(16) uint8_t tile[];        // rows of a, then rows of w
  const uint32_t tiles_n = (p.n + kTileCols - 1) / kTileCols;
  const uint32_t row0 = blockIdx.x / tiles_n * kTileRows, col0 = blockIdx.x % tiles_n * kTileCols;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t wr = (warp >> 1) * 32, wc = (warp & 1) * 32;
  const uint32_t g = lane >> 2, t = lane & 3;
  const uint32_t base = cpt::smem_addr(tile);
  wait_for_previous();
  uint4 v[kPieces];
  auto fetch = [&](uint32_t k0) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t piece = threadIdx.x + i * kAnyThreads, r = piece / 8;
      const bool of_a = r < kTileRows;
      const uint32_t row = of_a ? row0 + r : col0 + r - kTileRows;
      const uint32_t col = k0 + piece % 8 * 16;
      v[i] = make_uint4(0, 0, 0, 0);
      if (row < (of_a ? p.m : p.n) && col < p.k)
        v[i] = load_any_piece(of_a ? p.a + row * p.lda : p.w + row * p.ldw, col, p.k);
    }
  };
  float acc[2][4][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
  const float* sw = p.sw + static_cast<uint64_t>(col0 / 128) * p.groups;
  // this lane's row and half of k in the 16 x 16 (a) and 8 x 16 pairs (w) that ldmatrix loads
  const uint32_t at_a = base + (wr + (lane & 15)) * kPitch + (lane >> 4) * 16;
  const uint32_t at_w =
      base + (kTileRows + wc + (lane & 7) + (lane >> 4) * 8) * kPitch + (lane >> 3 & 1) * 16;
  if (p.groups != 0) fetch(0);
  for (uint32_t kb = 0; kb < p.groups; ++kb) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t piece = threadIdx.x + i * kAnyThreads;
      const uint2 a = widen4(v[i].x), b = widen4(v[i].y), c = widen4(v[i].z), d = widen4(v[i].w);
      uint4* to = reinterpret_cast<uint4*>(tile + piece / 8 * kPitch + piece % 8 * 32);
      to[0] = make_uint4(a.x, a.y, b.x, b.y);
      to[1] = make_uint4(c.x, c.y, d.x, d.y);
    }
    __syncthreads();
    if (kb + 1 < p.groups) fetch((kb + 1) * 128);
    float c[2][4][4] = {};
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t fa[2][4], fb[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        load_matrices(fa[i], at_a + i * 16 * kPitch + ks * 32);
        load_matrices(fb[i], at_w + i * 16 * kPitch + ks * 32);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_f16(c[i][j], fa[i], fb[j / 2][j % 2 * 2], fb[j / 2][j % 2 * 2 + 1]);
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

// ------------------------------------------------------------------- few rows of a
//
// Up to 64 rows of a: the product reads w once and little else, so it is bound by memory.
// A warp has 16 rows of w (the tensor core's 16 x 32 operand) and every 8th group of 128 of
// the CTA's share of k; its lanes load whole 16-byte pieces straight into fragments (the same
// order of k on both operands, whatever it is, gives the same sums), several groups ahead.
// The eight warps' sums are added in order through shared memory, and those of the
// `splits` CTAs of a cluster, which share the rows when w has few, through theirs.
// 1 x 1024 x 1024: 2.9 us; bound by latency there, by the warp-level product beyond 10 MB of w.

// Which kernel takes operands on 16-byte boundaries.  Few rows of a and little of w: this one
// (1 x 1024 x 1024: 3.0 us against the thin kernel's 4.9; 16 x 1024 x 1024: 3.8 against 4.9; with
// 17 MB of w they are even, 6.3 us, and with 101 MB the thin one leads, 20 us against 28: the
// warp-level e4m3 product costs about 70 clocks each).  Up to 128 rows of a: the thin kernel
// (128 x 4096 x 24576: 31 us against the pairs' 42; 128 x 4096 x 4096: 10.8 against 13.7; at 256 rows
// 54 against 43 and 14.9 against 14.1).  More: the pairs.  Rows on other boundaries: this one for
// few rows of a whatever the size of w, matmul_any_kernel for more.
constexpr uint32_t kFewRows = 16;
constexpr uint64_t kFewBytes = 8 << 20;
constexpr uint32_t kThinRows = 128;
constexpr int kFewThreads = 256;
constexpr uint32_t kFewWarps = kFewThreads / 32;

struct FewGroup {
  uint4 w[2][2];           // rows g and g + 8; bytes 16 t.. and 64 + 16 t..
};

template <int kTokens>
struct FewRows {
  uint4 b[kTokens][2];
  float scale[kTokens][2];
  float scale_w;
};

// Sixteen bytes of a row of w (read once: not kept in L1) or of a.
template <bool kAligned>
__device__ __forceinline__ uint4 load_piece(const uint8_t* row, uint32_t col, uint32_t k) {
  if (kAligned && static_cast<uint64_t>(col) + 16 <= k) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(row + col));
    return v;
  }
  return load_any_piece(row, col, k);
}
template <bool kAligned>
__device__ __forceinline__ uint4 load_piece_cached(const uint8_t* row, uint32_t col, uint32_t k) {
  if (kAligned && static_cast<uint64_t>(col) + 16 <= k)
    return __ldg(reinterpret_cast<const uint4*>(row + col));
  return load_any_piece(row, col, k);
}

// kTokens: rows of a / 8.  kAhead: groups of w in flight per warp.  kAligned: rows on 16-byte
// boundaries.
template <int kTokens, int kAhead, bool kAligned>
__global__ void __launch_bounds__(kFewThreads, 2) matmul_few_kernel(MatmulParams p, uint32_t splits) {
  __shared__ float part[kFewWarps][16][kTokens * 8];
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t g = lane >> 2, t = lane & 3;
  const uint32_t rank = splits == 1 ? 0 : cpt::cluster_rank();
  const uint32_t row0 = blockIdx.x / splits * 16;
  const uint32_t first = rank * kFewWarps + warp, step = splits * kFewWarps;
  const bool live[2] = {row0 + g < p.n, row0 + g + 8 < p.n};
  const uint8_t* wrow[2] = {p.w + static_cast<uint64_t>(live[0] ? row0 + g : 0) * p.ldw,
                            p.w + static_cast<uint64_t>(live[1] ? row0 + g + 8 : 0) * p.ldw};
  const float* sw = p.sw + static_cast<uint64_t>(row0 / 128) * p.groups;
  FewGroup ring[kAhead];
  wait_for_previous();
  auto fetch = [&](FewGroup& f, uint32_t kb) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        f.w[r][h] = kb < p.groups && live[r]
                        ? load_piece<kAligned>(wrow[r], kb * 128 + 64 * h + 16 * t, p.k)
                        : make_uint4(0, 0, 0, 0);
  };
  // The rows of a and the scales of a group, one group ahead of their use.
  FewRows<kTokens> rows;
  auto fetch_rows = [&](uint32_t kb) {
    const bool in = kb < p.groups;
    rows.scale_w = in ? __ldg(sw + kb) : 0.0f;
#pragma unroll
    for (int n = 0; n < kTokens; ++n) {
      const uint32_t row = 8 * n + g, c0 = 8 * n + 2 * t;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        rows.b[n][h] = in && row < p.m
                           ? load_piece_cached<kAligned>(p.a + static_cast<uint64_t>(row) * p.lda,
                                               kb * 128 + 64 * h + 16 * t, p.k)
                           : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        rows.scale[n][e] =
            in && c0 + e < p.m ? __ldg(p.sa + static_cast<uint64_t>(c0 + e) * p.groups + kb) : 0.0f;
    }
  };
  float acc[kTokens][4];
#pragma unroll
  for (int n = 0; n < kTokens; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(ring[i], first + i * step);
  fetch_rows(first);
  for (uint32_t kb0 = first; kb0 < p.groups; kb0 += kAhead * step) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint32_t kb = kb0 + i * step;
      if (kb < p.groups) {
        const FewRows<kTokens> now = rows;
        fetch_rows(kb + step);
#pragma unroll
        for (int n = 0; n < kTokens; ++n) {
          float c[4] = {};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 &x = ring[i].w[0][h], &y = ring[i].w[1][h];
            mma_e4m3(c, {x.x, y.x, x.y, y.y}, now.b[n][h].x, now.b[n][h].y);
            mma_e4m3(c, {x.z, y.z, x.w, y.w}, now.b[n][h].z, now.b[n][h].w);
          }
          const float f0 = now.scale[n][0] * now.scale_w, f1 = now.scale[n][1] * now.scale_w;
          acc[n][0] = fmaf(f0, c[0], acc[n][0]);
          acc[n][1] = fmaf(f1, c[1], acc[n][1]);
          acc[n][2] = fmaf(f0, c[2], acc[n][2]);
          acc[n][3] = fmaf(f1, c[3], acc[n][3]);
        }
        fetch(ring[i], kb + kAhead * step);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < kTokens; ++n) {
    *reinterpret_cast<float2*>(&part[warp][g][8 * n + 2 * t]) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(&part[warp][g + 8][8 * n + 2 * t]) =
        make_float2(acc[n][2], acc[n][3]);
  }
  __syncthreads();
  // output (token, row): consecutive threads take consecutive rows of w
  for (uint32_t i = threadIdx.x; i < kTokens * 8 * 16; i += kFewThreads) {
    const uint32_t r = i % 16, token = i / 16;
    float s = part[0][r][token];
#pragma unroll
    for (uint32_t w = 1; w < kFewWarps; ++w) s += part[w][r][token];
    if (splits == 1) {
      if (token < p.m && row0 + r < p.n)
        store_from_f32(p.out, token * p.ldo + row0 + r, p.out_dtype, s);
    } else {
      part[0][r][token] = s;         // read by this thread alone before
    }
  }
  if (splits == 1) return;
  cpt::cluster_sync();
  if (rank == 0) {
    for (uint32_t i = threadIdx.x; i < kTokens * 8 * 16; i += kFewThreads) {
      const uint32_t r = i % 16, token = i / 16;
      const uint32_t at = cpt::smem_addr(&part[0][r][token]);
      float s = part[0][r][token];
      for (uint32_t q = 1; q < splits; ++q) {
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cpt::map_rank(at, q)));
        s += v;
      }
      if (token < p.m && row0 + r < p.n)
        store_from_f32(p.out, token * p.ldo + row0 + r, p.out_dtype, s);
    }
  }
  cpt::cluster_sync();               // no CTA leaves while another may read its shared memory
}

template <int kTokens, int kAhead, bool kAligned>
cudaError_t launch_few(const MatmulParams& p, uint32_t splits, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((p.n + 15) / 16 * splits);
  cfg.blockDim = dim3(kFewThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = splits == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, &matmul_few_kernel<kTokens, kAhead, kAligned>, p, splits);
}

cp_status launch_few(const MatmulParams& p, bool aligned, cudaStream_t s) {
  // Share rows among CTAs until there are about two per SM, as long as each warp keeps two
  // groups or more.
  uint32_t splits = 1;
  while (splits < 8 && static_cast<uint64_t>((p.n + 15) / 16) * splits < 256 &&
         p.groups >= 2 * kFewWarps * 2 * splits)
    splits *= 2;
  cudaError_t e;
  if (p.m <= 8)
    e = aligned ? launch_few<1, 4, true>(p, splits, s) : launch_few<1, 2, false>(p, splits, s);
  else
    e = aligned ? launch_few<2, 3, true>(p, splits, s) : launch_few<2, 2, false>(p, splits, s);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul launch");
  return CP_OK;
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
  // Tensor maps want 16-byte boundaries (and a row stride of their own: not one row for all).
  if (k != 0 && cpx::aligned(a, 16) && cpx::aligned(w, 16) &&
      (m == 1 || (a_stride % 16 == 0 && a_stride != 0)) &&
      (n == 1 || (w_stride % 16 == 0 && w_stride != 0)))
    return m > kThinRows                          ? cpm::launch_pairs(p, s)
           : m <= kFewRows && n * k <= kFewBytes ? launch_few(p, true, s)
                                                 : cpm::launch_thin(p, s);
  if (m <= kFewRows) return launch_few(p, false, s);
  const uint64_t tiles =
      ((m + kTileRows - 1) / kTileRows) * ((n + kTileCols - 1) / kTileCols);
  if (tiles >= kMost) {
    cpx::set_error("m and n make more than 2^31 tiles");
    return CP_ERR_INVALID_ARG;
  }
  cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&matmul_any_kernel),
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kAnySmem);
  if (e == cudaSuccess) {
    e = launch_after(&matmul_any_kernel, dim3(static_cast<unsigned>(tiles)), kAnyThreads, kAnySmem, s,
                     p);
  }
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul launch");
  return CP_OK;
}

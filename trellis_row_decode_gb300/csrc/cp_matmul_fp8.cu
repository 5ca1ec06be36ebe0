// cp_matmul_fp8.cu -- product of e4m3 matrices with a scale for each block of 128
// (include/cp.h, cp_matmul_fp8).
//
//   out[i][j] = sum over g of sa[i][g] sw[j / 128][g] * (a[i] . w[j] over group g)
//
// The products of a group are exact in the tensor core's fp32 sums; a group's sum is
// scaled and added to the running fp32 sum before the next group begins.
#include <algorithm>
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

// d = a (16 x 32) * b (32 x 8) + d on the tensor core, e4m3 operands.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Sixteen bytes from row + col on, zeros behind the row's k bytes: shifted out of two aligned
// pieces, or byte by byte where those reach outside the row.
__device__ __forceinline__ uint4 load_any_piece(const uint8_t* row, uint32_t col, uint32_t k) {
  const uint8_t* p = row + col;
  const uint32_t skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15);
  if (col >= skew && static_cast<uint64_t>(col) + (skew != 0 ? 32 - skew : 16) <= k) {
    const uint4* q = reinterpret_cast<const uint4*>(p - skew);
    const uint4 lo = q[0], hi = skew != 0 ? q[1] : make_uint4(0, 0, 0, 0);
    uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (skew & 8) {
#pragma unroll
      for (int i = 0; i < 6; ++i) x[i] = x[i + 2];
    }
    if (skew & 4) {
#pragma unroll
      for (int i = 0; i < 5; ++i) x[i] = x[i + 1];
    }
    const uint32_t bits = 8 * (skew & 3);
    return make_uint4(__funnelshift_r(x[0], x[1], bits), __funnelshift_r(x[1], x[2], bits),
                      __funnelshift_r(x[2], x[3], bits), __funnelshift_r(x[3], x[4], bits));
  }
  uint32_t w[4] = {};
#pragma unroll
  for (int b = 0; b < 16; ++b)
    if (static_cast<uint64_t>(col) + b < k) w[b / 4] |= static_cast<uint32_t>(p[b]) << (8 * (b & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------- rows on any byte boundary
//
// Tensor maps want rows on 16-byte boundaries.  Operands that lie elsewhere are copied to such
// rows, zeros behind their ends, in the caller's workspace, in one launch for both; the product
// starts while the copy ends.  A warp moves 2 KB of a row at a time, four pieces a lane in flight.
// Bound by memory; the product then costs what it costs on such rows from the start.
// 101 MB of w: 35 us at 5.8 TB/s read and written; 466 x 827 x 22133: 31.6 us in all,
// 2048 x 2048 x 2047 17.4 (14.1 for the product of rows on 16-byte boundaries).  A warp-level fp16
// product of the shifted bytes, without a copy, ran at 125 TFLOP/s and took 738 and 137.

constexpr int kAlignThreads = 256;
constexpr uint64_t kAlignCtas = 152 * 6;                  // as many as run at once
constexpr uint32_t kAlignPieces = 4;                      // 16-byte pieces of a lane
constexpr uint32_t kAlignBytes = 32 * 16 * kAlignPieces;  // of a row, by one warp at a time

struct AlignOperand {
  const uint8_t* from;
  uint8_t* to;
  uint64_t ld, rows;       // rows: 0 for an operand that stays where it is
};
struct AlignParams {
  AlignOperand of[2];
  uint32_t k, chunks;      // chunks of kAlignBytes in a row
  uint64_t pitch;
};

__global__ void __launch_bounds__(kAlignThreads) align_rows_kernel(AlignParams p) {
  wait_for_previous();
  let_next_start();
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t warps = static_cast<uint64_t>(gridDim.x) * (kAlignThreads / 32);
  const uint64_t units = (p.of[0].rows + p.of[1].rows) * p.chunks;
  for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * (kAlignThreads / 32) + threadIdx.x / 32;
       u < units; u += warps) {
    uint64_t row = u / p.chunks;
    const uint32_t col = static_cast<uint32_t>(u - row * p.chunks) * kAlignBytes + lane * 16;
    const bool second = row >= p.of[0].rows;
    if (second) row -= p.of[0].rows;
    const uint8_t* from = (second ? p.of[1].from : p.of[0].from) +
                          row * (second ? p.of[1].ld : p.of[0].ld);
    uint8_t* to = (second ? p.of[1].to : p.of[0].to) + row * p.pitch;
    uint4 v[kAlignPieces];
#pragma unroll
    for (uint32_t i = 0; i < kAlignPieces; ++i)
      if (col + i * 512 < p.k) v[i] = load_any_piece(from, col + i * 512, p.k);
#pragma unroll
    for (uint32_t i = 0; i < kAlignPieces; ++i)
      if (col + i * 512 < p.k) *reinterpret_cast<uint4*>(to + col + i * 512) = v[i];
  }
}

// Rows that a tensor map takes (and a row stride of their own: not one row for all).
bool rows_ok(const void* p, uint64_t stride, uint64_t rows) {
  return cpx::aligned(p, 16) && (rows == 1 || (stride % 16 == 0 && stride != 0));
}

uint64_t aligned_pitch(uint64_t k) { return (k + 15) / 16 * 16; }

// ------------------------------------------------------------------- few rows of a
//
// Up to 16 rows of a and 8 MB of w (kFewRows, kFewBytes): the product reads w once and little
// else, and is over in a few microseconds, so what counts is how soon the loads are under way.
// A warp has 16 rows of w (the tensor core's 16 x 32 operand) and every 8th group of 128 of
// the CTA's share of k; its lanes load whole 16-byte pieces straight into fragments (the same
// order of k on both operands, whatever it is, gives the same sums), several groups ahead.
// The eight warps' sums are added in order through shared memory, and those of the
// `splits` CTAs of a cluster, which share the rows when w has few, through theirs.
// 1 x 1024 x 1024: 3.1 us; bound by latency there, by the warp-level product beyond 10 MB of w.

// Which kernel takes operands on 16-byte boundaries.  Few rows of a and little of w: this one
// (1 x 1024 x 1024: 3.1 us against the thin kernel's 4.9; 16 x 1024 x 1024: 3.8 against 4.9; with
// 17 MB of w they are even, 6.3 us, and with 101 MB the thin one leads, 20 us against 28: the
// warp-level e4m3 product costs about 70 clocks each).  Up to 128 rows of a: the thin kernel
// (128 x 4096 x 24576: 31 us against the pairs' 42; 128 x 4096 x 4096: 10.8 against 13.7; at 256 rows
// 54 against 43 and 14.9 against 14.1).  More: the pairs.  Rows on other boundaries: the
// same rule, with align_rows_kernel in front of the thin kernel and the pairs (1 x 4096 x 4097:
// 12.2 us against 11.0 here; 16 x 4096 x 24577: 55 against 103).
constexpr uint32_t kFewRows = 16;
constexpr uint64_t kFewBytes = 8 << 20;
constexpr uint32_t kThinRows = 128;
constexpr uint64_t kMost = 1ull << 31;                   // m, n and k stay below
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
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(row + col));
    return v;
  }
  return load_any_piece(row, col, k);
}
template <bool kAligned>
__device__ __forceinline__ uint4 load_piece_cached(const uint8_t* row, uint32_t col, uint32_t k) {
  if (kAligned && static_cast<uint64_t>(col) + 16 <= k)
    return *reinterpret_cast<const uint4*>(row + col);
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
    rows.scale_w = in ? sw[kb] : 0.0f;
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
            in && c0 + e < p.m ? p.sa[static_cast<uint64_t>(c0 + e) * p.groups + kb] : 0.0f;
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
        __syncwarp();                // (a lane's pieces at a row's end take a branch of their own)
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

namespace {
bool few_rows(uint64_t m, uint64_t n, uint64_t k) { return m <= kFewRows && n * k <= kFewBytes; }
}  // namespace

extern "C" uint64_t cp_matmul_fp8_workspace_bytes(const uint8_t* a, uint64_t a_stride,
                                                  const uint8_t* w, uint64_t w_stride, uint64_t m,
                                                  uint64_t n, uint64_t k) {
  if (m >= kMost || n >= kMost || k >= kMost - 128 || m == 0 || n == 0 || k == 0 ||
      few_rows(m, n, k))
    return 0;
  return ((rows_ok(a, a_stride, m) ? 0 : m) + (rows_ok(w, w_stride, n) ? 0 : n)) *
         aligned_pitch(k);
}

extern "C" cp_status cp_matmul_fp8(const uint8_t* a, uint64_t a_stride, const float* a_scales,
                                   const uint8_t* w, uint64_t w_stride, const float* w_scales,
                                   uint64_t m, uint64_t n, uint64_t k, void* out, int out_dtype,
                                   uint64_t out_stride, void* workspace, uint64_t workspace_bytes,
                                   void* stream) {
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
  if (k == 0) {                      // sums over nothing; zero is all zero bits in each type
    const uint64_t size = dtype_size(out_dtype);
    const cudaError_t e = cudaMemset2DAsync(out, out_stride * size, 0, n * size, m, s);
    return e == cudaSuccess ? CP_OK : cpx::cuda_fail(e, "fp8 matmul, k = 0");
  }
  const bool a_ok = rows_ok(a, a_stride, m), w_ok = rows_ok(w, w_stride, n);
  if (few_rows(m, n, k))
    return launch_few(p, a_ok && w_ok, s);
  const uint64_t need = cp_matmul_fp8_workspace_bytes(a, a_stride, w, w_stride, m, n, k);
  if (need != 0) {
    if (workspace == nullptr || !cpx::aligned(workspace, 16) || workspace_bytes < need) {
      cpx::set_error("workspace must be 16-byte aligned and hold cp_matmul_fp8_workspace_bytes bytes");
      return CP_ERR_INVALID_ARG;
    }
    AlignParams c{};
    c.k = p.k;
    c.pitch = aligned_pitch(k);
    c.chunks = (p.k + kAlignBytes - 1) / kAlignBytes;
    uint8_t* to = static_cast<uint8_t*>(workspace);
    if (!a_ok) {
      c.of[0] = AlignOperand{a, to, a_stride, m};
      p.a = to;
      p.lda = c.pitch;
      to += m * c.pitch;
    }
    if (!w_ok) {
      c.of[1] = AlignOperand{w, to, w_stride, n};
      p.w = to;
      p.ldw = c.pitch;
    }
    const uint64_t units = (c.of[0].rows + c.of[1].rows) * c.chunks;
    const uint64_t ctas = (units + kAlignThreads / 32 - 1) / (kAlignThreads / 32);
    const cudaError_t e =
        launch_after(&align_rows_kernel, dim3(static_cast<unsigned>(std::min(ctas, kAlignCtas))),
                     kAlignThreads, 0, s, c);
    if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul launch");
  }
  return m > kThinRows ? cpm::launch_pairs(p, s) : cpm::launch_thin(p, s);
}

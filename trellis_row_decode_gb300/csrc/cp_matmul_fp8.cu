// cp_matmul_fp8.cu -- product of e4m3 matrices with a scale for each block of 128
// (include/cp.h, cp_matmul_fp8).
//
//   out[i][j] = sum over g of sa[i][g] sw[j / 128][g] * (a[i] . w[j] over group g)
//
// The products of a group are exact in the tensor core's fp32 sums; a group's sum is
// scaled and added to the running fp32 sum before the next group begins.
#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "cp.h"
#include "cp_internal.h"
#include "cp_layer.cuh"
#include "cp_tcgen05.cuh"

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

// ------------------------------------------------------------------- few rows of a
//
// Up to 64 rows of a: the product reads w once and little else, so it is bound by memory.
// A warp has 16 rows of w (the tensor core's 16 x 32 operand) and every 8th group of 128 of
// the CTA's share of k; its lanes load whole 16-byte pieces straight into fragments (the same
// order of k on both operands, whatever it is, gives the same sums), several groups ahead.
// The eight warps' sums are added in order through shared memory, and those of the
// `splits` CTAs of a cluster, which share the rows when w has few, through theirs.

constexpr uint32_t kFewRows = 16;
constexpr uint64_t kFewBytes = 8 << 20;
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

// Sixteen bytes of a row from column `col` on, zeros behind the row's k bytes.
__device__ __forceinline__ uint4 load_piece(const uint8_t* row, uint32_t col, uint32_t k) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (col + 16 <= k) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(row + col));
  } else if (col < k) {
    uint32_t u[4] = {};
    for (uint32_t b = 0; col + b < k; ++b)
      u[b / 4] |= static_cast<uint32_t>(row[col + b]) << (8 * (b & 3));
    v = make_uint4(u[0], u[1], u[2], u[3]);
  }
  return v;
}
__device__ __forceinline__ uint4 load_piece_cached(const uint8_t* row, uint32_t col, uint32_t k) {
  if (col + 16 <= k) return __ldg(reinterpret_cast<const uint4*>(row + col));
  return load_piece(row, col, k);
}

// kTokens: rows of a / 8.  kAhead: groups of w in flight per warp.
template <int kTokens, int kAhead>
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
  auto fetch = [&](FewGroup& f, uint32_t kb) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        f.w[r][h] = kb < p.groups && live[r] ? load_piece(wrow[r], kb * 128 + 64 * h + 16 * t, p.k)
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
                           ? load_piece_cached(p.a + static_cast<uint64_t>(row) * p.lda,
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

template <int kTokens, int kAhead>
cudaError_t launch_few(const MatmulParams& p, uint32_t splits, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((p.n + 15) / 16 * splits);
  cfg.blockDim = dim3(kFewThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = splits == 1 ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, &matmul_few_kernel<kTokens, kAhead>, p, splits);
}

cp_status launch_few(const MatmulParams& p, cudaStream_t s) {
  // Share rows among CTAs until there are about two per SM, as long as each warp keeps two
  // groups or more.
  uint32_t splits = 1;
  while (splits < 8 && static_cast<uint64_t>((p.n + 15) / 16) * splits < 256 &&
         p.groups >= 2 * kFewWarps * 2 * splits)
    splits *= 2;
  cudaError_t e;
  if (p.m <= 8) e = launch_few<1, 4>(p, splits, s);
  else e = launch_few<2, 3>(p, splits, s);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul launch");
  return CP_OK;
}

// ------------------------------------------------- rows on 16-byte boundaries: tcgen05
//
// A pair of CTAs (two SMs) makes 256 x bn outputs, bn a multiple of 32 up to 256.  Each
// CTA stages its 128 rows of a and its half of the bn rows of w (128 bytes of k a stage,
// 128-byte swizzle), so a byte that enters an SM feeds both tensor cores.  Roles: one
// thread per CTA issues the TMA loads; one thread of the first CTA issues four
// tcgen05.mma (k = 32 each) per group of 128 into one of two tensor-memory buffers; eight
// warps per CTA read the other buffer, scale it and add it to their registers (a lane has
// a row, a warp half of the columns).  The scales differ from group to group, so the
// running sum cannot stay in tensor memory; the two buffers let the tensor core work on
// the next group meanwhile.  With few tiles, `splits` pairs of one cluster share a tile's
// groups and add their sums, in the order of the pairs, through distributed shared memory.

constexpr int kSumWarps = 8;
constexpr int kTcThreads = (kSumWarps + 4) * 32;       // + the TMA warp, the MMA warp and two idle
// Registers: launched with 168 a thread (65,536 over 12 warps); the summing warps (128 sums and 64
// values in flight a thread) take what the other four give up.
constexpr int kLaunchRegs = 168, kSumRegs = 208, kOtherRegs = 88;
static_assert(2 * kSumRegs + kOtherRegs <= 3 * kLaunchRegs, "a warpgroup's share of the launch");
constexpr uint32_t kMaxStages = 8;
constexpr uint32_t kTileA = 128 * 128;                 // bytes of a's rows per stage and CTA
constexpr uint32_t kSmemMost = 224 * 1024;             // dynamic shared memory of a CTA

// A wait that ran out sets this word; cp_matmul_fp8_status reads and clears it.
__device__ uint32_t g_matmul_gave_up;

struct TcParams {
  const float* sa;
  const float* sw;
  void* out;
  uint64_t ldo;
  uint32_t m, n, groups;
  int out_dtype;
  uint32_t tiles_m, tiles, stages, splits, tmem_columns;
  uint32_t a_rows;          // rows of a's TMA box
  uint32_t out_align;       // 32, 16 or 0: bytes on whose boundaries out's rows lie
};

// Eight consecutive outputs of a row.
__device__ __forceinline__ void store8(const TcParams& p, uint32_t row, uint32_t col,
                                       const float* v) {
  const uint64_t at = static_cast<uint64_t>(row) * p.ldo + col;
  if (p.out_align >= 16 && col + 8 <= p.n) {
    if (p.out_dtype == CP_F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = v[e];
      if (p.out_dtype == CP_F16) store_octet(static_cast<__half*>(p.out) + at, pack<__half>(u));
      else store_octet(static_cast<__nv_bfloat16*>(p.out) + at, pack<__nv_bfloat16>(u));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < p.n) store_from_f32(p.out, at + e, p.out_dtype, v[e]);
  }
}

// Sixteen, whole 32-byte sectors of L2 where the rows allow it: a lane's outputs are its own
// row's, so only whole sectors keep the writes from being merged in L2.
__device__ __forceinline__ void store16(const TcParams& p, uint32_t row, uint32_t col,
                                        const float* v) {
  if (p.out_dtype != CP_F32 && p.out_align >= 32 && col + 16 <= p.n) {
    Packed<float> r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = v[8 * h + e];
      if (p.out_dtype == CP_F16) {
        const Packed<__half> x = pack<__half>(u);
#pragma unroll
        for (int e = 0; e < 4; ++e) r.w[4 * h + e] = x.w[e];
      } else {
        const Packed<__nv_bfloat16> x = pack<__nv_bfloat16>(u);
#pragma unroll
        for (int e = 0; e < 4; ++e) r.w[4 * h + e] = x.w[e];
      }
    }
    store_octet(reinterpret_cast<float*>(static_cast<uint16_t*>(p.out) +
                                         static_cast<uint64_t>(row) * p.ldo + col), r);
  } else {
    store8(p, row, col, v);
    store8(p, row, col + 8, v + 8);
  }
}

// f(std::integral_constant) for 0 .. kCount - 1.
template <uint32_t kCount, typename F, uint32_t kFrom = 0>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (kFrom < kCount) {
    f(std::integral_constant<uint32_t, kFrom>{});
    static_for<kCount, F, kFrom + 1>(static_cast<F&&>(f));
  }
}

// Up to 32 columns of a warp's share of 8 * kEights, from column 32 * kChunk on.
template <uint32_t kEights, uint32_t kChunk>
__device__ __forceinline__ void load_chunk(float (&x)[32], uint32_t at) {
  constexpr uint32_t kLeft = kEights - 4 * kChunk;
  if constexpr (kLeft >= 4) {
    cpt::tmem_load32<0>(x, at + 32 * kChunk);
  } else {
    if constexpr ((kLeft & 2) != 0) cpt::tmem_load16<0>(x, at + 32 * kChunk);
    if constexpr ((kLeft & 1) != 0)
      cpt::tmem_load8<(kLeft & 2) * 8>(x, at + 32 * kChunk + (kLeft & 2) * 8);
  }
}

// acc += x * scale over those columns; those from `turn` eights on have the second scale.
template <uint32_t kEights, uint32_t kChunk>
__device__ __forceinline__ void add_chunk(float (&acc)[kEights * 8], const float (&x)[32],
                                          uint32_t turn, float scale0, float scale1) {
  constexpr uint32_t kLeft = kEights - 4 * kChunk, kHere = kLeft < 4 ? kLeft : 4;
#pragma unroll
  for (uint32_t c = 0; c < kHere; ++c) {
    const float f = 4 * kChunk + c < turn ? scale0 : scale1;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
      acc[32 * kChunk + 8 * c + i] = fmaf(x[8 * c + i], f, acc[32 * kChunk + 8 * c + i]);
  }
}

template <uint32_t kEights>            // columns of a warp's share / 8 = kBn / 16
__global__ void __launch_bounds__(kTcThreads, 1)
    matmul_tc_kernel(const __grid_constant__ CUtensorMap map_a,
                     const __grid_constant__ CUtensorMap map_w, const TcParams p) {
  constexpr uint32_t kBn = kEights * 16, kShare = kEights * 8;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 4];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cpt::cluster_rank();
  const uint32_t half = rank & 1, split = rank >> 1, first = rank & ~1u;
  const uint32_t stage_bytes = kTileA + kBn * 64;
  const uint32_t full = cpt::smem_addr(bars), empty = full + 8 * kMaxStages;
  const uint32_t acc_full = empty + 8 * kMaxStages, acc_empty = acc_full + 16;
  // the first CTA's barriers hold the pair's loads and reads
  const uint32_t pair_full = cpt::map_rank(full, first);
  const uint32_t pair_acc_empty = cpt::map_rank(acc_empty, first);

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < p.stages; ++s) {
      cpt::mbar_init(full + 8 * s, 1);
      cpt::mbar_init(empty + 8 * s, 1);
    }
    for (uint32_t b = 0; b < 2; ++b) {
      cpt::mbar_init(acc_full + 8 * b, 1);
      cpt::mbar_init(acc_empty + 8 * b, 2 * kSumWarps);
    }
    cpt::mbar_init_fence();
    gave_up = 0;
  }
  if (warp == kSumWarps + 1) cpt::tmem_alloc_pair(cpt::smem_addr(&tmem_base), p.tmem_columns);
  cpt::tc_fence_before();
  __syncthreads();
  cpt::cluster_sync();
  cpt::tc_fence_after();
  const uint32_t tmem = tmem_base;
  const uint32_t kb0 = static_cast<uint32_t>(static_cast<uint64_t>(p.groups) * split / p.splits);
  const uint32_t kb1 =
      static_cast<uint32_t>(static_cast<uint64_t>(p.groups) * (split + 1) / p.splits);
  const uint32_t step = gridDim.x / (2 * p.splits), tile0 = blockIdx.x / (2 * p.splits);

  if (warp >= kSumWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // Both warps run their loops whole and elect a thread to issue.
    if (warp == kSumWarps) {
      // -------------------------------------------------------------- loads
      if (cpt::elect_one()) {
        cpt::tma_prefetch_map(&map_a);
        cpt::tma_prefetch_map(&map_w);
      }
      __syncwarp();
      const uint32_t w_bytes = kBn * 64;
      uint32_t s = 0, round = 0;
      bool ok = true;
      for (uint32_t tile = tile0; tile < p.tiles && ok; tile += step) {
        const uint32_t tile_n = tile / p.tiles_m;
        const uint32_t row0 = (tile - tile_n * p.tiles_m) * 256, col0 = tile_n * kBn;
        const bool a1 = row0 + 128 < p.m;               // the second CTA has rows of a
        const bool mine = half == 0 || a1;
        const uint32_t bytes = 2 * w_bytes + (a1 ? 2 : 1) * p.a_rows * 128;
        for (uint32_t kb = kb0; kb < kb1; ++kb) {
          if (round > 0) {
            ok = cpt::mbar_wait(empty + 8 * s, (round - 1) & 1, &gave_up);
            if (!ok) break;
          }
          const uint32_t dst = cpt::smem_addr(tiles) + s * stage_bytes;
          if (cpt::elect_one()) {
            if (half == 0) cpt::mbar_expect(full + 8 * s, bytes);
            if (mine)
              cpt::tma_load_pair(dst, &map_a, kb * 128, row0 + half * 128, pair_full + 8 * s);
            cpt::tma_load_pair(dst + kTileA, &map_w, kb * 128, col0 + half * (kBn / 2),
                               pair_full + 8 * s);
          }
          __syncwarp();
          if (++s == p.stages) {
            s = 0;
            ++round;
          }
        }
      }
      // Given up: the loads in flight land before the CTA leaves (stages s.. of the round
      // before, stages ..s of this one).
      if (!ok && half == 0) {
        int unused = 0;
        for (uint32_t k = 0; k < p.stages; ++k) {
          const uint32_t r = k < s ? round : round - 1;
          if (k < s || round > 0) cpt::mbar_wait(full + 8 * k, r & 1, &unused);
        }
      }
    } else if (warp == kSumWarps + 1 && half == 0) {
      // ----------------------------------------------------------- products
      const uint32_t instr = cpt::e4m3_instr_desc(256, kBn);
      const uint16_t pair = static_cast<uint16_t>(3u << first);
      uint32_t it = 0, s = 0, round = 0;
      bool ok = true;
      for (uint32_t tile = tile0; tile < p.tiles && ok; tile += step) {
        for (uint32_t kb = kb0; kb < kb1; ++kb, ++it) {
          const uint32_t b = it & 1;
          ok = (it < 2 || cpt::mbar_wait(acc_empty + 8 * b, ((it >> 1) - 1) & 1, &gave_up)) &&
               cpt::mbar_wait(full + 8 * s, round & 1, &gave_up);
          if (!ok) break;
          cpt::tc_fence_after();
          const uint32_t at = cpt::smem_addr(tiles) + s * stage_bytes;
          const uint64_t da = cpt::operand_desc(at), dw = cpt::operand_desc(at + kTileA);
          if (cpt::elect_one()) {
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
              cpt::mma_pair(tmem + b * kBn, da + 2 * k, dw + 2 * k, instr, k != 0);
            cpt::mma_commit_pair(empty + 8 * s, pair);
            cpt::mma_commit_pair(acc_full + 8 * b, pair);
          }
          __syncwarp();
          if (++s == p.stages) {
            s = 0;
            ++round;
          }
        }
      }
    }
  } else {
    // ----------------------------------------------------------------- sums
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    const uint32_t lanes = (warp & 3) * 32;              // tensor-memory lanes of this warp
    const uint32_t share = (warp >> 2) * kShare;         // its first column of the tile
    const uint32_t tmem_warp = tmem + (lanes << 16) + share;
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t tile = tile0; tile < p.tiles && ok; tile += step) {
      const uint32_t tile_n = tile / p.tiles_m;
      const uint32_t row0 = (tile - tile_n * p.tiles_m) * 256 + half * 128 + lanes;
      const uint32_t row = row0 + lane;
      const uint32_t col = tile_n * kBn + share;
      const bool any = row0 < p.m && col < p.n;          // the warp has outputs
      const uint32_t turn = (128 - col % 128) / 8;       // eights from here on are in the next block
      constexpr uint32_t kChunks = (kEights + 3) / 4;    // of 32 columns, the last may be shorter
      float acc[kShare];
#pragma unroll
      for (uint32_t i = 0; i < kShare; ++i) acc[i] = 0.0f;
      if (!any) {
        for (uint32_t kb = kb0; kb < kb1 && ok; ++kb, ++it) {
          ok = cpt::mbar_wait(acc_full + 8 * (it & 1), (it >> 1) & 1, &gave_up);
          if (ok && lane == 0) cpt::mbar_arrive_cluster(pair_acc_empty + 8 * (it & 1));
        }
      } else {
        // scales are loaded two groups ahead, each into the registers of its parity
        const float* sa = p.sa + static_cast<uint64_t>(min(row, p.m - 1)) * p.groups;
        const uint32_t last = (p.n + 127) / 128 - 1;
        const float* sw0 = p.sw + static_cast<uint64_t>(col / 128) * p.groups;
        const float* sw1 = p.sw + static_cast<uint64_t>(min(col / 128 + 1, last)) * p.groups;
        float fa[2] = {}, f0[2] = {}, f1[2] = {};
        auto load_scales = [&](uint32_t k, uint32_t kb) {
          if (kb < kb1) {
            fa[k] = __ldg(sa + kb);
            f0[k] = __ldg(sw0 + kb);
            f1[k] = __ldg(sw1 + kb);
          }
        };
        load_scales(0, kb0);
        load_scales(1, kb0 + 1);
        float v[2][32];
        for (uint32_t kb = kb0; kb < kb1 && ok; kb += 2) {
#pragma unroll
          for (uint32_t k = 0; k < 2; ++k) {
            if (kb + k < kb1 && ok) {
              const uint32_t b = it & 1;
              const uint32_t at = tmem_warp + b * kBn;
              ok = cpt::mbar_wait(acc_full + 8 * b, (it >> 1) & 1, &gave_up);
              if (ok) {
                cpt::tc_fence_after();
                load_chunk<kEights, 0>(v[0], at);
                const float scale0 = fa[k] * f0[k], scale1 = fa[k] * f1[k];
                load_scales(k, kb + k + 2);
                static_for<kChunks>([&](auto chunk) {
                  constexpr uint32_t c = decltype(chunk)::value;
                  float(&x)[32] = v[c & 1];
                  cpt::tmem_load_wait(x);
                  if constexpr (c + 1 < kChunks) {
                    load_chunk<kEights, c + 1>(v[(c + 1) & 1], at);
                  } else {                // the buffer is read: the tensor core may have it back
                    cpt::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) cpt::mbar_arrive_cluster(pair_acc_empty + 8 * b);
                  }
                  add_chunk<kEights, c>(acc, x, turn, scale0, scale1);
                });
                ++it;
              }
            }
          }
        }
      }
      if (!ok) break;
      if (p.splits == 1) {
        if (any && row < p.m) {
#pragma unroll
          for (uint32_t c = 0; c < kEights; c += 2)
            if (col + 8 * c < p.n) store16(p, row, col + 8 * c, acc + 8 * c);
        }
      } else if (any) {
        // this pair's sums, [row][kBn + 4] floats over the stages (all loads are used up)
        float* part = reinterpret_cast<float*>(tiles) + (lanes + lane) * (kBn + 4) + share;
#pragma unroll
        for (uint32_t i = 0; i < kEights * 2; ++i)
          *reinterpret_cast<float4*>(part + 4 * i) =
              make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
      }
    }
    if (!ok && lane == 0) atomicOr(&g_matmul_gave_up, 1u);
  }
  __syncwarp();
  cpt::tc_fence_before();
  __syncthreads();
  cpt::cluster_sync();
  if (p.splits > 1 && gave_up == 0 && warp < kSumWarps) {
    // the pairs' sums, added in order: each pair takes a share of the tile's columns
    const uint32_t row0 = tile0 % p.tiles_m * 256 + half * 128, col0 = tile0 / p.tiles_m * kBn;
    const uint32_t rows = row0 < p.m ? min(128u, p.m - row0) : 0;
    const uint32_t c0 = kBn * split / p.splits, c1 = kBn * (split + 1) / p.splits;
    const uint32_t wide = c1 - c0, base = cpt::smem_addr(tiles);
    for (uint32_t i = threadIdx.x; i < rows * wide / 4; i += kSumWarps * 32) {
      const uint32_t r = i / (wide / 4), c = c0 + (i - r * (wide / 4)) * 4;
      if (col0 + c < p.n) {
        const uint32_t off = base + (r * (kBn + 4) + c) * 4;
        float4 v[4];
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q)
          if (q < p.splits) v[q] = cpt::load_cluster4(cpt::map_rank(off, 2 * q + half));
        float4 sum = v[0];
#pragma unroll
        for (uint32_t q = 1; q < 4; ++q) {
          if (q < p.splits) {
            sum.x += v[q].x;
            sum.y += v[q].y;
            sum.z += v[q].z;
            sum.w += v[q].w;
          }
        }
        const uint64_t at = static_cast<uint64_t>(row0 + r) * p.ldo + col0 + c;
        const float out[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
          if (col0 + c + e < p.n) store_from_f32(p.out, at + e, p.out_dtype, out[e]);
      }
    }
  }
  __syncwarp();
  cpt::cluster_sync();                 // no CTA leaves while another may read its shared memory
  if (warp == kSumWarps + 1) cpt::tmem_free_pair(tmem, p.tmem_columns);
}

// ----------------------------------------------- few rows of a, many bytes of w: tcgen05
//
// With at most 128 rows of a the operands change places: 128 rows of w are the tensor core's
// 128 x 32 operand, up to 64 rows of a its N (16, 32 or 64) columns, and the kernel is bound by
// the stream of w (a second tile of rows of a finds it in L2).  A unit is 128 columns of tensor memory, 128 / kN groups side by side, so
// the sums (a lane has a row of w) wait once a unit; two units alternate.  Two CTAs share an
// SM; `splits` CTAs of a cluster share a tile's groups and add their sums in order through
// distributed shared memory.

constexpr int kThinThreads = 256;      // four summing warps, TMA, MMA, scales, one idle
constexpr uint32_t kThinUnit = 128;    // columns of tensor memory
constexpr uint32_t kThinRows = 128;
constexpr uint32_t kThinMaxStages = 6;
constexpr uint32_t kThinSmem = 111616;  // dynamic shared memory of a CTA, two to an SM

struct ThinParams {
  const float* sa;
  const float* sw;
  void* out;
  uint64_t ldo;
  uint32_t m, n, groups, splits, stages, tiles_m;
  int out_dtype;
};

template <uint32_t kN>
__global__ void __launch_bounds__(kThinThreads, 2)
    matmul_thin_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_w, const ThinParams p) {
  constexpr uint32_t kPer = kThinUnit / kN;            // groups of a unit
  constexpr uint32_t kStage = kTileA + kN * 128;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[2 * kThinMaxStages + 6];
  __shared__ __align__(16) float scales[2][kThinUnit];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = p.splits == 1 ? 0 : cpt::cluster_rank();
  const uint32_t tile = blockIdx.x / p.splits;       // those of one part of w come together
  const uint32_t row0 = tile / p.tiles_m * 128;
  const uint32_t token0 = tile % p.tiles_m * kN, tokens = min(p.m - token0, kN);
  const uint32_t full = cpt::smem_addr(bars), empty = full + 8 * kThinMaxStages;
  const uint32_t acc_full = empty + 8 * kThinMaxStages, acc_empty = acc_full + 16;
  const uint32_t scale_full = acc_empty + 16;
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < p.stages; ++s) {
      cpt::mbar_init(full + 8 * s, 1);
      cpt::mbar_init(empty + 8 * s, 1);
    }
    for (uint32_t b = 0; b < 2; ++b) {
      cpt::mbar_init(acc_full + 8 * b, 1);
      cpt::mbar_init(acc_empty + 8 * b, 4);
      cpt::mbar_init(scale_full + 8 * b, 32);
    }
    cpt::mbar_init_fence();
    gave_up = 0;
  }
  if (warp == 5) cpt::tmem_alloc(cpt::smem_addr(&tmem_base), 2 * kThinUnit);
  cpt::tc_fence_before();
  __syncthreads();
  cpt::tc_fence_after();
  const uint32_t tmem = tmem_base;
  // whole units go to each CTA of the cluster
  const uint32_t units = (p.groups + kPer - 1) / kPer;
  const uint32_t u0 = units * rank / p.splits, u1 = units * (rank + 1) / p.splits;
  const uint32_t kb0 = u0 * kPer, kb1 = min(u1 * kPer, p.groups);
  float acc[kN];
#pragma unroll
  for (uint32_t i = 0; i < kN; ++i) acc[i] = 0.0f;
  bool ok = true;

  if (warp == 4) {
    // ------------------------------------------------------------------ loads
    if (cpt::elect_one()) {
      cpt::tma_prefetch_map(&map_a);
      cpt::tma_prefetch_map(&map_w);
    }
    __syncwarp();
    uint32_t s = 0, round = 0;
    for (uint32_t kb = kb0; kb < kb1; ++kb) {
      if (round > 0) {
        ok = cpt::mbar_wait(empty + 8 * s, (round - 1) & 1, &gave_up);
        if (!ok) break;
      }
      const uint32_t dst = cpt::smem_addr(tiles) + s * kStage;
      if (cpt::elect_one()) {
        cpt::mbar_expect(full + 8 * s, kStage);
        cpt::tma_load(dst, &map_w, kb * 128, row0, full + 8 * s);
        cpt::tma_load(dst + kTileA, &map_a, kb * 128, token0, full + 8 * s);
      }
      __syncwarp();
      if (++s == p.stages) {
        s = 0;
        ++round;
      }
    }
    if (!ok) {          // given up: the loads in flight land before the CTA leaves
      int unused = 0;
      for (uint32_t k = 0; k < p.stages; ++k) {
        const uint32_t r = k < s ? round : round - 1;
        if (k < s || round > 0) cpt::mbar_wait(full + 8 * k, r & 1, &unused);
      }
    }
  } else if (warp == 5) {
    // --------------------------------------------------------------- products
    constexpr uint32_t instr = cpt::e4m3_instr_desc(128, kN);
    uint32_t s = 0, round = 0, kb = kb0;
    for (uint32_t u = 0; kb < kb1; ++u) {
      const uint32_t b = u & 1;
      ok = u < 2 || cpt::mbar_wait(acc_empty + 8 * b, ((u >> 1) - 1) & 1, &gave_up);
      for (uint32_t g = 0; g < kPer && kb < kb1 && ok; ++g, ++kb) {
        ok = cpt::mbar_wait(full + 8 * s, round & 1, &gave_up);
        if (!ok) break;
        cpt::tc_fence_after();
        const uint32_t at = cpt::smem_addr(tiles) + s * kStage;
        const uint64_t dw = cpt::operand_desc(at), da = cpt::operand_desc(at + kTileA);
        if (cpt::elect_one()) {
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k)
            cpt::mma_one(tmem + b * kThinUnit + g * kN, dw + 2 * k, da + 2 * k, instr, k != 0);
          cpt::mma_commit(empty + 8 * s);
          if (g + 1 == kPer || kb + 1 == kb1) cpt::mma_commit(acc_full + 8 * b);
        }
        __syncwarp();
        if (++s == p.stages) {
          s = 0;
          ++round;
        }
      }
      if (!ok) break;
    }
  } else if (warp == 6) {
    // ----------------------------------------------------------------- scales
    const float* sw = p.sw + static_cast<uint64_t>(row0 / 128) * p.groups;
    uint32_t u = 0;
    for (uint32_t kb = kb0; kb < kb1; kb += kPer, ++u) {
      const uint32_t b = u & 1;
      float f[4];
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t e = lane + 32 * i, group = kb + e / kN, token = e % kN;
        f[i] = group < kb1 && token < tokens
                   ? __ldg(p.sa + static_cast<uint64_t>(token0 + token) * p.groups + group) *
                         __ldg(sw + group)
                   : 0.0f;
      }
      if (u >= 2) {
        ok = cpt::mbar_wait(acc_empty + 8 * b, ((u >> 1) - 1) & 1, &gave_up);
        if (!ok) break;
      }
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) scales[b][lane + 32 * i] = f[i];
      cpt::mbar_arrive(scale_full + 8 * b);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------------- sums
    const uint32_t tmem_warp = tmem + ((warp * 32) << 16);
    uint32_t u = 0;
    for (uint32_t kb = kb0; kb < kb1; kb += kPer, ++u) {
      const uint32_t b = u & 1;
      ok = cpt::mbar_wait(scale_full + 8 * b, (u >> 1) & 1, &gave_up) &&
           cpt::mbar_wait(acc_full + 8 * b, (u >> 1) & 1, &gave_up);
      if (!ok) break;
      cpt::tc_fence_after();
      const uint32_t columns = min(kPer, kb1 - kb) * kN;     // of the unit that are filled
#pragma unroll
      for (uint32_t c = 0; c < 4; ++c) {
        if (32 * c < columns) {          // (a last unit of 16-column groups may fill half of it)
          float x[32];
          cpt::tmem_load32<0>(x, tmem_warp + b * kThinUnit + 32 * c);
          float f[32];
#pragma unroll
          for (uint32_t i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(&f[4 * i]) =
                *reinterpret_cast<const float4*>(&scales[b][32 * c + 4 * i]);
          cpt::tmem_load_wait(x);
          const uint32_t here = min(32u, columns - 32 * c);
#pragma unroll
          for (uint32_t i = 0; i < 32; ++i)
            if (kN >= 32 || i < 16 || here == 32)
              acc[(32 * c + i) % kN] = fmaf(x[i], f[i], acc[(32 * c + i) % kN]);
        }
      }
      cpt::tc_fence_before();
      __syncwarp();
      if (lane == 0) cpt::mbar_arrive(acc_empty + 8 * b);
    }
  }
  if (!ok && lane == 0) atomicOr(&g_matmul_gave_up, 1u);
  __syncwarp();
  cpt::tc_fence_before();
  __syncthreads();
  const uint32_t row = row0 + threadIdx.x;       // (of the summing warps)
  if (p.splits == 1) {
    if (warp < 4 && row < p.n) {
#pragma unroll
      for (uint32_t i = 0; i < kN; ++i)
        if (i < tokens)
          store_from_f32(p.out, static_cast<uint64_t>(token0 + i) * p.ldo + row, p.out_dtype,
                         acc[i]);
    }
  } else {
    // sums as [row of a][row of w] over the stages (all loads are used up); each CTA of the cluster
    // then adds a share of the tokens
    float* part = reinterpret_cast<float*>(tiles);
    if (warp < 4) {
#pragma unroll
      for (uint32_t i = 0; i < kN; ++i) part[i * 128 + threadIdx.x] = acc[i];
    }
    __syncthreads();
    cpt::cluster_sync();
    const uint32_t i0 = tokens * 32 * rank / p.splits, i1 = tokens * 32 * (rank + 1) / p.splits;
    for (uint32_t i = i0 + threadIdx.x; i < i1; i += kThinThreads) {
      const uint32_t at = cpt::smem_addr(part + 4 * i);
      float4 v[8];
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q)
        if (q < p.splits) v[q] = cpt::load_cluster4(cpt::map_rank(at, q));
      float4 sum = v[0];
#pragma unroll
      for (uint32_t q = 1; q < 8; ++q) {
        if (q < p.splits) {
          sum.x += v[q].x;
          sum.y += v[q].y;
          sum.z += v[q].z;
          sum.w += v[q].w;
        }
      }
      const uint32_t token = token0 + i / 32, r = row0 + i % 32 * 4;
      const float out[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e)
        if (r + e < p.n)
          store_from_f32(p.out, static_cast<uint64_t>(token) * p.ldo + r + e, p.out_dtype, out[e]);
    }
    __syncwarp();
    cpt::cluster_sync();             // no CTA leaves while another may read its shared memory
  }
  if (warp == 5) cpt::tmem_free(tmem, 2 * kThinUnit);
}

// What a launch needs to know of the device, found once.
using TcKernel = void (*)(CUtensorMap, CUtensorMap, TcParams);
constexpr TcKernel kTcKernels[8] = {      // tiles of 32, 64, .. 256 columns
    &matmul_tc_kernel<2>,  &matmul_tc_kernel<4>,  &matmul_tc_kernel<6>,  &matmul_tc_kernel<8>,
    &matmul_tc_kernel<10>, &matmul_tc_kernel<12>, &matmul_tc_kernel<14>, &matmul_tc_kernel<16>};

struct TcDevice {
  std::atomic<int> state{0};           // 0: not asked, 1: usable, 2: not
  int clusters[3] = {0, 0, 0};         // clusters of 2, 4, 8 CTAs that run at once
};
TcDevice g_devices[64];

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::atomic<EncodeTiled> g_encode{nullptr};

void launch_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, uint32_t cluster,
                   uint32_t ctas, size_t smem, cudaStream_t s) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3(ctas);
  cfg->blockDim = dim3(kTcThreads);
  cfg->dynamicSmemBytes = smem;
  cfg->stream = s;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

const TcDevice* tc_device(cudaError_t* err) {
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err != cudaSuccess || dev >= 64) return nullptr;
  TcDevice& d = g_devices[dev];
  if (d.state.load(std::memory_order_acquire) == 1) return &d;
  // several threads may get here at once: each finds the same values
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  *err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                          &found);
  if (*err != cudaSuccess) return nullptr;
  if (fn == nullptr || found != cudaDriverEntryPointSuccess) {
    *err = cudaErrorNotSupported;
    return nullptr;
  }
  g_encode.store(reinterpret_cast<EncodeTiled>(fn));
  for (TcKernel kernel : kTcKernels) {
    const void* k = reinterpret_cast<const void*>(kernel);
    cudaFuncAttributes attrs{};
    *err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSmemMost));
    if (*err == cudaSuccess) *err = cudaFuncGetAttributes(&attrs, k);
    if (*err == cudaSuccess && attrs.numRegs != kLaunchRegs) *err = cudaErrorInvalidConfiguration;
    if (*err != cudaSuccess) return nullptr;
  }
  for (const void* k : {reinterpret_cast<const void*>(&matmul_thin_kernel<16>),
                        reinterpret_cast<const void*>(&matmul_thin_kernel<32>),
                        reinterpret_cast<const void*>(&matmul_thin_kernel<64>)}) {
    *err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kThinSmem));
    if (*err != cudaSuccess) return nullptr;
  }
  for (int i = 0; i < 3 && *err == cudaSuccess; ++i) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    launch_config(&cfg, attr, 2u << i, (2u << i) * 64, kSmemMost, nullptr);
    int most = 0;
    *err = cudaOccupancyMaxActiveClusters(&most, reinterpret_cast<const void*>(kTcKernels[7]),
                                          &cfg);
    d.clusters[i] = most;
  }
  if (*err != cudaSuccess) return nullptr;
  if (d.clusters[0] < 1) {
    *err = cudaErrorInvalidConfiguration;
    return nullptr;
  }
  d.state.store(1, std::memory_order_release);
  return &d;
}

bool encode_map(CUtensorMap* map, const uint8_t* base, uint64_t k, uint64_t rows, uint64_t ld,
                uint32_t box_rows) {
  const cuuint64_t dims[2] = {k, rows};
  const cuuint64_t strides[1] = {rows == 1 ? (k + 15) / 16 * 16 : ld};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t elem[2] = {1, 1};
  return g_encode.load()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims,
                         strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Columns of a tile and pairs that share one, by the time that the busiest pair needs.  In
// nanoseconds, measured on tiles of one turn (k = 4096 and 24576, 64 to 256 columns): a group
// takes 250 + 0.85 a column, a tile's outputs 14 a column, and sharing a tile 4000.
void choose_tile(const TcDevice& d, uint32_t m, uint32_t n, uint32_t groups, uint32_t* bn,
                 uint32_t* splits) {
  const uint64_t tiles_m = (static_cast<uint64_t>(m) + 255) / 256;
  double best = 1e300;
  for (uint32_t i = 0; i < 3; ++i) {
    const uint32_t s = 1u << i;
    if (s > 1 && groups < 4 * s) break;
    for (uint32_t b = 256; b >= 32; b -= 32) {
      const uint64_t tiles = tiles_m * ((static_cast<uint64_t>(n) + b - 1) / b);
      const uint64_t at_once = static_cast<uint64_t>(d.clusters[i]);
      if (at_once == 0 || (s > 1 && tiles > at_once)) continue;
      const double turns = static_cast<double>((tiles + at_once - 1) / at_once);
      const double cost =
          turns * ((groups + s - 1) / s * (250.0 + 0.85 * b) + 14.0 * b) + (s > 1 ? 4000.0 : 0.0);
      if (cost < best) {
        best = cost;
        *bn = b;
        *splits = s;
      }
    }
  }
}

cp_status launch_tc(const MatmulParams& q, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const TcDevice* d = tc_device(&e);
  if (d == nullptr) return cpx::cuda_fail(e, "fp8 matmul device query");
  uint32_t bn = 32, splits = 1;
  choose_tile(*d, q.m, q.n, q.groups, &bn, &splits);
  TcParams p{};
  p.sa = q.sa;
  p.sw = q.sw;
  p.out = q.out;
  p.ldo = q.ldo;
  p.m = q.m;
  p.n = q.n;
  p.groups = q.groups;
  p.out_dtype = q.out_dtype;
  p.splits = splits;
  p.tiles_m = (q.m + 255) / 256;
  p.a_rows = q.m >= 128 ? 128 : (q.m + 7) / 8 * 8;
  const uint64_t tiles = static_cast<uint64_t>(p.tiles_m) * ((q.n + bn - 1) / bn);
  if (tiles >= (1ull << 31)) {
    cpx::set_error("m and n make more than 2^31 tiles");
    return CP_ERR_INVALID_ARG;
  }
  p.tiles = static_cast<uint32_t>(tiles);
  const uint32_t stage = kTileA + bn * 64;
  p.stages = (kSmemMost - 1024) / stage;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.tmem_columns = 64;
  while (p.tmem_columns < 2 * bn) p.tmem_columns *= 2;
  const uint64_t elt = dtype_size(q.out_dtype);
  p.out_align = cpx::aligned(q.out, 32) && q.ldo * elt % 32 == 0   ? 32
                : cpx::aligned(q.out, 16) && q.ldo * elt % 16 == 0 ? 16
                                                                   : 0;
  CUtensorMap map_a, map_w;
  if (!encode_map(&map_a, q.a, q.k, q.m, q.lda, p.a_rows) ||
      !encode_map(&map_w, q.w, q.k, q.n, q.ldw, bn / 2)) {
    cpx::set_error("tensor map refused");
    return CP_ERR_CUDA;
  }
  const uint32_t at_once = static_cast<uint32_t>(d->clusters[splits == 1 ? 0 : splits == 2 ? 1 : 2]);
  const uint32_t clusters = splits > 1 || p.tiles < at_once ? p.tiles : at_once;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  launch_config(&cfg, attr, 2 * splits, 2 * splits * clusters, kSmemMost, s);
  e = cudaLaunchKernelEx(&cfg, kTcKernels[bn / 32 - 1], map_a, map_w, p);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul launch");
  return CP_OK;
}

cp_status launch_thin(const MatmulParams& q, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (tc_device(&e) == nullptr) return cpx::cuda_fail(e, "fp8 matmul device query");
  const uint32_t kn = q.m <= 16 ? 16 : q.m <= 32 ? 32 : 64;
  const uint32_t units = (q.groups + kThinUnit / kn - 1) / (kThinUnit / kn);
  const uint32_t tiles_m = (q.m + kn - 1) / kn;
  const uint32_t tiles = (q.n + 127) / 128 * tiles_m;
  // CTAs share a tile until there are enough to keep every SM's loads in flight.
  uint32_t splits = 1;
  while (splits < 8 && static_cast<uint64_t>(tiles) * splits * 2 <= 304 && units >= 2 * splits)
    splits *= 2;
  ThinParams p{q.sa, q.sw, q.out, q.ldo, q.m, q.n, q.groups, splits, 0, tiles_m, q.out_dtype};
  const uint32_t stage = kTileA + kn * 128;
  p.stages = (kThinSmem - 1024) / stage;
  if (p.stages > kThinMaxStages) p.stages = kThinMaxStages;
  CUtensorMap map_a, map_w;
  if (!encode_map(&map_a, q.a, q.k, q.m, q.lda, kn) ||
      !encode_map(&map_w, q.w, q.k, q.n, q.ldw, 128)) {
    cpx::set_error("tensor map refused");
    return CP_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  launch_config(&cfg, attr, splits, splits * tiles, kThinSmem, s);
  cfg.blockDim = dim3(kThinThreads);
  auto* fn = kn == 16 ? &matmul_thin_kernel<16> : kn == 32 ? &matmul_thin_kernel<32>
                                                            : &matmul_thin_kernel<64>;
  e = cudaLaunchKernelEx(&cfg, fn, map_a, map_w, p);
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul launch");
  return CP_OK;
}

}  // namespace

extern "C" cp_status cp_matmul_fp8_status(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul");
  uint32_t word = 0;
  e = cudaMemcpyFromSymbol(&word, g_matmul_gave_up, sizeof(word));
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul status");
  if (word == 0) return CP_OK;
  const uint32_t zero = 0;
  e = cudaMemcpyToSymbol(g_matmul_gave_up, &zero, sizeof(zero));
  if (e != cudaSuccess) return cpx::cuda_fail(e, "fp8 matmul status");
  cpx::set_error("a wait inside cp_matmul_fp8 ran out of time; its output is not valid");
  return CP_ERR_CUDA;
}

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
    return m > kThinRows ? launch_tc(p, s)
           : m <= kFewRows && n * k <= kFewBytes ? launch_few(p, s) : launch_thin(p, s);
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

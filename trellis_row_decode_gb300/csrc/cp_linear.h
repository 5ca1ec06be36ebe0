// cp_linear.h -- host side of cp_linear and cp_linear_grad shared by their translation units.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "cp.h"
#include "cp_epilogue.cuh"

namespace cplin {

// A 16-bit operand on 16-byte boundaries: `rows` of the product's rows (or columns) by k.
struct Operand {
  const void* p;
  uint64_t ld;             // elements between the array's rows
  bool across;             // stored [k][rows] instead of [rows][k]
};

// out[i][j] = epilogue(sum over k of a[i][k] b[j][k]), e.m rows by e.n columns.
struct Product {
  Operand a, b;
  uint32_t k;
  int dtype;               // CP_F16 or CP_BF16
  cpe::Epilogue e;
};

// Sums over rows: out[j] (+)= sum of parts[i][j], which another kernel left, or of rows of 16 bits
// themselves (few of them, on 16-byte boundaries).
struct ColumnSums {
  const float* parts;      // [count][pitch]
  const void* rows;        // [count][pitch] of rows_dtype, or null
  void* out;               // null: none
  uint64_t pitch;
  uint32_t count, n;
  int dtype, accumulate, rows_dtype;
};

// Products of one launch on CTA pairs (cp_linear_tc.cu), two at most.
constexpr int kMostProducts = 2, kWidths = 8;

// How a product may be cut: columns of a tile, units that share a tile's k, and what that costs.
struct Tiling {
  uint32_t bn, splits;
  uint64_t units;
  double each, extra;      // ns of a unit, of sharing k
};
// The ways of up to two products, m x n x k each (none of them 0), by width of the tiles.
struct Tilings {
  uint32_t m[kMostProducts], n[kMostProducts];
  Tiling way[kMostProducts][kWidths];
};
Tilings tilings(const uint32_t* m, const uint32_t* n, const uint32_t* k, int count);
// Those of products `first` on that are launched together.
void choose(const Tilings& t, int first, int count, Tiling* out);
// The first product's again where it has dropout: another width, never another split.
void choose_dropped(const Tilings& t, Tiling* chosen);
// Floats for the sums of products whose k is split, so chosen.
uint64_t part_floats(const Tilings& t, int first, int count);

// `chosen` is for the products that have outputs and sums, in their order; `part` holds part_floats.
cp_status launch_products(const Product* q, int count, const Tiling* chosen, const ColumnSums& sums,
                          float* part, cudaStream_t s);

// k of a unit above which sums are read in segments, by the type they are rounded to.  The tensor core
// cuts its running sum and each product that it adds: a sum of positive products loses 6.4e-9 k of itself
// (fp16; bf16 5.9e-9), all to one side.  In 16 bits that may come to an eighth of the rounding's half
// step (2^-11, 2^-8).  Segments cost 2 to 4 % (4096 x 4096 x 24576 fp16 468 us, 478 in segments).
constexpr uint32_t long_sum(int dtype) {
  return dtype == CP_F32 ? 512 : dtype == CP_F16 ? 8192 : 65536;
}

// Up to kThinRows rows of a: tiles of 128 rows of b, neither operand stored across.
constexpr uint32_t kThinRows = 128;
cp_status launch_thin(const Product& q, cudaStream_t s);

}  // namespace cplin

// cp_matmul_fp8.h -- host side of cp_matmul_fp8 shared by its translation units: the checked
// call, and the kernels of tensor memory behind one function each.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "cp.h"

namespace cpm {

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

// Operands whose rows lie on 16-byte boundaries (cp_matmul_tc.cu).
// More than 128 rows of a (kThinRows): tiles of 256 rows of a and 32 to 256 rows of w, a pair of
// SMs each.
cp_status launch_pairs(const MatmulParams& p, cudaStream_t s);
// Up to 128 rows of a: tiles of 128 rows of w and up to 64 rows of a.
cp_status launch_thin(const MatmulParams& p, cudaStream_t s);

}  // namespace cpm

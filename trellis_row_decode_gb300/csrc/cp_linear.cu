// cp_linear.cu -- the projection in 16 bits with its epilogue, and its gradient (include/cp.h,
// cp_linear, cp_linear_grad): the checked calls, and the gradient's pass over dy.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "cp.h"
#include "cp_align.cuh"
#include "cp_epilogue.cuh"
#include "cp_internal.h"
#include "cp_layer.cuh"
#include "cp_linear.h"
#include "cp_matmul_fp8.h"

namespace {

using namespace cpl;
using cpe::DropKey;
using cpe::DropParams;
using cplin::ColumnSums;
using cplin::Operand;
using cplin::Product;
using cplin::Tiling;
using cplin::Tilings;

// ------------------------------------------------------------------ dz and its column sums
//
// dz = D(dy) act'(pre), rounded to the products' type, and the sums of dz (before that rounding)
// over blocks of rows.  A CTA has 256 columns (an octet a lane) and one of `count` shares of the
// rows, eight at a time; its sums go to `parts`, which the products' kernel adds in order.  Column
// sums alone are bound by memory (4096 x 4096: 10 us), slopes and the generator by their instructions
// (270 an octet for silu and dropout, half of them the generator's: 28 us, silu alone 20, where dy, pre
// and dz would take 15).

constexpr int kGradThreads = 256;
constexpr uint32_t kGradColumns = 256;
constexpr uint32_t kMostParts = 64;
static_assert(kGradThreads == cpm::kAlignThreads, "CTAs of the copies are those of dz");
// Rows whose loads a thread has in flight, CTAs of an SM (by registers: slopes and the generator
// take more).
constexpr uint32_t grad_ahead(bool shape) { return shape ? 2 : 4; }
constexpr uint32_t grad_ctas(bool shape) { return shape ? 3 : 4; }

struct GradParams {
  const void* dy;
  const void* pre;
  void* dz;                // null: column sums alone
  float* parts;            // [count][pitch], or null
  uint64_t ldy, ldp, pitch;
  uint32_t m, n, count;
  int act;
  DropParams drop;
  uint32_t copy_rows;      // rows of CTAs (blockIdx.y) from `count` on that copy operands of the
  cpm::AlignParams copy;   // products to 16-byte boundaries meanwhile
};

template <uint32_t kCount>
struct Count {
  static constexpr uint32_t value = kCount;
};

// kShape: there is an activation or dropout.
template <typename T, typename D, bool VEC, bool kShape>
__global__ void __launch_bounds__(kGradThreads, grad_ctas(kShape))
    dz_kernel(const __grid_constant__ GradParams p) {
  constexpr uint32_t kAhead = grad_ahead(kShape);
  __shared__ float sums[8][kGradColumns];
  wait_for_previous();
  let_next_start();
  if (blockIdx.y >= p.count) {
    cpm::align_rows_of(p.copy, (blockIdx.y - p.count) * gridDim.x + blockIdx.x,
                       p.copy_rows * gridDim.x);
    return;
  }
  const uint32_t lane = threadIdx.x & 31, line = threadIdx.x >> 5;
  const uint32_t o = blockIdx.x * (kGradColumns / 8) + lane;
  const uint32_t r0 = static_cast<uint32_t>(static_cast<uint64_t>(p.m) * blockIdx.y / p.count);
  const uint32_t r1 =
      static_cast<uint32_t>(static_cast<uint64_t>(p.m) * (blockIdx.y + 1) / p.count);
  const DropKey key = cpe::drop_key(p.drop);
  float acc[8] = {};
  // kRows rows, eight apart, all of them there: their chains of arithmetic side by side
  auto rows = [&](uint32_t r, auto count) {
    constexpr uint32_t kRows = decltype(count)::value;
    Packed<D> dy[kRows];
    Packed<T> pre[kRows];
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) {
      dy[i] = load_row_octet<D, VEC>(static_cast<const D*>(p.dy) + (r + 8 * i) * p.ldy, o, p.n);
      if (kShape && p.act != CP_ACT_NONE)
        pre[i] = load_row_octet<T, VEC>(static_cast<const T*>(p.pre) + (r + 8 * i) * p.ldp, o, p.n);
    }
    float v[8 * kRows];
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) {
      float u[8];
      unpack(dy[i], u);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[8 * i + e] = u[e];
    }
    if constexpr (kShape) {
      if (p.act != CP_ACT_NONE) {
        float z[8 * kRows];
#pragma unroll
        for (uint32_t i = 0; i < kRows; ++i) {
          float u[8];
          unpack(pre[i], u);
#pragma unroll
          for (int e = 0; e < 8; ++e) z[8 * i + e] = u[e];
        }
        cpe::with_act(p.act, [&](auto tag) { cpe::slope_all<decltype(tag)::value>(z, v); });
      }
      if (p.drop.mode != 0) cpe::drop_block<2, kRows>(p.drop, key, 2 * o, r, 8, v);
    }
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) {
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[e] = v[8 * i + e];
        acc[e] += u[e];
      }
      if (p.dz != nullptr)           // (rows on 16-byte boundaries; what lies behind n is not read)
        store_octet(static_cast<T*>(p.dz) + (r + 8 * i) * p.pitch + 8ull * o, pack<T>(u));
    }
  };
  if (8ull * o < p.n) {
    uint32_t r = r0 + line;
    for (; r + 8 * (kAhead - 1) < r1; r += 8 * kAhead) rows(r, Count<kAhead>{});
    for (; r < r1; r += 8) rows(r, Count<1>{});
  }
  if (p.parts == nullptr) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[line][8 * lane + e] = acc[e];
  __syncthreads();
  const uint32_t col = blockIdx.x * kGradColumns + threadIdx.x;
  if (col < p.n) {
    float s = sums[0][threadIdx.x];
#pragma unroll
    for (uint32_t i = 1; i < 8; ++i) s += sums[i][threadIdx.x];
    p.parts[blockIdx.y * p.pitch + col] = s;
  }
}

// Shares of the rows: CTAs that all run at once, and few enough parts for the products' kernel to
// add.
uint32_t grad_parts(uint64_t m, uint64_t n, bool shape) {
  const uint64_t wide = (n + kGradColumns - 1) / kGradColumns;
  const uint64_t want = std::max<uint64_t>(1, 152 * grad_ctas(shape) / std::max<uint64_t>(wide, 1));
  return static_cast<uint32_t>(std::min({want, (m + 7) / 8, static_cast<uint64_t>(kMostParts)}));
}

template <typename T, typename D>
cudaError_t launch_dz(const GradParams& p, bool vec, cudaStream_t s) {
  const Launch l{dim3((p.n + kGradColumns - 1) / kGradColumns, p.count + p.copy_rows),
                 kGradThreads, 0, s};
  if (p.act != CP_ACT_NONE || p.drop.mode != 0)
    return vec ? launch(l, &dz_kernel<T, D, true, true>, p)
               : launch(l, &dz_kernel<T, D, false, true>, p);
  return vec ? launch(l, &dz_kernel<T, D, true, false>, p)
             : launch(l, &dz_kernel<T, D, false, false>, p);
}

// ---------------------------------------------------------------------------- host

constexpr uint64_t kMostRows = 1ull << 31, kMostK = 1ull << 30;
// Rows of dy, where it is dz itself, whose sums the products' kernel makes on the way: no launch and no
// workspace for them.  With up to 1,024 columns the two ways cross between 384 and 640 rows on the
// device (bf16, kernels here / in two launches: n x k of 384 x 256 with 256 rows 5.5 / 6.4 us, 512 7.5 / 6.8,
// 1,024 11.7 / 8.5; 1024 x 1024 7.0 / 8.5, 8.8 / 8.9, 13.8 / 10.5), with 4,096 columns and so more
// warps never up to 2,048 rows (512 rows 18.5 / 20.7); and a call is 2 to 7 us shorter on the host up to
// 1,024.  No further than a segment either: beside a dw that is read in segments the warps in
// question have few registers.
constexpr uint64_t kDirectRows = 512;
static_assert(kDirectRows <= cplin::long_sum(CP_F32), "no segments beside direct sums");

uint64_t up(uint64_t x, uint64_t to) { return (x + to - 1) / to * to; }
// Elements of a 16-bit row that is made here: whole lines of memory where it is long, so that 128 bytes
// of a stage's row lie in one line instead of two (333 x 1024 x 2321 from rows of 2328 13.7 us, of 2368
// 10.2).
uint64_t row_pitch(uint64_t k) { return up(k, k < 512 ? 8 : 64); }

// Rows that a tensor map takes (and a row stride of their own: not one row for all).
bool rows_ok(const void* p, uint64_t stride, uint64_t rows) {
  return cpx::aligned(p, 16) && (rows == 1 || (stride % 8 == 0 && stride != 0));
}

cp_status refuse(const char* what) {
  cpx::set_error(what);
  return CP_ERR_INVALID_ARG;
}

bool row_ok(uint64_t stride, uint64_t d) { return stride >= d || stride == 0; }

// Whether an operand of a product, read tile by tile where it lies, shares a byte with an output.
bool reads(const Operand& op, uint64_t rows, uint64_t k, const cpx::RowBytes& out) {
  return cpx::rows_meet({op.p, 2 * op.ld, 2 * k, rows}, out);
}

// Operands that lie on other boundaries, to be copied behind each other to `to`; false: none.
bool to_align(Operand* (&op)[2], const uint64_t (&rows)[2], uint64_t k, uint8_t*& to,
              cpm::AlignOperand (&of)[2]) {
  const uint64_t pitch = 2 * row_pitch(k);
  bool any = false;
  for (int i = 0; i < 2; ++i) {
    of[i] = cpm::AlignOperand{};
    if (op[i] == nullptr || rows_ok(op[i]->p, op[i]->ld, rows[i])) continue;
    of[i] = cpm::AlignOperand{static_cast<const uint8_t*>(op[i]->p), to, 2 * op[i]->ld, rows[i]};
    op[i]->p = to;
    op[i]->ld = pitch / 2;
    to += rows[i] * pitch;
    any = true;
  }
  return any;
}

// Bytes for the sums of products whose k is split; they begin on a 32-byte boundary, the workspace
// on a 16-byte one.
uint64_t part_bytes(const Tilings& t, int first, int count) {
  const uint64_t floats = cplin::part_floats(t, first, count);
  return floats == 0 ? 0 : 4 * floats + 16;
}
Tilings linear_tilings(uint64_t m, uint64_t n, uint64_t k) {
  const uint32_t ms = static_cast<uint32_t>(m), ns = static_cast<uint32_t>(n),
                 ks = static_cast<uint32_t>(k);
  return cplin::tilings(&ms, &ns, &ks, 1);
}
// Bytes for the copies of operands that lie on other boundaries.
uint64_t copy_bytes(const void* x, uint64_t x_stride, const void* w, uint64_t w_stride, uint64_t m,
                    uint64_t n, uint64_t k) {
  return ((rows_ok(x, x_stride, m) ? 0 : m) + (rows_ok(w, w_stride, n) ? 0 : n)) * 2 * row_pitch(k);
}
float* part_at(uint8_t* p) {
  return reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(p) + 31) & ~static_cast<uintptr_t>(31));
}

}  // namespace

extern "C" uint64_t cp_linear_workspace_bytes(const void* x, uint64_t x_stride, const void* w,
                                              uint64_t w_stride, uint64_t m, uint64_t n,
                                              uint64_t k) {
  if (m >= kMostRows || n >= kMostRows || k >= kMostK || m == 0 || n == 0 || k == 0) return 0;
  return copy_bytes(x, x_stride, w, w_stride, m, n, k) +
         (m > cplin::kThinRows ? part_bytes(linear_tilings(m, n, k), 0, 1) : 0);
}

extern "C" cp_status cp_linear(const void* x, uint64_t x_stride, const void* w, uint64_t w_stride,
                               int dtype, uint64_t m, uint64_t n, uint64_t k, const void* bias,
                               int bias_dtype, int activation, double p, uint64_t seed,
                               uint64_t offset, const uint64_t* rng, const void* residual,
                               uint64_t residual_stride, void* out, int out_dtype,
                               uint64_t out_stride, void* pre, uint64_t pre_stride,
                               void* workspace, uint64_t workspace_bytes, void* stream) {
  if ((dtype != CP_F16 && dtype != CP_BF16) || !dtype_ok(out_dtype) ||
      (bias != nullptr && !dtype_ok(bias_dtype)) || m >= kMostRows || n >= kMostRows ||
      k >= kMostK || !row_ok(x_stride, k) || !row_ok(w_stride, k) || out_stride < n ||
      (residual != nullptr && !row_ok(residual_stride, n)) ||
      (pre != nullptr && pre_stride < n))
    return refuse("bad dtype, m, n, k or row stride");
  Product q{};
  if (!cpe::act_ok(activation) || !cpe::drop_params(&q.e.drop, p, seed, offset, rng) ||
      !cpx::aligned(rng, 8))
    return refuse("bad activation, p or rng");
  if (m == 0 || n == 0) return CP_OK;
  const uint64_t elt = dtype_size(out_dtype);
  if (out == nullptr || !cpx::aligned(out, elt) || !cpx::aligned(residual, elt) ||
      !cpx::aligned(pre, 2) || (bias != nullptr && !cpx::aligned(bias, dtype_size(bias_dtype))) ||
      (k != 0 && (x == nullptr || w == nullptr || !cpx::aligned(x, 2) || !cpx::aligned(w, 2))))
    return refuse("null or misaligned x, w, bias, residual, out or pre");
  const cpx::RowBytes o{out, out_stride * elt, n * elt, m}, kept{pre, 2 * pre_stride, 2 * n, m},
      stream_rows{residual, residual_stride * elt, n * elt, m};
  if (cpx::rows_clash(o, stream_rows) || cpx::rows_meet(kept, o) || cpx::rows_meet(kept, stream_rows))
    return refuse("out lies on part of the residual, or pre on out or the residual");
  const bool thin = m <= cplin::kThinRows;
  Tilings ways{};
  Tiling chosen{};
  uint64_t need = 0;
  if (k != 0) {
    need = copy_bytes(x, x_stride, w, w_stride, m, n, k);
    if (!thin) {
      ways = linear_tilings(m, n, k);
      cplin::choose(ways, 0, 1, &chosen);
      if (q.e.drop.mode == 1) cplin::choose_dropped(ways, &chosen);
      need += part_bytes(ways, 0, 1);
    }
  }
  if (need != 0 &&
      (workspace == nullptr || !cpx::aligned(workspace, 16) || workspace_bytes < need))
    return refuse("workspace must be 16-byte aligned and hold cp_linear_workspace_bytes bytes");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  q.a = Operand{x, x_stride, false};
  q.b = Operand{w, w_stride, false};
  q.k = static_cast<uint32_t>(k);
  q.dtype = dtype;
  q.e.bias = bias;
  q.e.residual = residual;
  q.e.out = out;
  q.e.pre = pre;
  q.e.ldr = residual_stride;
  q.e.ldo = out_stride;
  q.e.ldp = pre_stride;
  q.e.m = static_cast<uint32_t>(m);
  q.e.n = static_cast<uint32_t>(n);
  q.e.bias_dtype = bias_dtype;
  q.e.out_dtype = out_dtype;
  q.e.pre_dtype = dtype;
  q.e.act = activation;
  q.e.aligned = cpx::sectors_ok(out, out_stride, elt) &&
                cpx::sectors_ok(residual, residual_stride, elt) &&
                cpx::sectors_ok(pre, pre_stride, 2);
  if (k == 0) return cplin::launch_products(&q, 1, &chosen, ColumnSums{}, nullptr, s);
  uint8_t* at = static_cast<uint8_t*>(workspace);
  Operand* op[2] = {&q.a, &q.b};
  cpm::AlignOperand of[2];
  const bool copies = to_align(op, {m, n}, k, at, of);
  if (reads(q.a, m, k, o) || reads(q.b, n, k, o) || reads(q.a, m, k, kept) || reads(q.b, n, k, kept))
    return refuse("out or pre lies on x or w, which are read while it is written");
  if (copies) {
    const cudaError_t e = cpm::align_rows(of, static_cast<uint32_t>(2 * k), 2 * row_pitch(k), s);
    if (e != cudaSuccess) return cpx::cuda_fail(e, "linear launch");
  }
  if (thin) return cplin::launch_thin(q, s);
  return cplin::launch_products(&q, 1, &chosen, ColumnSums{}, part_at(at), s);
}

namespace {

// The ways of a gradient's products, dx and dw.
Tilings grad_tilings(uint64_t m, uint64_t n, uint64_t k) {
  if (m == 0 || n == 0 || k == 0) return Tilings{};
  const uint32_t ms[2] = {static_cast<uint32_t>(m), static_cast<uint32_t>(n)};
  const uint32_t ns[2] = {static_cast<uint32_t>(k), static_cast<uint32_t>(k)};
  const uint32_t ks[2] = {static_cast<uint32_t>(n), static_cast<uint32_t>(m)};
  return cplin::tilings(ms, ns, ks, 2);
}
// Bytes for their sums, of both together or of either where the other is not wanted.
uint64_t grad_part_bytes(const Tilings& t) {
  if (t.m[0] == 0) return 0;
  return std::max({part_bytes(t, 0, 2), part_bytes(t, 0, 1), part_bytes(t, 1, 1)});
}
uint64_t dz_bytes(uint64_t m, uint64_t n) { return 2 * m * row_pitch(n); }
uint64_t db_bytes(uint64_t m, uint64_t n) { return 4ull * grad_parts(m, n, false) * row_pitch(n); }

// Whether the products' kernel makes the column sums from dy's rows.  (Not beside a dx whose k is so
// long that its sums are read in segments: the warps in question have few registers there.)
bool direct_sums(uint64_t m, uint64_t n, int dtype) {
  return m <= kDirectRows && n <= cplin::long_sum(dtype);
}

// Whether dz is dy itself.
bool dy_as_is(const void* dy, int dy_dtype, uint64_t dy_stride, int dtype, uint64_t m,
              int activation, double p) {
  return activation == CP_ACT_NONE && p == 0.0 && dy_dtype == dtype && rows_ok(dy, dy_stride, m);
}

// Bytes of a call with m and n above 0.
uint64_t grad_bytes(const Tilings& t, bool as_is, int dtype, const void* x, uint64_t x_stride,
                    const void* w, uint64_t w_stride, uint64_t m, uint64_t n, uint64_t k) {
  return (as_is ? 0 : dz_bytes(m, n)) + (as_is && direct_sums(m, n, dtype) ? 0 : db_bytes(m, n)) +
         copy_bytes(x, x_stride, w, w_stride, m, n, k) + grad_part_bytes(t);
}

}  // namespace

extern "C" uint64_t cp_linear_grad_workspace_bytes(uint64_t m, uint64_t n, uint64_t k) {
  if (m >= kMostK || n >= kMostK || k >= kMostK) return 0;
  // dz, copies of x and w, the parts of db, the sums of products whose k is split
  return std::max<uint64_t>(16, dz_bytes(m, n) + 2 * (m + n) * row_pitch(k) + db_bytes(m, n) +
                                    grad_part_bytes(grad_tilings(m, n, k)));
}

extern "C" uint64_t cp_linear_grad_call_bytes(const void* dy, int dy_dtype, uint64_t dy_stride,
                                              const void* x, uint64_t x_stride, const void* w,
                                              uint64_t w_stride, int dtype, uint64_t m, uint64_t n,
                                              uint64_t k, int activation, double p) {
  if (m >= kMostK || n >= kMostK || k >= kMostK || m == 0 || n == 0) return 0;
  return grad_bytes(grad_tilings(m, n, k),
                    dy_as_is(dy, dy_dtype, dy_stride, dtype, m, activation, p), dtype, x, x_stride,
                    w, w_stride, m, n, k);
}

extern "C" cp_status cp_linear_grad(const void* dy, int dy_dtype, uint64_t dy_stride,
                                    const void* x, uint64_t x_stride, const void* w,
                                    uint64_t w_stride, int dtype, const void* pre,
                                    uint64_t pre_stride, uint64_t m, uint64_t n, uint64_t k,
                                    int activation, double p, uint64_t seed, uint64_t offset,
                                    const uint64_t* rng, int accumulate, void* dx,
                                    uint64_t dx_stride, void* dw, int dw_dtype,
                                    uint64_t dw_stride, void* db, int db_dtype, void* workspace,
                                    uint64_t workspace_bytes, void* stream) {
  if ((dtype != CP_F16 && dtype != CP_BF16) || (dy_dtype != dtype && dy_dtype != CP_F32) ||
      (dw != nullptr && !dtype_ok(dw_dtype)) || (db != nullptr && !dtype_ok(db_dtype)) ||
      m >= kMostK || n >= kMostK || k >= kMostK || !row_ok(dy_stride, n) || !row_ok(x_stride, k) ||
      !row_ok(w_stride, k) || (pre != nullptr && !row_ok(pre_stride, n)) ||
      (dx != nullptr && dx_stride < k) || (dw != nullptr && dw_stride < k) ||
      (accumulate != 0 && accumulate != 1))
    return refuse("bad dtype, m, n, k, row stride or accumulate");
  GradParams g{};
  if (!cpe::act_ok(activation) || (activation != CP_ACT_NONE) != (pre != nullptr) ||
      !cpe::drop_params(&g.drop, p, seed, offset, rng) || !cpx::aligned(rng, 8))
    return refuse("bad activation, pre, p or rng");
  const bool want_dx = dx != nullptr && m != 0 && k != 0, want_dw = dw != nullptr && n != 0 && k != 0;
  if (!cpx::aligned(dx, 2) || (dw != nullptr && !cpx::aligned(dw, dtype_size(dw_dtype))) ||
      (db != nullptr && !cpx::aligned(db, dtype_size(db_dtype))) ||
      (m != 0 && n != 0 && (dy == nullptr || !cpx::aligned(dy, dtype_size(dy_dtype)))) ||
      !cpx::aligned(pre, 2) ||
      (want_dx && n != 0 && (w == nullptr || !cpx::aligned(w, 2))) ||
      (want_dw && m != 0 && (x == nullptr || !cpx::aligned(x, 2))))
    return refuse("null or misaligned dy, x, w, pre, dx, dw or db");
  if (!want_dx && !want_dw && (db == nullptr || n == 0)) return CP_OK;
  const bool as_is = dy_as_is(dy, dy_dtype, dy_stride, dtype, m, activation, p);
  const Tilings ways = grad_tilings(m, n, k);
  const uint64_t need =
      m == 0 || n == 0 ? 0 : grad_bytes(ways, as_is, dtype, x, x_stride, w, w_stride, m, n, k);
  if (need != 0 &&
      (workspace == nullptr || !cpx::aligned(workspace, 16) || workspace_bytes < need))
    return refuse("workspace must be 16-byte aligned and hold cp_linear_grad_call_bytes bytes");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* at = static_cast<uint8_t*>(workspace);

  // dz, where it is not dy on 16-byte boundaries already, and the parts of db
  Operand dz{dy, dy_stride, false};
  const bool has_dy = m != 0 && n != 0;
  const bool shape = activation != CP_ACT_NONE || g.drop.mode != 0;
  g.pitch = row_pitch(n);
  if (!as_is && has_dy) {
    dz = Operand{at, g.pitch, false};
    if (want_dx || want_dw) g.dz = at;
    at += dz_bytes(m, n);
  }
  ColumnSums sums{};
  if (db != nullptr && n != 0) {
    sums.out = db;
    sums.n = static_cast<uint32_t>(n);
    sums.dtype = db_dtype;
    sums.accumulate = accumulate;
    if (as_is && direct_sums(m, n, dtype)) {
      sums.rows = dy;
      sums.rows_dtype = dy_dtype;
      sums.pitch = dy_stride;
      sums.count = static_cast<uint32_t>(m);
    } else if (has_dy) {
      sums.parts = g.parts = reinterpret_cast<float*>(at);
      sums.pitch = g.pitch;
      sums.count = grad_parts(m, n, shape);
      at += db_bytes(m, n);
    }
  }
  // dx [m][k] = dz w: w is stored across n;  dw [n][k] = dz^T x: both are stored across m
  Operand xo{x, x_stride, true}, wo{w, w_stride, true};
  cpm::AlignOperand of[2];
  bool copies = false;
  if (has_dy && k != 0) {
    Operand* op[2] = {want_dw ? &xo : nullptr, want_dx ? &wo : nullptr};
    copies = to_align(op, {m, n}, k, at, of);
    for (const cpx::RowBytes& out :
         {cpx::RowBytes{dx, 2 * dx_stride, 2 * k, m},
          cpx::RowBytes{dw, dw_stride * dtype_size(dw_dtype), k * dtype_size(dw_dtype), n}}) {
      if (((want_dx || want_dw) && reads(dz, m, n, out)) || (want_dw && reads(xo, m, k, out)) ||
          (want_dx && reads(wo, n, k, out)))
        return refuse("dx or dw lies on dy, x or w, which are read while it is written");
    }
  }
  cudaError_t e = cudaSuccess;
  if (has_dy && (g.dz != nullptr || g.parts != nullptr)) {
    g.dy = dy;
    g.pre = pre;
    g.ldy = dy_stride;
    g.ldp = pre_stride;
    g.m = static_cast<uint32_t>(m);
    g.n = static_cast<uint32_t>(n);
    g.count = grad_parts(m, n, shape);
    g.act = activation;
    if (copies) {
      const uint32_t wide = (g.n + kGradColumns - 1) / kGradColumns;
      g.copy = cpm::align_params(of, static_cast<uint32_t>(2 * k), 2 * row_pitch(k));
      g.copy_rows = (cpm::align_ctas(g.copy) + wide - 1) / wide;
    }
    const bool vec = octets_ok(dy, dy_stride, g.n, dtype_size(dy_dtype)) &&
                     (pre == nullptr || octets_ok(pre, pre_stride, g.n, 2));
    if (dtype == CP_F16)
      e = dy_dtype == CP_F32 ? launch_dz<__half, float>(g, vec, s)
                             : launch_dz<__half, __half>(g, vec, s);
    else
      e = dy_dtype == CP_F32 ? launch_dz<__nv_bfloat16, float>(g, vec, s)
                             : launch_dz<__nv_bfloat16, __nv_bfloat16>(g, vec, s);
  } else if (copies) {
    e = cpm::align_rows(of, static_cast<uint32_t>(2 * k), 2 * row_pitch(k), s);
  }
  if (e != cudaSuccess) return cpx::cuda_fail(e, "linear gradient launch");

  Product q[cplin::kMostProducts] = {};
  int count = 0;
  if (want_dx) {
    Product& d = q[count++];
    d.a = dz;
    d.b = wo;
    d.k = static_cast<uint32_t>(n);
    d.e.out = dx;
    d.e.ldo = dx_stride;
    d.e.m = static_cast<uint32_t>(m);
    d.e.out_dtype = dtype;
  }
  if (want_dw && !(m == 0 && accumulate != 0)) {
    Product& d = q[count++];
    d.a = Operand{dz.p, dz.ld, true};
    d.b = xo;
    d.k = static_cast<uint32_t>(m);
    d.e.out = dw;
    d.e.ldo = dw_stride;
    d.e.m = static_cast<uint32_t>(n);
    d.e.out_dtype = dw_dtype;
    if (accumulate != 0) {
      d.e.residual = dw;
      d.e.ldr = dw_stride;
    }
  }
  for (int i = 0; i < count; ++i) {
    Product& d = q[i];
    d.dtype = dtype;
    d.e.n = static_cast<uint32_t>(k);
    d.e.aligned = cpx::sectors_ok(d.e.out, d.e.ldo, dtype_size(d.e.out_dtype));
  }
  Tiling chosen[cplin::kMostProducts] = {};
  if (count > 0) cplin::choose(ways, want_dx ? 0 : 1, count, chosen);
  return cplin::launch_products(q, count, chosen, sums, part_at(at), s);
}

// C entries of the MXFP4 quantiser and product and of the grouped products:
// argument checks before any launch, then one enqueue (two or three where a
// long sum is split).  Nothing here allocates or synchronises, so every call
// may be captured in a graph.
#include <hip/hip_runtime.h>

#include "../../include/moe_mxfp4.h"
#include "moe_internal.h"
#include "plan.h"

namespace {

using moe::fail;
using moe::hip_fail;
using moe::ok;

constexpr int32_t kMaxMatrixRows = 1 << 24;   // quantiser rows, grouped rows
constexpr int32_t kMaxMatmulDim = 1 << 19;
constexpr int32_t kMaxMatmulK = 1 << 16;
constexpr int64_t kMaxLd = 1 << 20;

// Scale bytes are read and written one by one or by unaligned loads, offsets
// one by one: a range of rows or of groups may start anywhere.
struct Ptr {
  const char* name;
  const void* p;
  unsigned align = 16;
};

template <int N>
moe_status check_ptrs(const Ptr (&ptrs)[N]) {
  for (const Ptr& q : ptrs) {
    if (!q.p) return fail(MOE_ERR_ARG, "%s is null", q.name);
    if (reinterpret_cast<uintptr_t>(q.p) % q.align)
      return fail(MOE_ERR_ALIGN, "%s must be %u-byte aligned, got %p", q.name, q.align, q.p);
  }
  return MOE_OK;
}

moe_status check_dtype(const char* name, int32_t dtype) {
  if (dtype != MOE_BF16 && dtype != MOE_F32)
    return fail(MOE_ERR_ARG, "%s must be MOE_BF16 (0) or MOE_F32 (1), got %d", name, dtype);
  return MOE_OK;
}

moe_status check_matrix(int32_t rows, int32_t cols) {
  if (rows < 0) return fail(MOE_ERR_ARG, "rows must be >= 0, got %d", rows);
  if (rows > kMaxMatrixRows) return fail(MOE_ERR_SHAPE, "rows must be at most %d, got %d", kMaxMatrixRows, rows);
  if (cols <= 0 || cols % 32) return fail(MOE_ERR_SHAPE, "cols must be a positive multiple of 32, got %d", cols);
  return MOE_OK;
}

moe_status check_grouped(int32_t rows, int32_t groups, int32_t n, int32_t k) {
  if (rows < 0) return fail(MOE_ERR_ARG, "rows must be >= 0, got %d", rows);
  if (rows > kMaxMatrixRows) return fail(MOE_ERR_SHAPE, "rows must be at most %d, got %d", kMaxMatrixRows, rows);
  if (groups < 0) return fail(MOE_ERR_ARG, "num_groups must be >= 0, got %d", groups);
  if (groups > moe::kGroupedMaxGroups)
    return fail(MOE_ERR_SHAPE, "num_groups must be at most %d, got %d", moe::kGroupedMaxGroups, groups);
  if (n < 8 || n > moe::kGroupedMaxDim || n % 8)
    return fail(MOE_ERR_SHAPE, "n must be a multiple of 8 in [8, %d], got %d", moe::kGroupedMaxDim, n);
  if (k < 8 || k > moe::kGroupedMaxDim || k % 8)
    return fail(MOE_ERR_SHAPE, "k must be a multiple of 8 in [8, %d], got %d", moe::kGroupedMaxDim, k);
  return MOE_OK;
}

moe_status check_ld(const char* name, int64_t ld, int32_t cols) {
  if (ld < cols || ld > kMaxLd || ld % 8)
    return fail(MOE_ERR_SHAPE, "%s must be a multiple of 8 in [%d, %lld], got %lld", name, cols, (long long)kMaxLd,
                (long long)ld);
  return MOE_OK;
}

// a workspace may be missing (nothing is split) but not too small
moe_status check_workspace(const void* p, size_t bytes, size_t need) {
  if (!p || !need) return MOE_OK;
  if (bytes < need) return fail(MOE_ERR_CAPACITY, "workspace must hold %zu bytes, got %zu", need, bytes);
  if (reinterpret_cast<uintptr_t>(p) & 15u) return fail(MOE_ERR_ALIGN, "workspace must be 16-byte aligned, got %p", p);
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_grouped_matmul_workspace(int32_t rows, int32_t num_groups, int32_t n, int32_t k) {
  if (check_grouped(rows, num_groups, n, k) || !rows || !num_groups) return 0;
  return moe::grouped_forward_workspace({nullptr, nullptr, rows, num_groups, n, k});
}

size_t moe_grouped_matmul_backward_workspace(int32_t rows, int32_t num_groups, int32_t n, int32_t k, int32_t need_dx,
                                             int32_t need_dw) {
  if (check_grouped(rows, num_groups, n, k) || !rows || !num_groups) return 0;
  return moe::grouped_backward_workspace({nullptr, nullptr, rows, num_groups, n, k}, need_dx, need_dw);
}

moe_status moe_mxfp4_quantize(const void* x, int32_t dtype, int32_t rows, int32_t cols, int64_t ldx, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream) {
  if (moe_status s = check_dtype("dtype", dtype)) return s;
  if (moe_status s = check_matrix(rows, cols)) return s;
  const int unit = dtype == MOE_F32 ? 4 : 8;   // elements in 16 bytes
  if (ldx < cols || ldx % unit)
    return fail(MOE_ERR_SHAPE, "ldx must be a multiple of %d of at least cols=%d, got %lld", unit, cols, (long long)ldx);
  if (rows == 0) return ok();
  if (moe_status s = check_ptrs({{"x", x}, {"codes", codes}, {"scales", scales, 1}})) return s;
  const hipError_t e = moe::launch_mxfp4_quantize(x, dtype == MOE_F32, rows, cols, ldx, codes, scales, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "mxfp4 quantise launch");
}

moe_status moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int32_t rows, int32_t cols, int32_t dtype,
                                void* out, hipStream_t stream) {
  if (moe_status s = check_dtype("dtype", dtype)) return s;
  if (moe_status s = check_matrix(rows, cols)) return s;
  if (rows == 0) return ok();
  if (moe_status s = check_ptrs({{"codes", codes}, {"scales", scales, 1}, {"out", out}})) return s;
  const hipError_t e = moe::launch_mxfp4_dequantize(codes, scales, rows, cols, dtype == MOE_F32, out, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "mxfp4 dequantise launch");
}

moe_status moe_mxfp4_matmul(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                            const uint8_t* b_scales, int32_t m, int32_t n, int32_t k, int32_t dtype, void* out,
                            hipStream_t stream) {
  if (moe_status s = check_dtype("dtype", dtype)) return s;
  if (m < 0 || n < 0) return fail(MOE_ERR_ARG, "m and n must be >= 0, got m=%d n=%d", m, n);
  if (m > kMaxMatmulDim || n > kMaxMatmulDim)
    return fail(MOE_ERR_SHAPE, "m and n must be at most %d, got m=%d n=%d", kMaxMatmulDim, m, n);
  if (k < 32 || k > kMaxMatmulK || k % 32)
    return fail(MOE_ERR_SHAPE, "k must be a multiple of 32 in [32, %d], got %d", kMaxMatmulK, k);
  if (m == 0 || n == 0) return ok();
  if (moe_status s = check_ptrs({{"a_codes", a_codes}, {"a_scales", a_scales, 1}, {"b_codes", b_codes},
                                 {"b_scales", b_scales, 1}, {"out", out}}))
    return s;
  const hipError_t e =
      moe::launch_mxfp4_matmul(a_codes, a_scales, b_codes, b_scales, m, n, k, dtype == MOE_F32, out, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "mxfp4 matmul launch");
}

moe_status moe_grouped_matmul(const uint16_t* x, int64_t ldx, const uint16_t* w, const int32_t* offsets, int32_t rows,
                              int32_t num_groups, int32_t n, int32_t k, uint16_t* out, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  if (moe_status s = check_grouped(rows, num_groups, n, k)) return s;
  if (moe_status s = check_ld("ldx", ldx, k)) return s;
  if (rows == 0 || num_groups == 0) return ok();
  if (moe_status s = check_ptrs({{"x", x}, {"w", w}, {"offsets", offsets, 4}, {"out", out}})) return s;
  const moe::GroupedArgs a{w, offsets, rows, num_groups, n, k};
  if (moe_status s = check_workspace(workspace, workspace_bytes, moe::grouped_forward_workspace(a))) return s;
  const hipError_t e = moe::launch_grouped_forward(a, x, ldx, out, workspace, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "grouped matmul launch");
}

moe_status moe_grouped_matmul_backward(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx,
                                       const uint16_t* w, const int32_t* offsets, int32_t rows, int32_t num_groups,
                                       int32_t n, int32_t k, uint16_t* dx, void* dw, int32_t dw_dtype,
                                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (moe_status s = check_dtype("dw_dtype", dw_dtype)) return s;
  if (moe_status s = check_grouped(rows, num_groups, n, k)) return s;
  if (moe_status s = check_ld("lddy", lddy, n)) return s;
  if (dw)   // x is read for dw only
    if (moe_status s = check_ld("ldx", ldx, k)) return s;
  if (rows == 0) dx = nullptr;   // no rows to write
  if (num_groups == 0 || (!dx && !dw)) return ok();
  if (moe_status s = check_ptrs({{"offsets", offsets, 4}})) return s;
  if (rows > 0)   // without rows every weight gradient is zero and nothing is read
    if (moe_status s = check_ptrs({{"dy", dy}})) return s;
  if (dx)
    if (moe_status s = check_ptrs({{"w", w}, {"dx", dx}})) return s;
  if (dw) {
    if (moe_status s = check_ptrs({{"dw", dw}})) return s;
    if (rows > 0)
      if (moe_status s = check_ptrs({{"x", x}})) return s;
  }
  const moe::GroupedArgs a{w, offsets, rows, num_groups, n, k};
  if (moe_status s = check_workspace(workspace, workspace_bytes, moe::grouped_backward_workspace(a, dx, dw))) return s;
  const hipError_t e =
      moe::launch_grouped_backward(a, dy, lddy, x, ldx, dx, dw_dtype == MOE_F32, dw, workspace, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "grouped matmul backward launch");
}

}  // extern "C"

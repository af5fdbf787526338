// C entries of the operators beside the layer (MXFP4 quantiser and products,
// grouped products, scored router, experts' combine): argument checks before
// any launch, then one enqueue (two or three where a long sum is split).
// Nothing here allocates or synchronises, so every call may be captured in a
// graph.
#include <hip/hip_runtime.h>

#include <cmath>

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
constexpr int32_t kMaxCombineRows = 1 << 26;
constexpr int32_t kMaxCombineTokens = 1 << 21;   // a workgroup of up to 1024 threads each, in one launch

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

moe_status check_product(int32_t m, int32_t n, int32_t k) {
  if (m < 0 || n < 0) return fail(MOE_ERR_ARG, "m and n must be >= 0, got m=%d n=%d", m, n);
  if (m > kMaxMatmulDim || n > kMaxMatmulDim)
    return fail(MOE_ERR_SHAPE, "m and n must be at most %d, got m=%d n=%d", kMaxMatmulDim, m, n);
  if (k < 32 || k > kMaxMatmulK || k % 32)
    return fail(MOE_ERR_SHAPE, "k must be a multiple of 32 in [32, %d], got %d", kMaxMatmulK, k);
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

moe_status check_ld(const char* name, int64_t ld, int32_t cols, int unit = 8) {
  if (ld < cols || ld > kMaxLd || ld % unit)
    return fail(MOE_ERR_SHAPE, "%s must be a multiple of %d in [%d, %lld], got %lld", name, unit, cols,
                (long long)kMaxLd, (long long)ld);
  return MOE_OK;
}

moe_status check_router(int32_t dtype, int32_t tokens, int32_t experts, int32_t top_k, int64_t ld, int32_t score,
                        float scale) {
  if (moe_status s = check_dtype("dtype", dtype)) return s;
  if (tokens < 0) return fail(MOE_ERR_ARG, "num_tokens must be >= 0, got %d", tokens);
  if (tokens > kMaxMatrixRows) return fail(MOE_ERR_SHAPE, "num_tokens must be at most %d, got %d", kMaxMatrixRows, tokens);
  if (experts < 1 || experts > moe::kRouterMaxExperts)
    return fail(MOE_ERR_SHAPE, "num_experts must be in [1, %d], got %d", moe::kRouterMaxExperts, experts);
  if (top_k < 1 || top_k > moe::kMaxTopK || top_k > experts)
    return fail(MOE_ERR_SHAPE, "top_k must be in [1, min(%d, num_experts=%d)], got %d", moe::kMaxTopK, experts, top_k);
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_ARG, "score must be MOE_SCORE_SOFTMAX (0) or MOE_SCORE_SIGMOID (1), got %d", score);
  if (!std::isfinite(scale)) return fail(MOE_ERR_ARG, "scale must be finite, got %g", (double)scale);
  return check_ld("ldl", ld, experts, 1);
}

moe_status check_combine(int32_t rows, int32_t tokens, int32_t top_k, int32_t hidden) {
  if (rows < 0 || tokens < 0) return fail(MOE_ERR_ARG, "rows and num_tokens must be >= 0, got rows=%d num_tokens=%d", rows, tokens);
  if (rows > kMaxCombineRows) return fail(MOE_ERR_SHAPE, "rows must be at most %d, got %d", kMaxCombineRows, rows);
  if (tokens > kMaxCombineTokens)
    return fail(MOE_ERR_SHAPE, "num_tokens must be at most %d, got %d", kMaxCombineTokens, tokens);
  if (top_k < 1 || top_k > moe::kMaxTopK)
    return fail(MOE_ERR_SHAPE, "top_k must be in [1, %d], got %d", moe::kMaxTopK, top_k);
  if (hidden < 8 || hidden > moe::kGroupedMaxDim || hidden % 8)
    return fail(MOE_ERR_SHAPE, "hidden must be a multiple of 8 in [8, %d], got %d", moe::kGroupedMaxDim, hidden);
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
  if (moe_status s = check_product(m, n, k)) return s;
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

moe_status moe_router_select(const void* logits, int32_t dtype, int64_t ldl, int32_t num_tokens, int32_t num_experts,
                             int32_t top_k, int32_t score, const float* bias, int32_t num_groups, int32_t group_limit,
                             int32_t group_top, int32_t renormalize, float scale, int32_t* topk_ids,
                             float* topk_weights, hipStream_t stream) {
  if (moe_status s = check_router(dtype, num_tokens, num_experts, top_k, ldl, score, scale)) return s;
  if (num_groups < 1 || num_groups > moe::kRouterMaxGroups || num_experts % num_groups)
    return fail(MOE_ERR_SHAPE, "num_groups must divide num_experts=%d and be in [1, %d], got %d", num_experts,
                moe::kRouterMaxGroups, num_groups);
  if (group_limit < 1 || group_limit > num_groups)
    return fail(MOE_ERR_SHAPE, "group_limit must be in [1, num_groups=%d], got %d", num_groups, group_limit);
  if (group_top < 1 || group_top > 2) return fail(MOE_ERR_SHAPE, "group_top must be 1 or 2, got %d", group_top);
  if (top_k > group_limit * (num_experts / num_groups))
    return fail(MOE_ERR_SHAPE, "top_k=%d is more than the %d experts of group_limit groups", top_k,
                group_limit * (num_experts / num_groups));
  if (num_tokens == 0) return ok();
  if (moe_status s = check_ptrs({{"logits", logits, dtype == MOE_F32 ? 4u : 2u}, {"topk_ids", topk_ids, 4},
                                 {"topk_weights", topk_weights, 4}}))
    return s;
  if (bias)
    if (moe_status s = check_ptrs({{"bias", bias, 4}})) return s;
  const hipError_t e = moe::launch_router_select(
      {logits, ldl, bias, topk_ids, topk_weights, num_tokens, num_experts, top_k, num_groups, group_limit, group_top,
       score, scale, renormalize != 0}, dtype == MOE_F32, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "router select launch");
}

moe_status moe_router_select_backward(const float* dweights, const void* logits, int32_t dtype, int64_t ldl,
                                      const int32_t* topk_ids, int32_t num_tokens, int32_t num_experts, int32_t top_k,
                                      int32_t score, int32_t renormalize, float scale, void* dlogits,
                                      hipStream_t stream) {
  if (moe_status s = check_router(dtype, num_tokens, num_experts, top_k, ldl, score, scale)) return s;
  if (num_tokens == 0) return ok();
  const unsigned size = dtype == MOE_F32 ? 4 : 2;
  if (moe_status s = check_ptrs({{"dweights", dweights, 4}, {"logits", logits, size}, {"topk_ids", topk_ids, 4},
                                 {"dlogits", dlogits}}))
    return s;
  const hipError_t e = moe::launch_router_select_backward(
      {dweights, logits, ldl, topk_ids, dlogits, num_tokens, num_experts, top_k, score, scale, renormalize != 0},
      dtype == MOE_F32, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "router select backward launch");
}

moe_status moe_mxfp4_linear(const uint16_t* x, int64_t ldx, const uint8_t* codes, const uint8_t* scales, int32_t m,
                            int32_t n, int32_t k, int32_t gate, int32_t dtype, void* out, hipStream_t stream) {
  if (moe_status s = check_dtype("dtype", dtype)) return s;
  if (moe_status s = check_product(m, n, k)) return s;
  if (gate && n % 2) return fail(MOE_ERR_SHAPE, "a gated product needs an even n, got %d", n);
  if (moe_status s = check_ld("ldx", ldx, k)) return s;
  if (m == 0 || n == 0) return ok();
  if (moe_status s = check_ptrs({{"x", x}, {"codes", codes}, {"scales", scales, 1}, {"out", out}})) return s;
  const hipError_t e = moe::launch_mxfp4_linear({x, ldx, codes, scales, out, m, n, k}, gate, dtype == MOE_F32, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "mxfp4 linear launch");
}

moe_status moe_expert_combine(const uint16_t* y, int64_t ldy, int32_t rows, const int32_t* rowpos,
                              const float* weights, int32_t num_tokens, int32_t top_k, int32_t hidden, int32_t dtype,
                              void* out, hipStream_t stream) {
  if (moe_status s = check_dtype("dtype", dtype)) return s;
  if (moe_status s = check_combine(rows, num_tokens, top_k, hidden)) return s;
  if (moe_status s = check_ld("ldy", ldy, hidden)) return s;
  if (num_tokens == 0) return ok();
  if (moe_status s = check_ptrs({{"rowpos", rowpos, 4}, {"out", out}})) return s;
  if (rows > 0)   // without rows every output is zero
    if (moe_status s = check_ptrs({{"y", y}})) return s;
  if (weights)
    if (moe_status s = check_ptrs({{"weights", weights, 4}})) return s;
  const hipError_t e = moe::launch_expert_combine({y, ldy, rowpos, weights, out, rows, num_tokens, top_k, hidden},
                                                  dtype == MOE_F32, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "expert combine launch");
}

moe_status moe_expert_combine_backward(const void* dout, int32_t dout_dtype, int64_t lddout, const uint16_t* y,
                                       int64_t ldy, int32_t rows, const int32_t* rowpos, const int32_t* perm,
                                       const float* weights, int32_t num_tokens, int32_t top_k, int32_t hidden,
                                       uint16_t* dy, float* dweights, hipStream_t stream) {
  if (moe_status s = check_dtype("dout_dtype", dout_dtype)) return s;
  if (moe_status s = check_combine(rows, num_tokens, top_k, hidden)) return s;
  if (moe_status s = check_ld("lddout", lddout, hidden, dout_dtype == MOE_F32 ? 4 : 8)) return s;
  if (dweights)   // y is read for them only
    if (moe_status s = check_ld("ldy", ldy, hidden)) return s;
  if (rows == 0) dy = nullptr;   // no rows to write
  if (num_tokens == 0 || (!dy && !dweights)) return ok();
  if (moe_status s = check_ptrs({{"dout", dout}, {"rowpos", rowpos, 4}})) return s;
  if (weights)
    if (moe_status s = check_ptrs({{"weights", weights, 4}})) return s;
  if (dy)
    if (moe_status s = check_ptrs({{"perm", perm, 4}, {"dy", dy}})) return s;
  if (dweights) {
    if (moe_status s = check_ptrs({{"dweights", dweights, 4}})) return s;
    if (rows > 0)
      if (moe_status s = check_ptrs({{"y", y}})) return s;
  }
  const hipError_t e = moe::launch_expert_combine_backward(
      {dout, lddout, y, ldy, rowpos, perm, weights, dy, dweights, rows, num_tokens, top_k, hidden},
      dout_dtype == MOE_F32, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "expert combine backward launch");
}

}  // extern "C"

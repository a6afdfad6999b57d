// C ABI of the products in 8-bit floating point (moe_fp8.h): argument checks,
// plans, the launch sequences.
#include <algorithm>

#include "api_checks.h"
#include "fp8.h"

namespace moe {

namespace {

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

bool is_gated(moe_fp8_op op) { return op == MOE_FP8_GATED || op == MOE_FP8_GATED_BACKWARD; }

moe_status check_shape(const moe_product* p, moe_fp8_op op) {
  if (!p) return api_fail(MOE_ERR_INVALID_ARG, "null pointer argument");
  if (op < MOE_FP8_PRODUCT || op > MOE_FP8_GATED_BACKWARD)
    return api_fail(MOE_ERR_INVALID_ARG, "op=%d is no moe_fp8_op", (int)op);
  const bool gated = is_gated(op);
  if (p->rows < 0 || p->rows > kMaxRows)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "rows=%d outside [0, %d]", p->rows, kMaxRows);
  const int max_n = gated ? kMaxWidth / 2 : kMaxWidth;
  if (p->n < 16 || p->n > max_n || p->n % 16)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "n=%d must be a multiple of 16 in [16, %d]", p->n, max_n);
  if (p->k < 16 || p->k > kMaxWidth || p->k % 16)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "k=%d must be a multiple of 16 in [16, %d]", p->k, kMaxWidth);
  if (p->groups < 1 || p->groups > kMaxGroups)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "groups=%d outside [1, %d]", p->groups, kMaxGroups);
  if (p->type != MOE_TYPE_BF16 && p->type != MOE_TYPE_FP16)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "type=%d must be bf16 or fp16", p->type);
  if (gated ? (p->activation != MOE_ACT_SILU && p->activation != MOE_ACT_GELU) : p->activation != 0)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "activation=%d is not supported here", p->activation);
  return MOE_OK;
}

// Codes of rows and their scales; null allowed only without rows.
moe_status check_codes(const uint8_t* codes, int64_t ld, const float* scale, int64_t ldscale, int rows, int width) {
  MOE_TRY(check_rows("codes", codes, ld, rows, width, 16));
  if (!scale && rows > 0) return api_fail(MOE_ERR_INVALID_ARG, "scale is null");
  if (reinterpret_cast<uintptr_t>(scale) % 4) return api_fail(MOE_ERR_INVALID_ARG, "scale is not 4-byte aligned");
  if (ldscale < rows || ldscale > kMaxRows)
    return api_fail(MOE_ERR_INVALID_ARG, "stride %lld of scale's blocks must be in [%d, %d]", (long long)ldscale, rows,
                    kMaxRows);
  return MOE_OK;
}

moe_status check_weights(const uint8_t* w, const float* w_scale) {
  MOE_TRY(check_plain("w", w));
  if (!w_scale) return api_fail(MOE_ERR_INVALID_ARG, "w_scale is null");
  if (reinterpret_cast<uintptr_t>(w_scale) % 4) return api_fail(MOE_ERR_INVALID_ARG, "w_scale is not 4-byte aligned");
  return MOE_OK;
}

// The products' shapes (the operands are filled in by the caller).
Fp8Args shape_args(const moe_product* p, bool gated) {
  Fp8Args a;
  const int64_t nb = scale_blocks(p->n), kb = scale_blocks(p->k);
  a.groups = p->groups;
  a.rows = p->rows;
  a.ldq = p->k;
  a.q_group = (int64_t)p->n * (gated ? 2 : 1) * p->k;
  a.out_type = p->type;
  a.act = p->activation;
  a.qs_half = nb * kb;
  a.qs_group = nb * kb * (gated ? 2 : 1);
  return a;
}
Fp8Args forward_args(const moe_product* p, bool gated) {
  Fp8Args a = shape_args(p, gated);
  a.contract = p->k;
  a.cols = gated ? 2 * p->n : p->n;
  a.qs_cols = scale_blocks(p->k);
  a.qs_stage = 1;
  return a;
}
Fp8Args input_grad_args(const moe_product* p, bool gated) {
  Fp8Args a = shape_args(p, gated);
  a.contract = p->n;
  a.halves = gated ? 2 : 1;
  a.cols = p->k;
  a.qs_cols = 1;
  a.qs_stage = scale_blocks(p->k);
  return a;
}
// The rules of the integer codes (ops_api.hip), whose operands have the same bytes,
// fit.  us by streaming, 128-wide tiles and 256-wide tiles; rows / groups, columns
// of contraction.  Streamed: 64 / 1, 1024 of 4096 10.4, 14.1, 16.5; 256 / 1, 2048
// of 2048 10.4, 14.6, 19.7; 128 / 8, 4096 of 14336 86.6, 100, 116; gated 128 / 8,
// 14336 of 4096 171, 183, 208.  128: 256 / 8, 4096 of 14336 115, 101, 118; gated
// 256 / 8, 14336 of 4096 226, 185, 210; 1600 / 8, 4096 of 4096 111, 40.9, 50.0.  256:
// 3000 / 1, 4096 of 4096 167, 63.2, 55.6.  The input gradient (128 / 256): 2048 / 1,
// 4096 and 4096 45.3, 55.2; 3000 / 1 64.0, 57.2; 32 / 8, 14336 and 4096 102, 120.
ProductPlan plan_fp8(const Fp8Args& a, Pass pass, Result res) {
  ProductArgs b = a;
  b.contract = a.halves * scale_blocks(a.contract) * kScaleBlock;
  return plan_product(Num::kInt8, pass, res, b);
}
Result result_of(bool gated) { return gated ? Result::kGated : Result::kHalf; }

// The gated backward pass's codes of (dg, du) and their scales.
size_t slopes_codes_bytes(const moe_product* p) {
  return align_up((size_t)p->rows * 2 * scale_blocks(p->n) * kScaleBlock);
}
size_t slopes_bytes(const moe_product* p) {
  return slopes_codes_bytes(p) + align_up((size_t)p->rows * 2 * scale_blocks(p->n) * sizeof(float));
}

size_t workspace_bytes_of(const moe_product* p, moe_fp8_op op) {
  switch (op) {
    case MOE_FP8_PRODUCT:
    case MOE_FP8_GATED:
      return plan_fp8(forward_args(p, is_gated(op)), Pass::kForward, result_of(is_gated(op))).partial_bytes;
    default: {
      const bool gated = is_gated(op);
      return plan_fp8(input_grad_args(p, gated), Pass::kInputGrad, Result::kHalf).partial_bytes +
             (gated ? slopes_bytes(p) : 0);
    }
  }
}

moe_status enqueue(Fp8Args& a, const ProductPlan& plan, Pass pass, Result res, void* partial, hipStream_t s) {
  a.splits = plan.splits;
  a.partial = static_cast<char*>(partial);
  if (plan.family == Family::kStream)
    launch_fp8_stream(a, res, s);
  else
    launch_fp8_tiles(a, plan, pass, res, s);
  return check_launch();
}

moe_status forward(const moe_product* p, moe_fp8_op op, const uint8_t* codes, int64_t ldcodes, const float* scale,
                   int64_t ldscale, const uint8_t* w, const float* w_scale, const int32_t* offsets, void* out,
                   int64_t ldout, uint16_t* keep, int64_t ldkeep, void* workspace, size_t workspace_bytes,
                   moe_stream stream) {
  MOE_TRY(check_shape(p, op));
  const bool gated = is_gated(op);
  MOE_TRY(check_codes(codes, ldcodes, scale, ldscale, p->rows, p->k));
  MOE_TRY(check_weights(w, w_scale));
  MOE_TRY(check_rows(gated ? "h" : "out", out, ldout, p->rows, p->n, 8));
  if (keep) MOE_TRY(check_rows("gate_up", keep, ldkeep, p->rows, 2 * p->n, 8));
  MOE_TRY(check_offsets(p, offsets));
  Fp8Args a = forward_args(p, gated);
  const Result res = result_of(gated);
  const ProductPlan plan = plan_fp8(a, Pass::kForward, res);
  MOE_TRY(check_workspace(workspace, workspace_bytes, plan.partial_bytes));
  if (p->rows == 0) return MOE_OK;
  a.p = reinterpret_cast<const char*>(codes);
  a.ldp = ldcodes;
  a.pscale = scale;
  a.ldscale = ldscale;
  a.q = reinterpret_cast<const char*>(w);
  a.qscale = w_scale;
  a.offsets = offsets;
  a.out = out;
  a.ldout = ldout;
  a.keep = keep;
  a.ldkeep = ldkeep;
  return enqueue(a, plan, Pass::kForward, res, workspace, static_cast<hipStream_t>(stream));
}

moe_status input_grad(const moe_product* p, bool gated, const uint8_t* codes, int64_t ldcodes, const float* scale,
                      int64_t ldscale, const uint8_t* w, const float* w_scale, const int32_t* offsets, void* dx,
                      int64_t lddx, void* partial, hipStream_t s) {
  Fp8Args a = input_grad_args(p, gated);
  const Result res = Result::kHalf;
  const ProductPlan plan = plan_fp8(a, Pass::kInputGrad, res);
  a.p = reinterpret_cast<const char*>(codes);
  a.ldp = ldcodes;
  a.pscale = scale;
  a.ldscale = ldscale;
  a.q = reinterpret_cast<const char*>(w);
  a.qscale = w_scale;
  a.offsets = offsets;
  a.out = dx;
  a.ldout = lddx;
  return enqueue(a, plan, Pass::kInputGrad, res, partial, s);
}

moe_status check_values(int32_t rows, int max_rows, int32_t k, int32_t type) {
  if (rows < 0 || rows > max_rows)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "rows=%d outside [0, %d]", rows, max_rows);
  if (k < 16 || k > kMaxWidth || k % 16)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "k=%d must be a multiple of 16 in [16, %d]", k, kMaxWidth);
  if (type != MOE_TYPE_BF16 && type != MOE_TYPE_FP16)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "type=%d must be bf16 or fp16", type);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_EXPORT moe_status moe_fp8_workspace(const moe_product* p, moe_fp8_op op, size_t* bytes) {
  MOE_TRY(check_shape(p, op));
  if (!bytes) return api_fail(MOE_ERR_INVALID_ARG, "null pointer argument");
  *bytes = workspace_bytes_of(p, op);
  return MOE_OK;
}

MOE_EXPORT moe_status moe_quantize_blocks(int32_t rows, int32_t k, int32_t type, const uint16_t* x, int64_t ldx,
                                          uint8_t* codes, int64_t ldcodes, float* scale, int64_t ldscale,
                                          moe_stream stream) {
  MOE_TRY(check_values(rows, kMaxRows, k, type));
  MOE_TRY(check_rows("x", x, ldx, rows, k, 8));
  MOE_TRY(check_codes(codes, ldcodes, scale, ldscale, rows, k));
  if (rows == 0) return MOE_OK;
  launch_quantize_blocks(rows, k, type, x, ldx, codes, ldcodes, scale, ldscale, static_cast<hipStream_t>(stream));
  return check_launch();
}

MOE_EXPORT moe_status moe_quantize_tiles(int32_t matrices, int32_t n, int32_t k, int32_t type, const uint16_t* x,
                                         uint8_t* codes, float* scale, moe_stream stream) {
  MOE_TRY(check_values(n, kMaxWidth, k, type));
  if (n < 1) return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "n=%d outside [1, %d]", n, kMaxWidth);
  if (matrices < 0 || matrices > 2 * kMaxGroups)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "matrices=%d outside [0, %d]", matrices, 2 * kMaxGroups);
  if (matrices == 0) return MOE_OK;
  MOE_TRY(check_plain("x", x));
  MOE_TRY(check_plain("codes", codes));
  if (!scale) return api_fail(MOE_ERR_INVALID_ARG, "scale is null");
  if (reinterpret_cast<uintptr_t>(scale) % 4) return api_fail(MOE_ERR_INVALID_ARG, "scale is not 4-byte aligned");
  launch_quantize_tiles(matrices, n, k, type, x, codes, scale, static_cast<hipStream_t>(stream));
  return check_launch();
}

MOE_EXPORT moe_status moe_fp8_product(const moe_product* p, const uint8_t* codes, int64_t ldcodes, const float* scale,
                                      int64_t ldscale, const uint8_t* w, const float* w_scale, const int32_t* offsets,
                                      uint16_t* out, int64_t ldout, void* workspace, size_t workspace_bytes,
                                      moe_stream stream) {
  return forward(p, MOE_FP8_PRODUCT, codes, ldcodes, scale, ldscale, w, w_scale, offsets, out, ldout, nullptr, 0,
                 workspace, workspace_bytes, stream);
}

MOE_EXPORT moe_status moe_fp8_gated(const moe_product* p, const uint8_t* codes, int64_t ldcodes, const float* scale,
                                    int64_t ldscale, const uint8_t* w, const float* w_scale, const int32_t* offsets,
                                    uint16_t* h, int64_t ldh, uint16_t* gate_up, int64_t ldgate_up, void* workspace,
                                    size_t workspace_bytes, moe_stream stream) {
  return forward(p, MOE_FP8_GATED, codes, ldcodes, scale, ldscale, w, w_scale, offsets, h, ldh, gate_up, ldgate_up,
                 workspace, workspace_bytes, stream);
}

MOE_EXPORT moe_status moe_fp8_product_backward(const moe_product* p, const uint8_t* codes, int64_t ldcodes,
                                               const float* scale, int64_t ldscale, const uint8_t* w,
                                               const float* w_scale, const int32_t* offsets, uint16_t* dx, int64_t lddx,
                                               void* workspace, size_t workspace_bytes, moe_stream stream) {
  MOE_TRY(check_shape(p, MOE_FP8_PRODUCT_BACKWARD));
  MOE_TRY(check_codes(codes, ldcodes, scale, ldscale, p->rows, p->n));
  MOE_TRY(check_weights(w, w_scale));
  MOE_TRY(check_rows("dx", dx, lddx, p->rows, p->k, 8));
  MOE_TRY(check_offsets(p, offsets));
  MOE_TRY(check_workspace(workspace, workspace_bytes, workspace_bytes_of(p, MOE_FP8_PRODUCT_BACKWARD)));
  if (p->rows == 0) return MOE_OK;
  return input_grad(p, false, codes, ldcodes, scale, ldscale, w, w_scale, offsets, dx, lddx, workspace,
                    static_cast<hipStream_t>(stream));
}

MOE_EXPORT moe_status moe_fp8_gated_backward(const moe_product* p, const uint16_t* dh, int64_t lddh,
                                             const uint16_t* gate_up, int64_t ldgate_up, const uint8_t* w,
                                             const float* w_scale, const int32_t* offsets, uint16_t* dx, int64_t lddx,
                                             uint16_t* slopes, int64_t ldslopes, void* workspace,
                                             size_t workspace_bytes, moe_stream stream) {
  MOE_TRY(check_shape(p, MOE_FP8_GATED_BACKWARD));
  MOE_TRY(check_rows("dh", dh, lddh, p->rows, p->n, 8));
  MOE_TRY(check_rows("gate_up", gate_up, ldgate_up, p->rows, 2 * p->n, 8));
  if (dx) {
    MOE_TRY(check_rows("dx", dx, lddx, p->rows, p->k, 8));
    MOE_TRY(check_weights(w, w_scale));
  }
  if (slopes) MOE_TRY(check_rows("slopes", slopes, ldslopes, p->rows, 2 * p->n, 8));
  MOE_TRY(check_offsets(p, offsets));
  MOE_TRY(check_workspace(workspace, workspace_bytes, workspace_bytes_of(p, MOE_FP8_GATED_BACKWARD)));
  if (p->rows == 0 || (!dx && !slopes)) return MOE_OK;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  // the codes first in the workspace, then their scales, then the parts of a split contraction
  char* at = static_cast<char*>(workspace);
  uint8_t* codes = dx ? reinterpret_cast<uint8_t*>(at) : nullptr;
  float* scale = reinterpret_cast<float*>(at + slopes_codes_bytes(p));
  launch_fp8_slopes(p->rows, p->n, p->type, p->activation, dh, lddh, gate_up, ldgate_up, offsets, p->groups, slopes,
                    ldslopes, codes, scale, p->rows, s);
  MOE_TRY(check_launch());
  if (!dx) return MOE_OK;
  return input_grad(p, true, codes, 2 * scale_blocks(p->n) * kScaleBlock, scale, p->rows, w, w_scale, offsets, dx, lddx,
                    at + slopes_bytes(p), s);
}

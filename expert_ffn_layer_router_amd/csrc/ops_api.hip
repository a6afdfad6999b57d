// C ABI of the grouped products (moe_ops.h): argument checks, plans, the
// launch sequences.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "products.h"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

namespace moe {
moe_status api_fail(moe_status st, const char* fmt, ...);

namespace {

constexpr int kMaxRows = 1 << 22, kMaxWidth = 65536, kMaxGroups = 256;
constexpr int64_t kMaxStride = 1 << 20;
// The streaming kernel takes calls with up to 16 rows per group on average:
// reading the used groups' weights is then most of the time, and it reads them
// faster than the tiles do, whose rows are mostly padding (16 rows x one group
// of 6400 gated columns of 4096 in bf16: 25.8 against 38.4 us; 256 rows over
// 16 groups of 4096 columns of 2048: 55 against 75; 384 over 64 of 2048 gated
// columns of 4096: 374 against 565; uneven groups cost it: 128 rows over 16
// groups of 4096 columns of 6400, 47 in the largest: 169 against 158).
constexpr int kStreamGroupRows = 16;
// With more rows its blocks read them again for every 32 columns, and the
// weights again for every 64 rows of a group.  That still beats the tiles'
// fixed costs, a second kernel for the split contraction among them, as long
// as these reads are few, in bytes (what the caches deliver) and in 64-byte
// steps' worth of rows (short rows: what a block's start and end cost).
// Below the limits, in bf16: 256 rows x 2048 columns of 2048 (89 MB, 22 k
// rows): 11.2 against 23.0 us; 128 x 4096 of 4096 (161 MB): 17.7 against 23.5;
// 1000 x 512 of 4096 (193 MB): 18.8 against 24.6; 2000 x 512 of 512 (49 MB,
// 49 k rows): 9.0 against 9.9; 40 x 25600 of 1024 (31 k rows): 22.6 against
// 20.0.  Above: 64 x 12800 of 4096 (201 MB): 44.8 against 39.9; 300 x 4096 of
// 1024 (54 k rows): 15.4 against 13.8; 512 x 8192 of 192 (185 k): 14.4 against
// 8.6; 1536 rows over 64 groups of 4096 columns of 2048 (774 MB): 281 against
// 218.  The rows of one of many uneven groups are few blocks' work: 1000 rows
// over 16 groups of 1024 columns of 1024, 202 in the largest: 18.4 against
// 15.2; 800 over 8 of 2048: 22.7 against 24.8.  The limits were fitted to bf16
// and are the same for codes, whose rows have half the bytes.
constexpr int64_t kStreamExtraBytes = 196 << 20, kStreamExtraRows = 48 << 10;
constexpr int kStreamExtraGroups = 8;

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

ProductPlan plan_product(Num num, Pass pass, Result res, const ProductArgs& a) {
  ProductPlan p;
  const bool gated = res == Result::kGated, wg = pass == Pass::kWeightGrad;
  if (pass == Pass::kForward) {
    const int64_t row_bytes = (int64_t)a.contract * (num == Num::kInt8 ? 1 : 2);
    const int64_t row_reads = (int64_t)(a.cols / 32 + 1) * a.rows;
    const int64_t weight_reads = (a.rows - 1) / (64 * a.groups) * ((int64_t)a.groups * a.cols);
    const int64_t extra = row_reads + weight_reads;  // rows of either operand
    if (a.rows <= kStreamGroupRows * a.groups ||
        (a.groups <= kStreamExtraGroups && extra <= kStreamExtraRows && extra * row_bytes <= kStreamExtraBytes)) {
      p.family = Family::kStream;
      return p;
    }
  }
  // rows of an average group: the tiles' rows, or in the weight gradient the
  // contraction; the offsets themselves are on the device
  const int group_rows = std::max(1, ceil_div(a.rows, a.groups));
  const int cols = gated ? a.cols / 2 : a.cols;
  auto blocks = [&](int tile) {
    const int64_t m = (int64_t)a.groups * ceil_div(wg ? a.wrows : group_rows, tile);
    return m * ceil_div(cols, gated ? tile / 2 : tile);
  };
  // 256 x 256 blocks run 25% faster (1460 against 1180 TFLOP/s at 8192^3 in
  // bf16) where they nearly fill the compute units: 192 blocks (3000 rows x
  // 4096 columns of 4096): 97 against 115 us, 128 blocks (2048 rows): 88
  // against 72.  Groups of up to 128 rows leave half of such a block empty.
  const bool large = blocks(256) >= 160 && (wg || group_rows > 128);
  p.family = large ? Family::kTile256 : Family::kTile128;
  const int tile = large ? 256 : 128;
  const int stages = ceil_div(wg ? group_rows : a.contract, num == Num::kInt8 ? 128 : 64);
  size_t units;
  if (wg) {
    // fewer tiles than the compute units hold: split the contraction, in
    // parts of at least 4 stages of an average group
    const int64_t tiles = blocks(tile);
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({8, 512 / tiles, stages / 4}));
    if (large) p.splits = 1;
    units = tiles * p.splits;
  } else {
    // the most parts of a tile that can pay (rounds_of)
    const int64_t tiles = (int64_t)row_tile_bound(a.rows, a.groups, tile) * ceil_div(cols, gated ? tile / 2 : tile);
    p.splits = std::max(1, std::min(8, stages / 4));
    if (stages * (p.splits - 1) / p.splits <= (large ? 6 : 12)) p.splits = 1;
    units = split_units(tile, (int)std::min<int64_t>(tiles, 1 << 20), p.splits);
  }
  if (p.splits > 1) p.partial_bytes = units * tile * tile * 4;
  return p;
}

namespace {

moe_status check_shape(const moe_product* p, moe_op op) {
  if (!p) return api_fail(MOE_ERR_INVALID_ARG, "null pointer argument");
  if (op < MOE_OP_INT8_PRODUCT || op > MOE_OP_GATED_PRODUCT_BACKWARD)
    return api_fail(MOE_ERR_INVALID_ARG, "op=%d is no moe_op", (int)op);
  const bool codes = op == MOE_OP_INT8_PRODUCT || op == MOE_OP_INT8_GATED;
  const bool gated = op == MOE_OP_INT8_GATED || op == MOE_OP_GATED_PRODUCT || op == MOE_OP_GATED_PRODUCT_BACKWARD;
  if (p->rows < 0 || p->rows > kMaxRows)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "rows=%d outside [0, %d]", p->rows, kMaxRows);
  const int max_n = gated ? kMaxWidth / 2 : kMaxWidth;
  if (p->n < 8 || p->n > max_n || p->n % 8)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "n=%d must be a multiple of 8 in [8, %d]", p->n, max_n);
  const int unit = codes ? 16 : 8;
  if (p->k < unit || p->k > kMaxWidth || p->k % unit)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "k=%d must be a multiple of %d in [%d, %d]", p->k, unit, unit, kMaxWidth);
  if (p->groups < 1 || p->groups > kMaxGroups)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "groups=%d outside [1, %d]", p->groups, kMaxGroups);
  if (p->type != MOE_TYPE_BF16 && p->type != MOE_TYPE_FP16 && !(p->type == MOE_TYPE_FP32 && op == MOE_OP_INT8_PRODUCT))
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "type=%d is not supported here", p->type);
  if (gated ? (p->activation != MOE_ACT_SILU && p->activation != MOE_ACT_GELU) : p->activation != 0)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "activation=%d is not supported here", p->activation);
  return MOE_OK;
}

// A row matrix: null allowed only without rows.
moe_status check_rows(const char* name, const void* m, int64_t ld, int rows, int width, int unit) {
  if (!m && rows > 0) return api_fail(MOE_ERR_INVALID_ARG, "%s is null", name);
  if (reinterpret_cast<uintptr_t>(m) % 16) return api_fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (ld < width || ld > kMaxStride || ld % unit)
    return api_fail(MOE_ERR_INVALID_ARG, "row stride %lld of %s must be a multiple of %d in [%d, %lld]", (long long)ld,
                    name, unit, width, (long long)kMaxStride);
  return MOE_OK;
}

moe_status check_plain(const char* name, const void* m) {
  if (!m) return api_fail(MOE_ERR_INVALID_ARG, "%s is null", name);
  if (reinterpret_cast<uintptr_t>(m) % 16) return api_fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return MOE_OK;
}

moe_status check_offsets(const moe_product* p, const int32_t* offsets) {
  if (!offsets && p->groups != 1) return api_fail(MOE_ERR_INVALID_ARG, "offsets is null with %d groups", p->groups);
  if (reinterpret_cast<uintptr_t>(offsets) % 4) return api_fail(MOE_ERR_INVALID_ARG, "offsets is not 4-byte aligned");
  return MOE_OK;
}

moe_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MOE_OK;
  if (have < need) return api_fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, the call needs %zu", have, need);
  return check_plain("workspace", ws);
}

moe_status check_launch() {
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return api_fail(MOE_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(err));
  return MOE_OK;
}

#define MOE_TRY(call)                       \
  do {                                      \
    const moe_status st_ = (call);          \
    if (st_ != MOE_OK) return st_;          \
  } while (0)

Num half_num(const moe_product* p) { return p->type == MOE_TYPE_FP16 ? Num::kFp16 : Num::kBf16; }

// The forward product's shape (the operands are filled in by the caller).
ProductArgs forward_args(const moe_product* p, bool codes, bool gated) {
  ProductArgs a;
  a.groups = p->groups;
  a.rows = p->rows;
  a.contract = p->k;
  a.cols = gated ? 2 * p->n : p->n;
  a.ldq = (int64_t)p->k * (codes ? 1 : 2);
  a.q_group = a.cols * a.ldq;
  a.out_type = p->type;
  a.act = p->activation;
  return a;
}
// dx = dy w: wide = rows of w
ProductArgs input_grad_args(const moe_product* p, int wide) {
  ProductArgs a;
  a.groups = p->groups;
  a.rows = p->rows;
  a.contract = wide;
  a.cols = p->k;
  a.ldq = (int64_t)p->k * 2;
  a.q_group = wide * a.ldq;
  a.out_type = p->type;
  return a;
}
ProductArgs weight_grad_args(const moe_product* p, int wide) {
  ProductArgs a;
  a.groups = p->groups;
  a.rows = p->rows;
  a.wrows = wide;
  a.cols = p->k;
  a.ldout = p->k;
  a.out_type = p->type;
  return a;
}

// Result of the forward product of an op
Result forward_result(const moe_product* p, bool gated) {
  return gated ? Result::kGated : p->type == MOE_TYPE_FP32 ? Result::kWide : Result::kHalf;
}

// The gated backward pass's (dg, du), and each group's largest behind them (used in
// fp16; reserved in both types, so that one workspace serves either).
size_t slopes_only_bytes(const moe_product* p) { return align_up((size_t)p->rows * 2 * p->n * 2); }
size_t slopes_bytes(const moe_product* p) {
  return slopes_only_bytes(p) + (p->rows > 0 ? align_up(p->groups * sizeof(uint32_t)) : 0);
}

size_t workspace_bytes_of(const moe_product* p, moe_op op) {
  const bool codes = op == MOE_OP_INT8_PRODUCT || op == MOE_OP_INT8_GATED;
  const Num num = codes ? Num::kInt8 : half_num(p);
  switch (op) {
    case MOE_OP_INT8_PRODUCT:
    case MOE_OP_INT8_GATED:
    case MOE_OP_EXPERT_PRODUCT:
    case MOE_OP_GATED_PRODUCT: {
      const bool gated = op == MOE_OP_INT8_GATED || op == MOE_OP_GATED_PRODUCT;
      return plan_product(num, Pass::kForward, forward_result(p, gated), forward_args(p, codes, gated)).partial_bytes;
    }
    default: {
      // both gradients' parts use the same bytes, one after the other
      const bool gated = op == MOE_OP_GATED_PRODUCT_BACKWARD;
      const int wide = gated ? 2 * p->n : p->n;
      const size_t dx = plan_product(num, Pass::kInputGrad, Result::kHalf, input_grad_args(p, wide)).partial_bytes;
      const size_t dw = plan_product(num, Pass::kWeightGrad, Result::kHalf, weight_grad_args(p, wide)).partial_bytes;
      return std::max(dx, dw) + (gated ? slopes_bytes(p) : 0);
    }
  }
}

void enqueue(ProductArgs& a, const ProductPlan& plan, Num num, Pass pass, Result res, char* partial, hipStream_t s) {
  a.splits = plan.splits;
  a.partial = partial;
  if (plan.family == Family::kStream)
    launch_product_stream(a, num, res, s);
  else if (num == Num::kInt8)
    launch_product_int8(a, plan, res, s);
  else if (pass == Pass::kForward)
    launch_product_half(a, plan, num, res, s);
  else
    launch_product_grad(a, plan, num, pass, res, s);
}

moe_status forward(const moe_product* p, moe_op op, const void* x, int64_t ldx, const float* scale, const void* w,
                   const float* w_scale, const int32_t* offsets, void* out, int64_t ldout, uint16_t* keep,
                   int64_t ldkeep, void* workspace, size_t workspace_bytes, moe_stream stream) {
  MOE_TRY(check_shape(p, op));
  const bool codes = op == MOE_OP_INT8_PRODUCT || op == MOE_OP_INT8_GATED;
  const bool gated = op == MOE_OP_INT8_GATED || op == MOE_OP_GATED_PRODUCT;
  MOE_TRY(check_rows(codes ? "codes" : "x", x, ldx, p->rows, p->k, codes ? 16 : 8));
  MOE_TRY(check_rows(gated ? "h" : "out", out, ldout, p->rows, p->n, 8));
  if (keep) MOE_TRY(check_rows("gate_up", keep, ldkeep, p->rows, 2 * p->n, 8));
  MOE_TRY(check_plain("w", w));
  if (codes) {
    if (p->rows > 0) MOE_TRY(check_plain("scale", scale));
    MOE_TRY(check_plain("w_scale", w_scale));
  }
  MOE_TRY(check_offsets(p, offsets));
  ProductArgs a = forward_args(p, codes, gated);
  const Num num = codes ? Num::kInt8 : half_num(p);
  const Result res = forward_result(p, gated);
  const ProductPlan plan = plan_product(num, Pass::kForward, res, a);
  MOE_TRY(check_workspace(workspace, workspace_bytes, plan.partial_bytes));
  if (p->rows == 0) return MOE_OK;
  a.p = static_cast<const char*>(x);
  a.ldp = ldx * (codes ? 1 : 2);
  a.q = static_cast<const char*>(w);
  a.offsets = offsets;
  a.out = out;
  a.ldout = ldout;
  a.keep = keep;
  a.ldkeep = ldkeep;
  a.pscale = scale;
  a.qscale = w_scale;
  enqueue(a, plan, num, Pass::kForward, res, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
  return check_launch();
}

moe_status check_backward(const moe_product* p, const uint16_t* x, int64_t ldx, const uint16_t* w,
                          const int32_t* offsets, const uint16_t* dx, int64_t lddx, const void* dw, int32_t dw_type) {
  if (dx) {
    MOE_TRY(check_rows("dx", dx, lddx, p->rows, p->k, 8));
    MOE_TRY(check_plain("w", w));
  }
  if (dw) {
    MOE_TRY(check_plain("dw", dw));
    MOE_TRY(check_rows("x", x, ldx, p->rows, p->k, 8));
    if (dw_type != p->type && dw_type != MOE_TYPE_FP32)
      return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "dw_type=%d must be the type of the operands or MOE_TYPE_FP32", dw_type);
  }
  return check_offsets(p, offsets);
}

// dx and dw of a product whose outputs' gradient is dy [rows][wide] (tops: ProductArgs)
moe_status gradients(const moe_product* p, int wide, const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx,
                     const uint16_t* w, const int32_t* offsets, uint16_t* dx, int64_t lddx, void* dw, int32_t dw_type,
                     const uint32_t* tops, char* partial, hipStream_t s) {
  const Num num = half_num(p);
  if (dx && p->rows > 0) {
    ProductArgs a = input_grad_args(p, wide);
    const ProductPlan plan = plan_product(num, Pass::kInputGrad, Result::kHalf, a);
    a.p = reinterpret_cast<const char*>(dy);
    a.ldp = lddy * 2;
    a.q = reinterpret_cast<const char*>(w);
    a.offsets = offsets;
    a.out = dx;
    a.tops = tops;
    a.ldout = lddx;
    enqueue(a, plan, num, Pass::kInputGrad, Result::kHalf, partial, s);
    MOE_TRY(check_launch());
  }
  if (dw) {
    ProductArgs a = weight_grad_args(p, wide);
    const Result res = dw_type == MOE_TYPE_FP32 ? Result::kWide : Result::kHalf;
    const ProductPlan plan = plan_product(num, Pass::kWeightGrad, res, a);
    a.p = reinterpret_cast<const char*>(dy);
    a.ldp = lddy * 2;
    a.q = reinterpret_cast<const char*>(x);
    a.ldq = ldx * 2;
    a.offsets = offsets;
    a.out = dw;
    a.tops = tops;
    enqueue(a, plan, num, Pass::kWeightGrad, res, partial, s);
    MOE_TRY(check_launch());
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_EXPORT moe_status moe_product_workspace(const moe_product* p, moe_op op, size_t* bytes) {
  MOE_TRY(check_shape(p, op));
  if (!bytes) return api_fail(MOE_ERR_INVALID_ARG, "null pointer argument");
  *bytes = workspace_bytes_of(p, op);
  return MOE_OK;
}

MOE_EXPORT moe_status moe_quantize_rows(int32_t rows, int32_t k, int32_t type, const uint16_t* x, int64_t ldx,
                                        int8_t* codes, int64_t ldcodes, float* scale, moe_stream stream) {
  if (rows < 0 || rows > kMaxRows)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "rows=%d outside [0, %d]", rows, kMaxRows);
  if (k < 8 || k > kMaxWidth || k % 8)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "k=%d must be a multiple of 8 in [8, %d]", k, kMaxWidth);
  if (type != MOE_TYPE_BF16 && type != MOE_TYPE_FP16)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "type=%d must be bf16 or fp16", type);
  MOE_TRY(check_rows("x", x, ldx, rows, k, 8));
  MOE_TRY(check_rows("codes", codes, ldcodes, rows, k, 8));
  if (rows == 0) return MOE_OK;
  MOE_TRY(check_plain("scale", scale));
  launch_quantize(rows, k, type, x, ldx, codes, ldcodes, scale, static_cast<hipStream_t>(stream));
  return check_launch();
}

MOE_EXPORT moe_status moe_int8_product(const moe_product* p, const int8_t* codes, int64_t ldcodes, const float* scale,
                                       const int8_t* w, const float* w_scale, const int32_t* offsets, void* out,
                                       int64_t ldout, void* workspace, size_t workspace_bytes, moe_stream stream) {
  return forward(p, MOE_OP_INT8_PRODUCT, codes, ldcodes, scale, w, w_scale, offsets, out, ldout, nullptr, 0, workspace,
                 workspace_bytes, stream);
}

MOE_EXPORT moe_status moe_int8_gated(const moe_product* p, const int8_t* codes, int64_t ldcodes, const float* scale,
                                     const int8_t* w, const float* w_scale, const int32_t* offsets, uint16_t* h,
                                     int64_t ldh, void* workspace, size_t workspace_bytes, moe_stream stream) {
  return forward(p, MOE_OP_INT8_GATED, codes, ldcodes, scale, w, w_scale, offsets, h, ldh, nullptr, 0, workspace,
                 workspace_bytes, stream);
}

MOE_EXPORT moe_status moe_expert_product(const moe_product* p, const uint16_t* x, int64_t ldx, const uint16_t* w,
                                         const int32_t* offsets, uint16_t* out, int64_t ldout, void* workspace,
                                         size_t workspace_bytes, moe_stream stream) {
  return forward(p, MOE_OP_EXPERT_PRODUCT, x, ldx, nullptr, w, nullptr, offsets, out, ldout, nullptr, 0, workspace,
                 workspace_bytes, stream);
}

MOE_EXPORT moe_status moe_gated_product(const moe_product* p, const uint16_t* x, int64_t ldx, const uint16_t* w,
                                        const int32_t* offsets, uint16_t* h, int64_t ldh, uint16_t* gate_up,
                                        int64_t ldgate_up, void* workspace, size_t workspace_bytes, moe_stream stream) {
  return forward(p, MOE_OP_GATED_PRODUCT, x, ldx, nullptr, w, nullptr, offsets, h, ldh, gate_up, ldgate_up, workspace,
                 workspace_bytes, stream);
}

MOE_EXPORT moe_status moe_expert_product_backward(const moe_product* p, const uint16_t* dy, int64_t lddy,
                                                  const uint16_t* x, int64_t ldx, const uint16_t* w,
                                                  const int32_t* offsets, uint16_t* dx, int64_t lddx, void* dw,
                                                  int32_t dw_type, void* workspace, size_t workspace_bytes,
                                                  moe_stream stream) {
  MOE_TRY(check_shape(p, MOE_OP_EXPERT_PRODUCT_BACKWARD));
  MOE_TRY(check_rows("dy", dy, lddy, p->rows, p->n, 8));
  MOE_TRY(check_backward(p, x, ldx, w, offsets, dx, lddx, dw, dw_type));
  MOE_TRY(check_workspace(workspace, workspace_bytes, workspace_bytes_of(p, MOE_OP_EXPERT_PRODUCT_BACKWARD)));
  return gradients(p, p->n, dy, lddy, x, ldx, w, offsets, dx, lddx, dw, dw_type, nullptr,
                   static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
}

MOE_EXPORT moe_status moe_gated_product_backward(const moe_product* p, const uint16_t* dh, int64_t lddh,
                                                 const uint16_t* gate_up, int64_t ldgate_up, const uint16_t* x,
                                                 int64_t ldx, const uint16_t* w, const int32_t* offsets, uint16_t* dx,
                                                 int64_t lddx, void* dw, int32_t dw_type, void* workspace,
                                                 size_t workspace_bytes, moe_stream stream) {
  MOE_TRY(check_shape(p, MOE_OP_GATED_PRODUCT_BACKWARD));
  MOE_TRY(check_rows("dh", dh, lddh, p->rows, p->n, 8));
  MOE_TRY(check_rows("gate_up", gate_up, ldgate_up, p->rows, 2 * p->n, 8));
  MOE_TRY(check_backward(p, x, ldx, w, offsets, dx, lddx, dw, dw_type));
  MOE_TRY(check_workspace(workspace, workspace_bytes, workspace_bytes_of(p, MOE_OP_GATED_PRODUCT_BACKWARD)));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  // (dg, du) first in the workspace, then the groups' largest, then the parts of a split contraction
  uint16_t* dgu = static_cast<uint16_t*>(workspace);
  uint32_t* tops = nullptr;
  if (p->type == MOE_TYPE_FP16 && p->rows > 0)
    tops = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + slopes_only_bytes(p));
  const int wide = 2 * p->n;
  if ((dx || dw) && p->rows > 0) {
    launch_gated_slopes(p->rows, p->n, p->type, p->activation, dh, lddh, gate_up, ldgate_up, offsets, p->groups, dgu,
                        tops, s);
    MOE_TRY(check_launch());
  }
  return gradients(p, wide, dgu, wide, x, ldx, w, offsets, dx, lddx, dw, dw_type, tops,
                   static_cast<char*>(workspace) + slopes_bytes(p), s);
}

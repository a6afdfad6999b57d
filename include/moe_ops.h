/*
 * moe_ops.h -- grouped products of expert feed-forward blocks on MI355X
 * (gfx950), next to the layer of moe.h: the products that the layer runs on
 * int4 / 8-bit codes and 16-bit activations, here with 8-bit codes on both
 * sides (serving) and with 16-bit weights, forward and backward (training).
 *
 * Rows that belong to one expert stand together, as the layer's regroup
 * leaves them: group e owns rows offsets[e] .. offsets[e + 1] - 1 of every
 * row matrix of a call (moe_routing.offsets is such an array), and w[e] is its
 * weight matrix.  Row-major matrices throughout; act is the activation.
 *
 *   quantize_rows    a_r = max_k |x[r,k]|, scale[r] = a_r / 127,
 *                    codes[r,k] = rint(127 x[r,k] / a_r)
 *   int8_product     y[r,n] = scale[r] w_scale[e,n] sum_k codes[r,k] w[e,n,k]
 *   int8_gated       h[r,f] = act(y[r,f]) y[r,F+f], y the int8 product with
 *                    the 2F rows of w[e]
 *   expert_product   y = x w[e]^T
 *     backward       dx = dy w[e],  dw[e] = sum over the group's rows dy^T x
 *   gated_product    (g, u) = x w[e]^T,  h = act(g) u
 *     backward       dg = dh u act'(g), du = dh act(g),
 *                    dx = (dg, du) w[e],  dw[e] = sum over rows (dg, du)^T x
 *
 * Conventions
 *   - Those of moe.h: a moe_status each, the message in moe_last_error(), all
 *     argument checks before anything is enqueued, no device allocation, work
 *     on `stream` only (of the current device), no host synchronisation.
 *   - `ld...` arguments are row strides in elements; they are multiples of 8
 *     (of 16 for the products' codes), at least the row's length and at most
 *     2^20.  Pointers are 16-byte aligned.  Weights, their scales and dw are contiguous.
 *     Outputs overlap no other argument.
 *   - offsets: device int32 [groups + 1], ascending, within 0 .. rows, read
 *     when the kernels run; NULL with one group means all rows.  Rows outside
 *     every group are not read and their outputs are left as they were.
 *     Offsets out of order or out of range give unspecified rows but no
 *     access outside the matrices.
 *   - Sums run over fp32 (16-bit operands) or int32 (codes, exact) and are
 *     rounded once to the output's type.  Codes: (sum * scale) * w_scale, each
 *     product in fp32, so that sum * scale has to stay in its range too.  The same call gives the same bits.
 *   - A workspace needs no initialisation and keeps nothing between calls;
 *     calls that share one (captured graphs among them) must not overlap in
 *     time.  It may be NULL where moe_product_workspace says 0.
 *   - Every call can be captured into a HIP graph.
 */
#ifndef MOE_OPS_H_
#define MOE_OPS_H_

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_type { MOE_TYPE_BF16 = 0, MOE_TYPE_FP16 = 1, MOE_TYPE_FP32 = 2 } moe_type;

typedef enum moe_activation {
  MOE_ACT_SILU = 0,  /* g / (1 + exp(-g)) */
  MOE_ACT_GELU = 1   /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
} moe_activation;

typedef enum moe_op {
  MOE_OP_INT8_PRODUCT = 0,
  MOE_OP_INT8_GATED = 1,
  MOE_OP_EXPERT_PRODUCT = 2,
  MOE_OP_EXPERT_PRODUCT_BACKWARD = 3,
  MOE_OP_GATED_PRODUCT = 4,
  MOE_OP_GATED_PRODUCT_BACKWARD = 5
} moe_op;

/* The shape of one grouped product. */
typedef struct moe_product {
  int32_t rows;        /* R, rows of the row matrices, 0 .. 2^22 */
  int32_t n;           /* output columns (gated: F, the columns of h); multiple of 8, 8 .. 65536
                          (gated 32768) */
  int32_t k;           /* input columns; multiple of 8 (codes: 16), up to 65536 */
  int32_t groups;      /* G, 1 .. 256 */
  int32_t type;        /* moe_type: 16-bit products, of every 16-bit matrix; int8_product, of out
                          (FP32 allowed); int8_gated, of h */
  int32_t activation;  /* moe_activation of the gated ones, else 0 */
} moe_product;

/* Bytes of workspace that a call of `op` with this shape needs (0: none). */
moe_status moe_product_workspace(const moe_product *p, moe_op op, size_t *bytes);

/* Symmetric 8-bit codes of each row: x [rows][k] bf16 or fp16 (`type`), codes
 * [rows][k] in -127 .. 127, scale fp32 [rows].  The rounding is that of the
 * exact quotient, ties to even.  A row of zeros has scale 0; a row with an
 * infinity or NaN has scale NaN and codes 0 (its products are NaN).
 * k is a multiple of 8 in 8 .. 65536 and so is ldcodes (the products take
 * codes in 16s), rows 0 .. 2^22. */
moe_status moe_quantize_rows(int32_t rows, int32_t k, int32_t type, const uint16_t *x, int64_t ldx, int8_t *codes,
                             int64_t ldcodes, float *scale, moe_stream stream);

/* codes [R][k], scale [R], w [G][n][k], w_scale [G][n], out [R][n] of p->type.
 * Codes may be any int8 (-128 too). */
moe_status moe_int8_product(const moe_product *p, const int8_t *codes, int64_t ldcodes, const float *scale,
                            const int8_t *w, const float *w_scale, const int32_t *offsets, void *out, int64_t ldout,
                            void *workspace, size_t workspace_bytes, moe_stream stream);

/* w [G][2n][k] (the n gate rows, then the n up rows), w_scale [G][2n],
 * h [R][n] of p->type (BF16 or FP16). */
moe_status moe_int8_gated(const moe_product *p, const int8_t *codes, int64_t ldcodes, const float *scale,
                          const int8_t *w, const float *w_scale, const int32_t *offsets, uint16_t *h, int64_t ldh,
                          void *workspace, size_t workspace_bytes, moe_stream stream);

/* x [R][k], w [G][n][k], out [R][n]. */
moe_status moe_expert_product(const moe_product *p, const uint16_t *x, int64_t ldx, const uint16_t *w,
                              const int32_t *offsets, uint16_t *out, int64_t ldout, void *workspace,
                              size_t workspace_bytes, moe_stream stream);

/* dy [R][n], x [R][k], w [G][n][k]; dx [R][k] of p->type, dw [G][n][k] of
 * dw_type (p->type, or FP32).  Either of dx and dw may be NULL: it is not
 * computed (x is then not needed without dw, w not without dx).  A group
 * without rows gets dw = 0. */
moe_status moe_expert_product_backward(const moe_product *p, const uint16_t *dy, int64_t lddy, const uint16_t *x,
                                       int64_t ldx, const uint16_t *w, const int32_t *offsets, uint16_t *dx,
                                       int64_t lddx, void *dw, int32_t dw_type, void *workspace,
                                       size_t workspace_bytes, moe_stream stream);

/* x [R][k], w [G][2n][k] (the n gate rows, then the n up rows), h [R][n];
 * gate_up [R][2n] receives (g, u) rounded to p->type for the backward pass,
 * or is NULL.  h comes from g and u before that rounding. */
moe_status moe_gated_product(const moe_product *p, const uint16_t *x, int64_t ldx, const uint16_t *w,
                             const int32_t *offsets, uint16_t *h, int64_t ldh, uint16_t *gate_up, int64_t ldgate_up,
                             void *workspace, size_t workspace_bytes, moe_stream stream);

/* dh [R][n], gate_up [R][2n] from the forward call; the rest as for
 * moe_expert_product_backward with w and dw [G][2n][k].  (dg, du) are rounded
 * to p->type between the two steps.  In fp16 a group with one past 65504 has
 * them divided by a power of two s before, so that the largest is in 2^14 ..
 * 2^15, and the fp32 sums multiplied by s: its smaller ones are then off by up
 * to s 2^-25 beside the rounding, and dx and dw are infinite only where they
 * pass 65504 themselves. */
moe_status moe_gated_product_backward(const moe_product *p, const uint16_t *dh, int64_t lddh,
                                      const uint16_t *gate_up, int64_t ldgate_up, const uint16_t *x, int64_t ldx,
                                      const uint16_t *w, const int32_t *offsets, uint16_t *dx, int64_t lddx, void *dw,
                                      int32_t dw_type, void *workspace, size_t workspace_bytes, moe_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H_ */

/*
 * moe_optim.h -- the optimiser step that turns the gradients of moe_ops.h into
 * new weights, on MI355X (gfx950): AdamW over many tensors in one call.
 *
 *   g' = g grad_scale
 *   m  = beta1 m + (1 - beta1) g'
 *   v  = beta2 v + (1 - beta2) g'^2
 *   p  = p (1 - lr weight_decay)
 *        - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * in fp32.  The states m and v are kept in fp32, or in 8 bits with an fp32
 * scale for each 128 consecutive values: m as e4m3 (its scale is max |m| times
 * the fp32 nearest 1 / 448), v as e5m2 (max v times that nearest 1 / 57344).
 * An 8-bit state rounds to one of its two neighbouring codes at random, up with
 * the probability that keeps its mean, because a step moves v by a thousandth
 * and a code by an eighth: rounded to the nearest, v would stand still.  v above
 * 0 never becomes a code of 0 (it takes the smallest one), so that a step stays
 * bounded, unless its scale is 0 itself: a block whose largest v is below 2^-134.
 * The weights' update comes from m and v before that rounding.
 *
 * The random numbers follow from the seed, the step, the tensor's number in
 * the call and the value's number in the tensor alone, so the same call gives
 * the same bits, and two calls of one step (groups of parameters) draw the same
 * numbers unless each has a seed of its own.  With fold(x, c) = the two 32-bit
 * halves of x c, XORed, and
 * mix(x, key) = fold(fold(x ^ key, 0x9E3779B9) + key, 0xBB67AE85):
 *   key = low(seed); key = mix(y, key) for y = high(seed), step, tensor,
 *   high(value);  draw = mix(low(value), key)
 * m takes the draw's low 16 bits, v its high ones, as fractions of 2^16.
 */
#ifndef MOE_OPTIM_H_
#define MOE_OPTIM_H_

#include "moe_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Numbers of one step.  grad_scale, lr and step may stand on the device: a
 * pointer that is not NULL (one value, read when the kernels run) takes the
 * place of the number, so that a captured step can be replayed with others. */
typedef struct moe_adamw {
  double lr;             /* finite */
  double beta1, beta2;   /* 0 .. 1, 1 excluded */
  double eps;            /* >= 0, finite */
  double weight_decay;   /* finite */
  double grad_scale;     /* 1: gradients as they are */
  uint64_t seed;         /* 8-bit states */
  int32_t step;          /* t, 1 at the first step */
  int32_t state_bits;    /* 32 or 8 */
  const float *device_lr;
  const float *device_grad_scale;
  const int32_t *device_step; /* values below 1 count as 1 */
} moe_adamw;

/* One tensor: contiguous, 16-byte aligned pointers (scales and device numbers
 * 4-byte), 0 to 2^35 values. */
typedef struct moe_adamw_tensor {
  void *param;           /* of param_type, updated in place */
  const void *grad;      /* of grad_type */
  float *master;         /* the weights in fp32, updated in place; param then is only
                            written, as their rounding.  Or NULL. */
  void *m, *v;           /* fp32, or codes */
  float *m_scale, *v_scale; /* 8 bits: ceil(count / 128) each, else NULL */
  int64_t count;
  int32_t param_type;    /* moe_type; FP32 takes no master */
  int32_t grad_type;     /* param_type or FP32 */
} moe_adamw_tensor;

/* Enqueues the step of tensors[0 .. count).  Without a master a 16-bit param
 * is rounded to nearest.  States, weights and their scales may not overlap
 * each other, within a tensor or across.  An infinity or NaN in a gradient
 * makes NaN of the 8-bit states of its block of 128; the scale is then NaN
 * and the codes 0. */
moe_status moe_adamw_step(const moe_adamw *numbers, int32_t count, const moe_adamw_tensor *tensors,
                          moe_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPTIM_H_ */

/*
 * bi_optim.h -- C ABI of the update of the policy model's weights: one AdamW step over many tensors
 * in one launch.  Same library (libbi_isloss.so), status codes and conventions as bi_isloss.h.
 *
 * Source: "Zero Mismatch, Simple Async RL", section "Alignment permits a simpler learning path":
 * each update of the learner ends in an optimizer step on the gradients that bi_is_loss_fwd_bwd and
 * the layers' backward passes give.  The pages name no optimizer; this is AdamW (decoupled weight
 * decay) with bias correction.
 *
 * For each element, in fp32 with every operation rounded (no contraction), and t = step:
 *   g' = g * grad_scale                       (the product only where grad_scale is given)
 *   m  = beta1 m + (1 - beta1) g'
 *   v  = beta2 v + (1 - beta2) g'^2
 *   p  = p (1 - lr wd) - (m lr / (1 - beta1^t)) / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * The factors in parentheses of the hyper-parameters are computed in fp64 and rounded once.  Every
 * element depends on its own inputs alone (with 8-bit states, on its block's): no reduction crosses
 * tensors, so an update's bits do not depend on which tensors share a call.
 */
#ifndef BI_OPTIM_H
#define BI_OPTIM_H

#include "bi_isloss.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One tensor of n elements.  Device pointers; elements are contiguous, at their types' alignment. */
typedef struct bi_adamw_tensor {
  void* param;          /* updated: float (param_bf16 = 0) or bf16 bits (param_bf16 = 1) */
  float* master;        /* fp32 weights that are updated and of which a bf16 param is the rounded copy; or NULL */
  const void* grad;     /* float (grad_bf16 = 0) or bf16 bits (grad_bf16 = 1) */
  void* exp_avg;        /* m, updated: float, or float8 e4m3 codes with state_bits = 8 */
  void* exp_avg_sq;     /* v, updated: float, or with state_bits = 8 the float8 e4m3 codes of sqrt(v) */
  float* exp_avg_scale;    /* state_bits = 8: one scale for each block of 256 elements (ceil(n / 256)); else NULL */
  float* exp_avg_sq_scale; /* the same for sqrt(v) */
  int64_t n;            /* 0 <= n <= 2^40 */
} bi_adamw_tensor;

/*
 * 8-bit states: a block of 256 consecutive elements (the last one may be short) holds x as
 * code * scale with scale = max|x| * fl(1 / 448) (448 = the largest e4m3 value) and the code
 * y = x * (448 * fl(1 / max|x|)) rounded as below; x is m for exp_avg and sqrt(v) for exp_avg_sq, whose
 * root halves the range of exponents.  Where 448 * fl(1 / max|x|) is not finite (a maximum below 1.3e-36)
 * the block is held as zeros with scale 0.  A sqrt(v) above zero never becomes the code of zero (it takes the
 * smallest one, 2^-9): a zero there would turn a small gradient into an unbounded update.  max is taken of the
 * finite elements; one that is not finite is held as NaN, and the other elements of its block are what they would
 * be without it.
 * Rounding: m to nearest even for beta1 <= 17/18, sqrt(v) for beta2 <= 0.96.  Above, nearest would give most
 * elements their old code back at every step; y goes to the code below or above it in magnitude, spaced q, as
 * q * floor(|y| / q + r / 65536) in fp32, so that the held value is right on average (sqrt(v) scatters by about 20%
 * around it).  r is a number of 16 bits made of the element's index in its tensor and of t alone (kernels_adamw.cuh:
 * adam_bits; the low half for m, the high half for sqrt(v)): the same call gives the same bits.
 */
typedef struct bi_adamw_cfg {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;       /* t >= 1 of this update; ignored where step_dev is given */
  int32_t state_bits; /* 32 or 8 */
  int32_t param_bf16; /* type of every param: 1 bf16, 0 float */
  int32_t grad_bf16;  /* type of every grad */
  int32_t reserved;   /* 0 */
} bi_adamw_cfg;

/*
 * One step over `count` tensors (a host array, read before the call returns).
 *   grad_scale  device float[1] that multiplies every gradient (unscaling, clipping), or NULL
 *   step_dev    device int64[1] holding t, read when the kernel runs (a captured call can then be
 *               replayed for other steps), or NULL.  A t below 1 raises BI_ERR_INVALID_ARG in
 *               *dev_status and leaves the tensors as they were.
 * count = 0 and tensors of no elements are fine.  All tensors have a master or none has; a master
 * needs param_bf16 = 1.  Tensors of one call may not overlap (gradients may overlap each other).
 * Returns BI_ERR_INVALID_ARG for a NULL or misaligned pointer, masters given for some tensors only,
 * a step below 1, lr, eps or weight_decay below 0 or not finite, or a beta outside [0, 1).
 */
BI_API bi_status bi_adamw_step(const bi_adamw_tensor* tensors, int32_t count, const bi_adamw_cfg* cfg,
                               const float* grad_scale, const int64_t* step_dev, int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BI_OPTIM_H */

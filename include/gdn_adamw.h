/*
 * gdn_adamw.h -- one AdamW step over many tensors (libgdn.so): what the
 * gradients of the training entry points (gdn_train.h, gdn_linrec.h) go into.
 *
 * Conventions as in gdn.h and gdn_train.h: device pointers owned by the caller,
 * no allocation and no synchronisation, work enqueued on `stream`, host-side
 * validation that launches nothing on a refusal, kernels only (so that calls
 * can be captured into a HIP graph), the same bits run to run.
 */
#ifndef GDN_ADAMW_H
#define GDN_ADAMW_H

#include "gdn_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Consecutive values of a tensor that share one scale of an 8-bit state. */
#define GDN_ADAMW_GROUP 128

/* One tensor of n values.  The array of these is HOST memory, read before the
 * call returns; the pointers in it are device pointers. */
typedef struct gdn_adamw_tensor {
    void* w;              /* weights, updated in place: w_dtype */
    float* master;        /* with BF16 weights: the fp32 weights that are updated, w becoming
                             their rounding; or NULL, w is updated itself */
    const void* g;        /* gradients: g_dtype */
    void* m;              /* first moment: fp32, or with GDN_E4M3 states codes */
    void* v;              /* fp32: second moment; GDN_E4M3: codes of its square root */
    float* m_scale;       /* GDN_E4M3: fp32 [ceil(n / 128)], else NULL */
    float* v_scale;
    int64_t n;            /* >= 0 (0: nothing is done) */
    float weight_decay;   /* >= 0, finite */
    int32_t reserved;     /* 0 */
} gdn_adamw_tensor;

/* With f the gradient factor, t = step:
 *   g' = f g,  m <- beta1 m + (1 - beta1) g',  v <- beta2 v + (1 - beta2) g'^2,
 *   w <- (1 - lr weight_decay) w - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in fp32, each operation rounded by itself (no fused multiply-add), so that the
 * result is that of the same operations one by one; with GDN_E4M3 states the
 * quotient m / (...) is a division's save for one in a million, which rounds to the
 * float next to it, and for BF16 weights without master, which are rounded to 2^-9
 * at once, within 2^-22 of itself.
 *
 * state_dtype GDN_F32: m and v are kept as they are.  GDN_E4M3: the first moment
 * and the root of the second are each kept as e4m3 codes with one fp32 scale per
 * 128 values, the group's largest finite magnitude times fp32's 1 / 448 (0 where all
 * are zero, else at least 2^-126); a value is code * scale.  The root and not v, whose
 * range is the square of the root's; a root above zero has a code above zero, so
 * that no m is divided by a root that was lost.  Infinities and NaN become a
 * NaN code.  The update itself uses m and v before they are rounded.
 *
 * Rounding to 8 bits, and of BF16 weights without master, is to nearest even,
 * or with stochastic != 0 up with the probability that the part cut off has, by
 * 16 of the 32 bits that a hash of (seed, the tensor's place in the call, the
 * value's place in the tensor) gives, the lower ones for m, the upper ones for the
 * root; BF16 weights take the lower 16 of a second hash of those bits.  An average
 * that moves by 1 / 1000 a step never leaves an 8-bit value that it is rounded to
 * each time, and a BF16 weight loses every update below 2^-9 of it.  Give another
 * seed each step.  (GDN_E4M3 states with F32 weights: the weights are not rounded.)
 *
 * control: NULL, or device memory of 5 words, read by the kernels in place of
 * the arguments (for captured graphs): fp32 lr, 1 - beta1^t, 1 - beta2^t, the
 * gradient factor, and the seed's 32 bits.  lr, step, grad_factor and seed are
 * then not used.  Where its factor is not above zero and finite nothing is
 * changed: the step of gradients that overflowed is skipped on the device.
 *
 * With eps 0 a value that never had a gradient becomes NaN (0 / 0).
 * Any alignment of the element types; tensors must not overlap.  count >= 0
 * tensors; up to 64 (8-bit states: 48) of them go into one launch.
 * Limits: n <= 2^40, step >= 1, 0 <= beta < 1, eps >= 0 (with GDN_E4M3 states 0 or
 * at least 2^-126); eps, lr, grad_factor, lr / (1 - beta1^step) and each
 * 1 - lr weight_decay finite in fp32 (of a control's words nothing is checked).
 * Returns GDN_OK, GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE or GDN_ERR_HIP.
 */
int gdn_adamw_step(const gdn_adamw_tensor* tensors, int count, double lr, double beta1, double beta2,
                   double eps, int64_t step, double grad_factor, const float* control, int w_dtype,
                   int g_dtype, int state_dtype, int stochastic, uint32_t seed, hipStream_t stream);
int gdn_adamw_step_plan(const gdn_adamw_tensor* tensors, int count, double lr, double beta1, double beta2,
                        double eps, int64_t step, double grad_factor, const float* control, int w_dtype,
                        int g_dtype, int state_dtype, int stochastic, uint32_t seed);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ADAMW_H */

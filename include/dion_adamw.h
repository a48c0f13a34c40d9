/*
 * dion_adamw.h -- what steps beside the orthonormalized update: AdamW over
 * many tensors in one call, for the parameters that are no matrices of a
 * megabatch (embeddings, output heads, norm weights, biases), and the norm of
 * many gradients, whose clipping factor the step reads on the device.
 * ("microsoft/dion" repository summary: foreach AdamW, in-place multi-tensor
 * updates, capturable.)
 *
 * The conventions of dion.h hold (caller-owned device memory, no allocation,
 * no synchronization, host-side argument checks before any launch), except
 * that tensors are flat and may have any alignment that their type has.  A
 * list of tensors is an array in HOST memory, read before the call returns;
 * its pointers are device pointers.  Tensors that a call writes overlap no
 * other tensor of the list.
 */
#ifndef DION_ADAMW_H
#define DION_ADAMW_H

#include "dion.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Values of an 8-bit state that share a scale. */
#define DION_ADAMW_BLOCK 256

/*
 * One tensor of a list: n values (n = 0: skipped).
 *   p, g      parameter (type p_type) and gradient (type g_type)
 *   m, v      float32 states [n]; or, with m_scale and v_scale, 8-bit ones
 *   m_scale, v_scale  float32 [ceil(n / 256)] (both or neither)
 *   copy      bfloat16 [n] or NULL: the new p, rounded (p_type float32 only)
 *   lr_factor, decay_factor   this tensor's learning rate is lr * lr_factor,
 *             its weight decay weight_decay * decay_factor
 *
 * 8-bit states: blocks of 256 values, the last one short.  m holds E4M3 values
 * that stand for value * scale, scale = max(amax / 448, 2^-100); v holds
 * r = sqrt(second moment) in the same format.
 * r is rounded up with the probability of its place between two values, by a
 * hash of seed, step, the tensor's place in the list and the value's place in
 * the tensor (with beta2 = 0.999 a step changes r by less than half the
 * distance of two values, so rounding to nearest would never let it fall), and
 * an r above zero does not become zero.
 * m is rounded to nearest even where that holds no value in its place: with
 * 1 - beta1 >= 3/32, except values that nearest rounding takes below 2^-6 (of the
 * scale) while the gradient's part, (1 - beta1) g', is at most 2^-9.  Those, and
 * with a smaller 1 - beta1 all values, are rounded by the same hash, the magnitude
 * up with the probability of its place, so that an m whose gradient has stopped
 * reaches zero and its parameter comes to rest.
 * Infinities and NaN become the format's NaN and do not count for amax.
 *
 * What 8 bits cost, with Gaussian gradients: a held r has a standard deviation of
 * 16.5 % of its value with beta2 = 0.999 (1 % to 99 % of them: 0.71 to 1.43 of it),
 * 15.6 % with 0.99, 12 % with 0.95, since each step's rounding stays in it for
 * 1 / (1 - beta2) steps; r is without bias a step, but its square, which the next
 * step takes, is not: second moments are 5.4, 4.6 and 3.3 % too large in the mean.
 * An m that is rounded to nearest, under a gradient that does not change at all,
 * stays between a half and three times of it; a gradient's noise does what the
 * dither would.
 */
typedef struct {
    long long n;
    void* p;
    const void* g;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    void* copy;
    dion_dtype p_type, g_type;
    float lr_factor, decay_factor;
} dion_adamw_tensor;

/*
 * One AdamW step (t = step >= 1), all in float32:
 *   g' = f g                         f = *grad_scale (device; NULL: 1)
 *   m <- beta1 m + (1 - beta1) g'    v <- beta2 v + (1 - beta2) g'^2
 *   p <- (1 - lr wd) p - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * p is rounded once to its type (float32: p + (u - lr wd p), u the update, so that
 * a decay below 2^-24 counts, too); 8-bit states are rounded after p has used them.
 * An eps between zero and 2^-126 counts as 2^-126.
 * A factor f that is NaN skips the step: nothing is written.
 */
dion_status dion_adamw_step(int count, const dion_adamw_tensor* tensors, double lr, double beta1, double beta2,
                            double eps, double weight_decay, long long step, unsigned int seed,
                            const float* grad_scale, void* cuda_stream);

/*
 * The same with hyper = (lr, beta1, beta2, eps, weight_decay), five float64,
 * and the number of steps taken so far read on the device when the step runs,
 * so that a captured step follows what the caller writes there.  *step is
 * counted up first (unless the step is skipped); t is the new value.
 * workspace: 256 bytes, 16-byte aligned, scratch.
 */
dion_status dion_adamw_step_dev(int count, const dion_adamw_tensor* tensors, const double* hyper, long long* step,
                                unsigned int seed, const float* grad_scale, void* workspace, size_t workspace_bytes,
                                void* cuda_stream);

/* Workspace bytes of dion_grad_norm for a list of `count` tensors. */
dion_status dion_grad_norm_workspace_size(int count, size_t* bytes);

/*
 * out[0] = sqrt(sum of g^2 over all tensors), out[1] = min(1, max_norm /
 * (out[0] + 1e-6)), or NaN where the norm is not finite (dion_adamw_step then
 * skips).  Of the list, n, g and g_type are read.  Squares are float32 (a
 * gradient beyond 1.8e19 makes the norm infinite; below 2^-63 = 1.1e-19 a square is
 * off by up to 2^-150, and from 2^-75 = 2.6e-23 down it is nothing), their sums
 * float64 from a few hundred values on, in a fixed order (the same bits every time).
 * max_norm > 0 may be infinite.  workspace: 8-byte aligned; none is used, and
 * it may be NULL, for up to 256 tensors of 2^20 values in all, each counted up to
 * a multiple of 2048.
 */
dion_status dion_grad_norm(int count, const dion_adamw_tensor* tensors, double max_norm, float* out, void* workspace,
                           size_t workspace_bytes, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* DION_ADAMW_H */

/*
 * ssm_norm.h -- C ABI of the grouped norm with an activation on
 * (batch, L, dim) tensors, and of its gradients (gfx950).
 *
 * The channels of each step are cut into `groups` groups of n = dim / groups;
 * each (batch, step, group) is normalised by itself (time is not pooled: a
 * step of a causal model does not see later ones):
 *     m = mean(x)            (0 with SSM_NORM_RMS)
 *     a = (x - m) / sqrt(mean((x - m)^2) + eps) * weight + bias
 *     y = a                  by default
 *       = silu(a)            with SSM_NORM_SILU
 *       = a * silu(z)        when z is given
 * With SSM_NORM_GATE_FIRST (z required) x * silu(z) takes the place of x and
 * y = a.  groups = 1 is a layer (or RMS) norm over the whole step; groups =
 * heads is the norm that follows a multi-head scan.
 *
 * Conventions are those of ssm.h: caller-owned device pointers; nothing is
 * allocated or retained; argument errors return a status before anything is
 * enqueued (nothing is written); a failed launch returns SSM_ERR_HIP; calls
 * are asynchronous on `stream` (NULL = default).  Statistics and arithmetic
 * are fp32.  Every pointer must be aligned to its element size.  eps is a HOST
 * pointer, read during the call only; NULL means 1e-5.
 * Supported sizes: batch, seqlen, dim, groups >= 1, groups a divisor of dim,
 * dim <= 2^24, batch * seqlen < 2^31.
 */
#ifndef SSM_NORM_H
#define SSM_NORM_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_NORM_RMS 0x1u        /* no mean subtracted                          */
#define SSM_NORM_SILU 0x2u       /* y = silu(a); excludes z                     */
#define SSM_NORM_GATE_FIRST 0x4u /* normalise x * silu(z); requires z           */

/*
 * Element strides: element (b, t, c) at b * batch + t * step + c.  0 means
 * dense (step dim, batch seqlen * step); otherwise step >= dim and batch >=
 * seqlen * step.  Index order: x, z, y (forward); x, z, dy, dx, dz (gradients).
 * A NULL layout means all zero.  Overlap is checked on address ranges, except
 * that tensors with the same strides may lie beside each other in every step
 * (dx and dz as parts of one buffer).
 */
typedef struct {
    long long step[3], batch[3];
} ssm_norm_layout_t;
typedef struct {
    long long step[5], batch[5];
} ssm_norm_bwd_layout_t;

/*
 *   x, z     [batch][seqlen][dim] in_dtype; z or NULL (no gate)
 *   weight, bias  [dim] fp32, each or NULL (1, 0)
 *   y        [batch][seqlen][dim] out_dtype; may be exactly x or exactly z
 *            where type and strides agree, otherwise overlapping no input
 */
ssm_status_t ssm_group_norm_fwd(int batch, int seqlen, int dim, int groups, ssm_dtype_t in_dtype,
                                unsigned flags, const float *eps, const void *x, const float *weight,
                                const float *bias, const void *z, ssm_dtype_t out_dtype, void *y,
                                const ssm_norm_layout_t *layout, void *stream);

/* Device workspace of ssm_group_norm_bwd, in bytes (0 for sizes it refuses). */
size_t ssm_group_norm_bwd_workspace_bytes(int batch, int seqlen, int dim, int groups);

/*
 * Gradients for l = sum dy . y; the statistics are formed again from x.
 *   dy, dx, dz      grad_dtype; dz NULL exactly when z is NULL
 *   dweight, dbias  [dim] fp32 sums over batch and steps, each or NULL (not
 *                   wanted; allowed whether or not weight, bias are given)
 *   workspace       16-byte aligned, overlapping no input or output; may be
 *                   NULL when neither dweight nor dbias is wanted
 * Outputs overlap no input and no other output.  The sums are taken in a
 * fixed order.
 */
ssm_status_t ssm_group_norm_bwd(int batch, int seqlen, int dim, int groups, ssm_dtype_t in_dtype,
                                unsigned flags, const float *eps, const void *x, const float *weight,
                                const float *bias, const void *z, ssm_dtype_t grad_dtype,
                                const void *dy, void *dx, void *dz, float *dweight, float *dbias,
                                void *workspace, size_t workspace_bytes,
                                const ssm_norm_bwd_layout_t *layout, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_NORM_H */

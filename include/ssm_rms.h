/*
 * ssm_rms.h -- C ABI of the root-mean-square norm with the residual's addition
 * in front of it, on (batch, L, dim) tensors, and of its gradients (gfx950).
 *
 * A layer's entrance: the last layer's output x joins the residual stream, and
 * the new stream is normalised over its channels:
 *     h = x + residual
 *     y = h / sqrt(mean(h^2) + eps) * weight
 * With out_dtype SSM_E4M3 y is held in 8 bits with a scale for every block of
 * 128 channels of a step (the last block may be shorter), for a product that
 * takes such operands:
 *     scale = max(max |y| / 448, 2^-126),  q = y / scale rounded to e4m3
 * (finite range +-448, nearest, ties to even); y is about q * scale.  A block
 * that holds an infinity has an infinite scale, one that holds a NaN a NaN.
 *
 * Conventions are those of ssm.h: caller-owned device pointers; nothing is
 * allocated or retained; argument errors return a status before anything is
 * enqueued (nothing is written); a failed launch returns SSM_ERR_HIP; calls
 * are asynchronous on `stream` (NULL = default).  Sums and arithmetic are
 * fp32; y is formed from h before h is rounded to the stream's type.  Every
 * pointer must be aligned to its element size.  eps is a HOST pointer, read
 * during the call only; NULL means 1e-5.
 * Supported sizes: batch, seqlen, dim >= 1, dim <= 2^24, batch * seqlen < 2^31.
 */
#ifndef SSM_RMS_H
#define SSM_RMS_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_RMS_BLOCK 128 /* channels that share a scale */

/*
 * Element strides: element (b, t, c) at b * batch + t * step + c.  0 means
 * dense (step dim, batch seqlen * step); otherwise step >= dim and batch >=
 * seqlen * step.  Index order: x, residual, residual_out, y (forward); h, dy,
 * dh, dx, dresidual (gradients).  The scale of block k of step (b, t) is at
 * b * scale_batch + t * scale_step + k * scale_block: 0 means 1 for
 * scale_block, ceil(dim / 128) for scale_step and seqlen * scale_step for
 * scale_batch; any strides for which no two scales share a place are taken
 * (a transposed array: scale_step 1, scale_block batch * seqlen).  A NULL
 * layout means all zero.  Overlap is checked on address ranges, except that
 * tensors with the same strides may lie beside each other in every step.
 */
typedef struct {
    long long step[4], batch[4];
    long long scale_step, scale_batch, scale_block;
} ssm_rms_layout_t;
typedef struct {
    long long step[5], batch[5];
} ssm_rms_bwd_layout_t;

/*
 *   x             [batch][seqlen][dim] in_dtype
 *   residual      the same in stream_dtype, or NULL (h = x)
 *   weight        [dim] fp32, or NULL (1)
 *   residual_out  h in stream_dtype, or NULL (not returned); may be exactly
 *                 residual, or exactly x where type and strides agree
 *   y             out_dtype (SSM_F32, SSM_BF16 or SSM_E4M3); may be exactly x
 *                 or exactly residual where type and strides agree
 *   scales        fp32, with SSM_E4M3 only (NULL otherwise)
 * Otherwise no output overlaps an input or the other outputs.
 */
ssm_status_t ssm_rms_norm_fwd(int batch, int seqlen, int dim, ssm_dtype_t in_dtype,
                              ssm_dtype_t stream_dtype, const float *eps, const void *x,
                              const void *residual, const float *weight, void *residual_out,
                              ssm_dtype_t out_dtype, void *y, float *scales,
                              const ssm_rms_layout_t *layout, void *stream);

/* Device workspace of ssm_rms_norm_bwd, in bytes (0 for sizes it refuses). */
size_t ssm_rms_norm_bwd_workspace_bytes(int batch, int seqlen, int dim);

/*
 * Gradients for l = sum dy . y + sum dh . h.  The gradient of h is that of x
 * and of the residual alike; it is returned in either type, or in both.
 *   h          [batch][seqlen][dim] stream_dtype: the forward's residual_out (or
 *              its x, where there was no residual)
 *   dy, dx     grad_dtype
 *   dh         stream_dtype: what comes down the residual stream, or NULL
 *   dx, dresidual  grad_dtype, stream_dtype; one of them may be NULL.  dx may be
 *              exactly dy, dresidual exactly dh, where the strides agree
 *   dweight    [dim] fp32, summed over batch and steps in a fixed order, or NULL
 *   workspace  16-byte aligned, overlapping no input or output; may be NULL
 *              when dweight is not wanted
 * Otherwise no output overlaps an input or another output.
 */
ssm_status_t ssm_rms_norm_bwd(int batch, int seqlen, int dim, ssm_dtype_t stream_dtype,
                              ssm_dtype_t grad_dtype, const float *eps, const void *h,
                              const float *weight, const void *dy, const void *dh, void *dx,
                              void *dresidual, float *dweight, void *workspace,
                              size_t workspace_bytes, const ssm_rms_bwd_layout_t *layout,
                              void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_RMS_H */

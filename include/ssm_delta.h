/*
 * ssm_delta.h -- C ABI of the gated delta rule (gfx950): a recurrence whose
 * state is a matrix per head, over whole sequences, its gradients, and its
 * single-token decode step.
 *
 * Per sequence and value head, with a key and a query of K entries, a value
 * of V entries, a log decay g and a writing strength beta at every step:
 *     S_t = e^{g_t} S_{t-1} + beta_t k_t (v_t - e^{g_t} S_{t-1}^T k_t)^T
 *     y_t = scale S_t^T q_t            (read after the step-t update)
 * The state S is K x V.  With |k_t| = 1 and beta_t = 1 the step replaces what
 * the state answers to k_t by v_t; keys are used as given (normalise them
 * first, e.g. with ssm_group_norm_fwd over the heads' channels).
 *
 * Conventions are those of ssm.h: caller-owned device pointers; nothing is
 * allocated or retained; argument errors return a status before anything is
 * enqueued (nothing is written); a failed launch returns SSM_ERR_HIP; calls
 * are asynchronous on `stream` (NULL = default).
 *   - Layouts (dense; see the layout structs for views):
 *       q, k     [batch][seqlen][qk_heads][K]   in_dtype
 *       v, y     [batch][seqlen][heads][V]      in_dtype, out_dtype
 *       g, beta  [batch][seqlen][heads]         fp32
 *       h0, hL   [sequences][heads][K][V]       fp32
 *     heads is a multiple of qk_heads: value head h reads query and key head
 *     h / (heads / qk_heads).
 *   - scale is a HOST pointer, read during the call only; NULL means K^(-1/2).
 *   - Packed sequences: cu_seqlens is NULL (each batch row is one sequence),
 *     or a DEVICE array of num_seqs + 1 ints with batch = 1: sequence i is
 *     steps [cu_seqlens[i], cu_seqlens[i+1]) of the row.  cu_seqlens[0] is 0,
 *     entries do not decrease and the last is seqlen.  The array is read on
 *     the device only; entries outside [0, seqlen] or decreasing are clamped
 *     (nothing outside the tensors is touched), and steps that no sequence
 *     covers keep what the outputs held.  A sequence may be empty: its hL is
 *     its h0 (or zero).
 *   - Arithmetic: products run on the matrix cores with every operand that
 *     is not exact in bf16 split into bf16 terms, sums and the running state are
 *     fp32.  bf16 inputs: two terms (16 bits of significand); a bf16 y or gradient
 *     does not show it, fp32 outputs have relative errors of about 4e-6.  fp32
 *     inputs: three terms (24 bits), errors of fp32 arithmetic; a caller who wants
 *     those of bf16 values passes them as fp32 (y and the gradients may still be
 *     bf16).  The decode step computes in fp32 throughout.
 *   - g is a log decay: a real number or -inf (the state is cleared); below -110
 *     it acts as -110 (e^-110 is 0 in fp32).  Where g grows instead of decaying,
 *     its sums over neighbouring steps of a 64-step chunk have to stay below 88
 *     (e^88 is the largest power that fp32 holds).
 *   - A non-finite q, k, v or beta reaches the outputs of its own head and
 *     sequence from the start of its 64-step chunk on (steps are combined a
 *     chunk at a time); other sequences and heads are not touched by it.
 *   - Every pointer must be aligned to its element size; the decode `state`
 *     must be 16-byte aligned.
 * Supported sizes: batch, num_seqs and heads <= 65535, qk_heads a divisor of
 * heads, 1 <= K <= 256, 1 <= V <= 65536, 1 <= seqlen <= 2^28 - 4096.
 */
#ifndef SSM_DELTA_H
#define SSM_DELTA_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Element strides: element (b, t, h, i) of a tensor at
 * b * batch + t * step + h * head + i; the last index is contiguous (g and
 * beta: no last index).  0 means the dense default of that index given the
 * other strides' defaults: head K, V or 1, step heads * head, batch
 * seqlen * step.  Any order of the three is accepted ([batch][heads][seqlen]
 * tensors, slices of one projection's output); a negative stride, strides for
 * which two elements of the tensor would share a place, or a tensor spanning
 * 2^56 elements or more is SSM_ERR_BAD_SHAPE.
 * Overlap is checked on address ranges, except that tensors with the same
 * step and batch strides may lie beside each other in every step (q, k and v,
 * or dq, dk and dv, as slices of one projection's buffer; the larger of the
 * two strides is then a multiple of the smaller).
 * Index order: q, k, v, y, g, beta.  A NULL layout means all zero.
 */
typedef struct {
    long long step[6], head[6], batch[6];
} ssm_delta_layout_t;

/* Index order: q, k, v, g, beta, dy, dq, dk, dv. */
typedef struct {
    long long step[9], head[9], batch[9];
} ssm_delta_bwd_layout_t;

/* Device workspace ssm_delta_fwd needs, in bytes (0 for sizes it refuses).
 * num_seqs is the number of packed sequences, 0 when cu_seqlens is NULL.
 * A function of the sizes only. */
size_t ssm_delta_fwd_workspace_bytes(int batch, int seqlen, int qk_heads, int heads, int K, int V,
                                     int num_seqs);

/* Device workspace of ssm_delta_bwd, and of ssm_delta_fwd with
 * SSM_FLAG_CHECKPOINTS. */
size_t ssm_delta_bwd_workspace_bytes(int batch, int seqlen, int qk_heads, int heads, int K, int V,
                                     int num_seqs);

/*
 * The gated delta rule over whole sequences.
 *   flags   0 or SSM_FLAG_CHECKPOINTS: the state entering every 64-step chunk
 *           and what else the backward pass reads are left in `workspace`,
 *           which then has ssm_delta_bwd_workspace_bytes(...) bytes; y and hL
 *           are unchanged bit for bit
 *   h0      [sequences][heads][K][V] or NULL (zero)
 *   y       must not overlap any input
 *   hL      final states, or NULL (not returned); may be exactly h0, must not
 *           otherwise overlap an input or y
 *   layout  host pointer, read during the call only; NULL means dense
 *   workspace  16-byte aligned, overlapping no input or output
 */
ssm_status_t ssm_delta_fwd(int batch, int seqlen, int qk_heads, int heads, int K, int V,
                           ssm_dtype_t in_dtype, unsigned flags, const float *scale, const void *q,
                           const void *k, const void *v, const float *g, const float *beta,
                           const float *h0, const int *cu_seqlens, int num_seqs,
                           ssm_dtype_t out_dtype, void *y, float *hL, void *workspace,
                           size_t workspace_bytes, const ssm_delta_layout_t *layout, void *stream);

/*
 * Gradients of l = sum dy . y + sum dhL . hL for every input of
 * ssm_delta_fwd (scale is a constant).  dq and dk sum over the value heads
 * that share them.
 *   dy, dq, dk, dv   grad_dtype, laid out by `layout` (dq, dk as q, k)
 *   dhL, dh0         [sequences][heads][K][V] fp32, each may be NULL; dh0 may be
 *                    exactly dhL
 *   dg, dbeta        [batch][seqlen][heads] fp32, dense
 *   flags            with SSM_FLAG_CHECKPOINTS the workspace is one that
 *                    ssm_delta_fwd filled with that flag for the same inputs
 *                    (read, and used as scratch); without it the forward
 *                    recurrence is run here first
 * Outputs must not overlap any input or one another.  Results do not depend
 * on timing: nothing is summed with atomics.
 */
ssm_status_t ssm_delta_bwd(int batch, int seqlen, int qk_heads, int heads, int K, int V,
                           ssm_dtype_t in_dtype, unsigned flags, const float *scale, const void *q,
                           const void *k, const void *v, const float *g, const float *beta,
                           const float *h0, const int *cu_seqlens, int num_seqs,
                           ssm_dtype_t grad_dtype, const void *dy, const float *dhL, void *dq,
                           void *dk, void *dv, float *dg, float *dbeta, float *dh0,
                           void *workspace, size_t workspace_bytes,
                           const ssm_delta_bwd_layout_t *layout, void *stream);

/*
 * One decode step: the same recurrence for one token per batch row on
 * persistent states, updated in place.
 *   state   [num_slots][heads][K][V] fp32, 16-byte aligned
 *   q, k    [batch][qk_heads][K];  v, y [batch][heads][V];  g, beta [batch][heads]
 *   slots   DEVICE array of batch ints: the state of each row, or NULL (row b
 *           uses state b; num_slots is then batch).  A row whose slot is
 *           negative or not below num_slots is skipped: no state changes and
 *           its y is zero.  Two rows must not name the same slot.
 *   layout  as above; the step strides are not used
 */
ssm_status_t ssm_delta_update(int batch, int qk_heads, int heads, int K, int V,
                              ssm_dtype_t in_dtype, const float *scale, float *state, int num_slots,
                              const int *slots, const void *q, const void *k, const void *v,
                              const float *g, const float *beta, ssm_dtype_t out_dtype, void *y,
                              const ssm_delta_layout_t *layout, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_DELTA_H */

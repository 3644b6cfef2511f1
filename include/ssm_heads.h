/*
 * ssm_heads.h -- C ABI of the selective scan with one decay a head (gfx950):
 * the recurrence of ssm.h for heads whose state is a matrix, over whole
 * sequences, its gradients, and its single-token decode step.
 *
 * Per sequence and head, with an input B and a readout C of N entries, a value
 * x of P entries and a raw step size dt at every step:
 *     D_t = softplus(dt_t + dt_bias)
 *     S_t = e^{D_t A} S_{t-1} + D_t B_t x_t^T
 *     y_t = S_t^T C_t + Dskip x_t      (read after the step-t update)
 * The state S is N x P.  A, dt_bias and Dskip are numbers of the head; a gate
 * y silu(z) is ssm_group_norm_fwd's.
 *
 * Conventions are those of ssm.h: caller-owned device pointers; nothing is
 * allocated or retained; argument errors return a status before anything is
 * enqueued (nothing is written); a failed launch returns SSM_ERR_HIP; calls
 * are asynchronous on `stream` (NULL = default).
 *   - Layouts (dense; see the layout structs for views):
 *       x, y             [batch][seqlen][heads][P]    in_dtype, out_dtype
 *       dt               [batch][seqlen][heads]       in_dtype
 *       Bm, Cm           [batch][seqlen][groups][N]   in_dtype
 *       A, Dskip, dt_bias  [heads]                    fp32
 *       h0, hL           [sequences][heads][N][P]     fp32
 *     heads is a multiple of groups: head h reads the B and C of group
 *     h / (heads / groups).
 *   - Packed sequences: cu_seqlens is NULL (each batch row is one sequence),
 *     or a DEVICE array of num_seqs + 1 ints with batch = 1: sequence i is
 *     steps [cu_seqlens[i], cu_seqlens[i+1]) of the row.  cu_seqlens[0] is 0,
 *     entries do not decrease and the last is seqlen.  The array is read on
 *     the device only; entries outside [0, seqlen] or decreasing are clamped
 *     (nothing outside the tensors is touched), and steps that no sequence
 *     covers keep what the outputs held.  A sequence may be empty: its hL is
 *     its h0 (or zero).
 *   - Arithmetic: decay sums in double, states and all other sums in fp32.
 *     Products run on the matrix cores.  Where all tensors of a call are bf16
 *     (out_dtype and grad_dtype aside: see there), operands that are not exact
 *     in bf16 are split into bf16 terms: three (24 bits of significand) where
 *     they enter a state or form an fp32 y, two (16 bits) in what forms a bf16
 *     y, dx, dB and dC, 256 times under those outputs' own rounding (errors of
 *     fp32 arithmetic in dx, dB and dC for a caller who passes the same
 *     values as fp32).  Otherwise the products are fp32 ones.  The decode step
 *     computes in fp32 throughout.
 *   - A step's log decay D_t A below -110 acts as -110 (e^-110 is 0 in fp32).
 *     A > 0 (growth) is allowed as far as the states stay finite.
 *   - A non-finite x, dt, B or C reaches the outputs of its own head (B, C: of
 *     its group's heads) and sequence from the start of its 64-step chunk on
 *     (gradients: and of the chunks before it); other sequences and heads (dB,
 *     dC: other groups) are not touched by it.
 *   - Every pointer must be aligned to its element size; the decode `state`
 *     must be 16-byte aligned.
 * Supported sizes: batch, num_seqs and heads <= 65535, groups a divisor of
 * heads, 1 <= N <= 256, 1 <= P <= 65536, 1 <= seqlen <= 2^28 - 4096; for the
 * gradients and for kept checkpoints less than 2^23 chunks of 64 steps in all
 * (batch x ceil(seqlen / 64), packed ceil(seqlen / 64) + num_seqs).
 */
#ifndef SSM_HEADS_H
#define SSM_HEADS_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Element strides: element (b, t, h, i) of a tensor at
 * b * batch + t * step + h * head + i (Bm, Cm: head is the group's stride); the
 * last index is contiguous (dt: no last index).  0 means the dense default of
 * that index given the other strides' defaults: head P, N or 1, step heads *
 * head, batch seqlen * step.  Any order of the three is accepted; a negative
 * stride, strides for which two elements of the tensor would share a place, or
 * a tensor spanning 2^56 elements or more is SSM_ERR_BAD_SHAPE.
 * Overlap is checked on address ranges, except that tensors with the same
 * step and batch strides may lie beside each other in every step (x, Bm and Cm
 * as slices of one conv output, dx, dBm and dCm of its gradient; the larger of
 * the two strides is then a multiple of the smaller).
 * Index order: x, dt, Bm, Cm, y.  A NULL layout means all zero.
 */
typedef struct {
    long long step[5], head[5], batch[5];
} ssm_head_scan_layout_t;

/* Index order: x, dt, Bm, Cm, dy, dx, ddt, dBm, dCm. */
typedef struct {
    long long step[9], head[9], batch[9];
} ssm_head_scan_bwd_layout_t;

/* Device workspace ssm_head_scan_fwd needs, in bytes (0: none, or sizes it
 * refuses).  num_seqs is the number of packed sequences, 0 when cu_seqlens is
 * NULL.  A function of the sizes only. */
size_t ssm_head_scan_fwd_workspace_bytes(int batch, int seqlen, int groups, int heads, int N, int P,
                                         int num_seqs);

/* Device workspace of ssm_head_scan_bwd, and of ssm_head_scan_fwd with
 * SSM_FLAG_CHECKPOINTS (0 for sizes they refuse). */
size_t ssm_head_scan_bwd_workspace_bytes(int batch, int seqlen, int groups, int heads, int N, int P,
                                         int num_seqs);

/*
 * The scan over whole sequences.
 *   flags   0 or SSM_FLAG_CHECKPOINTS: the state entering every 64-step chunk
 *           is left in `workspace`, which then has
 *           ssm_head_scan_bwd_workspace_bytes(...) bytes; y and hL are
 *           unchanged bit for bit
 *   dt_bias, Dskip  [heads] or NULL (zero)
 *   h0      [sequences][heads][N][P] or NULL (zero)
 *   y       must not overlap any input
 *   hL      final states, or NULL (not returned); may be exactly h0, must not
 *           otherwise overlap an input or y
 *   layout  host pointer, read during the call only; NULL means dense
 *   workspace  16-byte aligned, overlapping no input or output
 */
ssm_status_t ssm_head_scan_fwd(int batch, int seqlen, int groups, int heads, int N, int P,
                               ssm_dtype_t in_dtype, unsigned flags, const void *x, const void *dt,
                               const float *dt_bias, const float *A, const void *Bm, const void *Cm,
                               const float *Dskip, const float *h0, const int *cu_seqlens,
                               int num_seqs, ssm_dtype_t out_dtype, void *y, float *hL,
                               void *workspace, size_t workspace_bytes,
                               const ssm_head_scan_layout_t *layout, void *stream);

/*
 * Gradients of l = sum dy . y + sum dhL . hL for every input of
 * ssm_head_scan_fwd.  dBm and dCm sum over the heads that share them.
 *   dy, dx, ddt, dBm, dCm  grad_dtype, laid out by `layout`.  Where it is not
 *                    in_dtype the products are fp32 ones and the rows are
 *                    loaded element by element
 *   dhL, dh0         [sequences][heads][N][P] fp32, each may be NULL; dh0 may
 *                    be exactly dhL
 *   dA               [heads] fp32; dDskip, ddt_bias [heads] fp32, each may be
 *                    NULL (not wanted), whether or not Dskip, dt_bias are given
 *   flags            with SSM_FLAG_CHECKPOINTS the workspace is one that
 *                    ssm_head_scan_fwd filled with that flag for the same
 *                    inputs (read, and used as scratch; the checkpoints stay);
 *                    without it the forward recurrence is run here first
 * Outputs must not overlap any input or one another.  Results do not depend
 * on timing: nothing is summed with atomics.
 */
ssm_status_t ssm_head_scan_bwd(int batch, int seqlen, int groups, int heads, int N, int P,
                               ssm_dtype_t in_dtype, unsigned flags, const void *x, const void *dt,
                               const float *dt_bias, const float *A, const void *Bm, const void *Cm,
                               const float *Dskip, const float *h0, const int *cu_seqlens,
                               int num_seqs, ssm_dtype_t grad_dtype, const void *dy,
                               const float *dhL, void *dx, void *ddt, float *ddt_bias, float *dA,
                               void *dBm, void *dCm, float *dDskip, float *dh0, void *workspace,
                               size_t workspace_bytes, const ssm_head_scan_bwd_layout_t *layout,
                               void *stream);

/*
 * One decode step: the same recurrence for one token per batch row on
 * persistent states, updated in place.
 *   state   [num_slots][heads][N][P] fp32, 16-byte aligned
 *   x, y    [batch][heads][P];  dt [batch][heads];  Bm, Cm [batch][groups][N]
 *   slots   DEVICE array of batch ints: the state of each row, or NULL (row b
 *           uses state b; num_slots is then batch).  A row whose slot is
 *           negative or not below num_slots is skipped: no state changes and
 *           its y is zero.  Two rows must not name the same slot.
 *   layout  as above; the step strides are not used
 */
ssm_status_t ssm_head_scan_update(int batch, int groups, int heads, int N, int P,
                                  ssm_dtype_t in_dtype, float *state, int num_slots,
                                  const int *slots, const void *x, const void *dt,
                                  const float *dt_bias, const float *A, const void *Bm,
                                  const void *Cm, const float *Dskip, ssm_dtype_t out_dtype,
                                  void *y, const ssm_head_scan_layout_t *layout, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_HEADS_H */

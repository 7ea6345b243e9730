/*
 * gtr_norm.h -- C ABI of the channels-last group norm on B200 (sm_100a), in the same
 * library as gtr_gla.h (libgtr_gla.so): the normalisation of a block's input or of a mixer's
 * output (one group a head) over the tokens of an image, in the same [B, N, channels] layout.
 * The statistics are over all N tokens: in a causal sequence each result depends on the tokens
 * behind it.  A norm of each token by itself is the call with the tokens as batch entries of
 * one row (B = tokens, N = 1).
 *
 *     mean, var over the N tokens and the C / groups channels of a group of one batch entry
 *     (var without Bessel's correction), rstd = 1 / sqrt(var + eps)
 *     out = act((x - mean) rstd gamma[c] + beta[c])
 *
 * Layouts (device pointers):
 *     x, out, d_out, grad_x   16-bit elements of one type (gtr_dtype_t), [B, N, C] dense,
 *                             aligned to 2 bytes (tensors on 16 bytes with C / groups a
 *                             multiple of 8 take the faster kernels)
 *     gamma, beta             float32 [C], each may be NULL (1 and 0)
 *     stats                   float32 [B, groups, 2]: mean, rstd
 * float32 tensors and the workspace are 16-byte aligned.
 *
 * Ownership, streams and errors as in gtr_gla.h: every buffer is the caller's, all work is
 * enqueued on `stream`, nothing synchronises the host and no call keeps anything.  out may be x
 * itself; nothing else may overlap.  Statistics and sums are held in float32, the variance as
 * parts of (count, mean, squared deviations) that are merged (so a mean far above the spread costs
 * no accuracy), and sums are taken in a fixed order: equal calls give equal bits.  An fp16
 * output that is stored as an infinity or NaN sets GTR_ERR_RANGE in the device error word
 * (gtr_gla_device_status).
 *   GTR_ERR_INVALID_ARG   null, misaligned, overlapping or negative arguments, groups that do
 *                         not divide C, an eps that is negative or not finite, an unknown type
 *                         or activation, N or C of 2^30 or more, B C of 2^31 or more, more than 2^40
 *                         elements, a workspace that is too small
 *   GTR_ERR_CUDA          a launch failed
 */
#ifndef GTR_NORM_H
#define GTR_NORM_H

#include <stddef.h>

#include "gtr_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of device workspace the two calls need (0: none, or arguments they would reject). */
size_t gtr_group_norm_fwd_workspace_bytes(int B, int N, int C, int groups);
size_t gtr_group_norm_bwd_workspace_bytes(int B, int N, int C, int groups);

/* stats: fully written, or NULL (not wanted).  Without any token nothing is written, stats neither. */
gtr_status_t gtr_group_norm_fwd(const void *x, const float *gamma, const float *beta, int B, int N, int C, int groups,
                                float eps, int dtype, int activation, void *out, float *stats, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * Gradients given d_out = dL/dout and the forward call's stats.  grad_gamma and grad_beta
 * (float32 [C]) may be NULL (not wanted).  Without any token they are zeros.
 */
gtr_status_t gtr_group_norm_bwd(const void *x, const void *d_out, const float *stats, const float *gamma,
                                const float *beta, int B, int N, int C, int groups, int dtype, int activation,
                                void *grad_x, float *grad_gamma, float *grad_beta, void *workspace,
                                size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GTR_NORM_H */

/*
 * gtr_ssm.h -- C ABI of the selective state-space mixer on B200 (sm_100a), in the same
 * library as gtr_gla.h (libgtr_gla.so): the second recurrent token mixer next to the
 * key-decay gated linear attention, over the same patch grids and the same four scan
 * orders (gtr_dir_t).  A sequence that is no grid is a 1 x N grid scanned GTR_L2R; a
 * single token is a 1 x 1 grid with the carried states.
 *
 * Short causal convolution (depthwise, width K in 2..4) over scan positions p:
 *     X = [init_state ; x in scan order]          K - 1 earlier inputs (or zeros), then x
 *     out_p = act(bias + sum_j w[d][j] X[p + j])
 *     final_state = the last K - 1 rows of X
 *
 * Selective scan over scan positions p, per batch b and channel d, S states n:
 *     t_p = softplus(dt_p + dt_bias)   (or dt_p + dt_bias)
 *     h_p[n] = exp(t_p A[d][n]) h_{p-1}[n] + t_p u_p Bm_p[n],   h_{-1} = init_state or 0
 *     out_p = (sum_n Cm_p[n] h_p[n] + D[d] u_p) * silu(z_p)     (no gate without z)
 * Bm and Cm are shared by all channels of a token.
 *
 * Layouts (device pointers).  Activations hold 16-bit elements of one type (gtr_dtype_t)
 * in grid order, one row of channels (or states) per token, rows `ld` elements apart
 * (ld_* = 0 means dense), so that a slice of a wider projection's output is taken as it is:
 *     x, u, dt, z, d_out                [B, N, D]       Bm, Cm   [B, N, S]    N = Hgrid * Wgrid
 *     out, grad_x, grad_u, grad_dt, grad_z   [B, N, D] dense;  grad_Bm, grad_Cm [B, N, S] dense
 *     conv init_state, final_state and their gradients: the activations' type, [B, K-1, D] dense
 *     scan init_state, final_state and their gradients: float32 [B, D, S] dense
 *     w float32 [D][K]; bias, D, dt_bias float32 [D]; A float32 [D][S]; grad_ of these alike
 * Activations are aligned to their 2 bytes, float32 tensors and the workspace to 16; sizes
 * and strides are otherwise free (rows of whole 16-byte pieces on 16 bytes are copied faster).
 *
 * Ownership, streams and errors as in gtr_gla.h: every buffer is the caller's, all work is
 * enqueued on `stream`, nothing synchronises the host, and no call keeps anything: calls
 * with buffers of their own may run at the same time on several streams.  Outputs and the
 * workspace may not overlap any input or each other, but final_state may be init_state
 * (in-place carry).  States, sums over tokens and softplus are held in float32; each output
 * is rounded once.  An fp16 output that is stored as an infinity or NaN sets GTR_ERR_RANGE in the
 * device error word (gtr_gla_device_status); bf16 outputs carry it themselves.  An infinity or
 * NaN among the inputs reaches only what the formulas send it to.
 *   GTR_ERR_INVALID_ARG   null, misaligned, overlapping or negative arguments, an unknown
 *                         direction, type or activation, N or D of 2^30 or more, more than 2^40
 *                         elements in a tensor, more than a launch's blocks cover (the scan's
 *                         gradients: B N near 2^29 and up), a workspace that is too small
 *   GTR_ERR_UNSUPPORTED   K outside 2..4; S outside 1..32
 *   GTR_ERR_CUDA          a launch failed
 */
#ifndef GTR_SSM_H
#define GTR_SSM_H

#include <stddef.h>

#include "gtr_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int B, Hgrid, Wgrid, D, K;      /* B, D >= 1; an empty grid is allowed */
    int direction;                  /* gtr_dir_t */
    int dtype;                      /* gtr_dtype_t of every activation */
    int activation;                 /* gtr_act_t */
    const void *x;
    long long ldx;                  /* elements between token rows of x; 0: D */
    const float *w;
    const float *bias;              /* or NULL */
    const void *init_state;         /* or NULL: zeros */
} gtr_conv_t;

/*
 * out: fully written.  final_state: or NULL.  An empty grid only copies init_state (or
 * zeros) to final_state.
 */
gtr_status_t gtr_causal_conv_fwd(const gtr_conv_t *conv, void *out, void *final_state, void *stream);

/* Bytes of device workspace gtr_causal_conv_bwd needs (0 for arguments it would reject). */
size_t gtr_causal_conv_bwd_workspace_bytes(int B, int Hgrid, int Wgrid, int D, int K);

/*
 * Gradients of a loss given d_out = dL/dout and d_final_state = dL/dfinal_state (or NULL).
 * grad_bias and grad_init_state may be NULL (not wanted).  The sums over tokens are taken
 * in a fixed order: equal calls give equal bits.  An empty grid writes zeros to the
 * parameters' gradients and d_final_state (or zeros) to grad_init_state.
 */
gtr_status_t gtr_causal_conv_bwd(const gtr_conv_t *conv, const void *d_out, long long ld_d_out,
                                 const void *d_final_state, void *grad_x, float *grad_w, float *grad_bias,
                                 void *grad_init_state, void *workspace, size_t workspace_bytes, void *stream);

typedef struct {
    int B, Hgrid, Wgrid, D, S;      /* B, D >= 1; S in 1..32; an empty grid is allowed */
    int direction;                  /* gtr_dir_t */
    int dtype;                      /* gtr_dtype_t of every activation */
    int dt_softplus;                /* 1: t = softplus(dt + dt_bias); 0: t = dt + dt_bias */
    const void *u, *dt, *Bm, *Cm;
    const void *z;                  /* or NULL: no gate */
    long long ldu, lddt, ldb, ldc, ldz;   /* elements between token rows; 0: dense */
    const float *A;
    const float *Dskip;             /* D above, or NULL: 0 */
    const float *dt_bias;           /* or NULL: 0 */
    const float *init_state;        /* or NULL: zeros */
} gtr_ssm_t;

/* Bytes of device workspace gtr_ssm_scan_fwd needs on the current device; 0: none needed
 * (or arguments it would reject). */
size_t gtr_ssm_scan_fwd_workspace_bytes(int B, int Hgrid, int Wgrid, int D, int S);

/*
 * out: fully written.  final_state: or NULL.  An empty grid only copies init_state (or
 * zeros) to final_state.
 */
gtr_status_t gtr_ssm_scan_fwd(const gtr_ssm_t *ssm, void *out, float *final_state, void *workspace,
                              size_t workspace_bytes, void *stream);

/* Bytes of device workspace gtr_ssm_scan_bwd needs (0 for arguments it would reject). */
size_t gtr_ssm_scan_bwd_workspace_bytes(int B, int Hgrid, int Wgrid, int D, int S);

typedef struct {
    void *u, *dt, *Bm, *Cm;         /* required */
    void *z;                        /* required with a gate, else not looked at */
    float *A;                       /* required */
    float *Dskip, *dt_bias;         /* or NULL: not wanted */
    float *init_state;              /* or NULL: not wanted */
} gtr_ssm_grads_t;

/*
 * Gradients of a loss given d_out = dL/dout and d_final_state = dL/dfinal_state (or NULL);
 * A's gradient is with respect to A as it is given.  The sums over tokens and over channels
 * are taken in a fixed order: equal calls give equal bits.  An empty grid writes zeros to the
 * parameters' gradients and d_final_state (or zeros) to init_state's.
 */
gtr_status_t gtr_ssm_scan_bwd(const gtr_ssm_t *ssm, const void *d_out, long long ld_d_out,
                              const float *d_final_state, const gtr_ssm_grads_t *grads, void *workspace,
                              size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GTR_SSM_H */

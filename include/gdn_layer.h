/*
 * gdn_layer.h -- C ABI of libgdn.so for the operators a recurrent layer needs
 * around the gated delta rule of gdn.h: the residual addition with the RMS
 * norm, microscaled (MX) quantisation and products, and a per-channel gated
 * linear recurrence.
 *
 * The conventions are those of gdn.h: device pointers on the current device,
 * contiguous row-major tensors whose bases are 16-byte aligned, every call
 * asynchronous on `stream`, memory owned by the caller, host-detectable
 * argument problems returned before anything is launched (gdn_last_error()
 * describes them), device-detected ones recorded for gdn_sync_status().
 */
#ifndef GDN_LAYER_H_
#define GDN_LAYER_H_

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Gated linear recurrence, per channel:
 *
 *     h_t = exp(l_t) h_{t-1} + x_t
 *
 * with the log decay l_t = g_t, or -gate_scale_d softplus(g_t) when gate_scale
 * is given (the same gate as gdn_fwd_args.gate_scale, per channel).  l <= 0 is
 * expected: the scan multiplies decays together, and a product of growing
 * factors can overflow where the recurrence itself would not. */
typedef struct gdn_linrec_fwd_args {
    const void *x;              /* [B, T, D], dtype                                  */
    const void *g;              /* [B, T, D], dtype: log decay, or gate logits       */
    const float *gate_scale;    /* NULL, or [D]                                      */
    const float *initial_state; /* [N, D], NULL = zeros                              */
    const int32_t *cu_seqlens;  /* NULL (N = B rows of T tokens), or [N + 1] as in
                                   gdn_fwd_args (B must be 1; sequences may be empty) */
    int32_t B, T, D, N;         /* N is read only with cu_seqlens                    */
    int32_t dtype;              /* GDN_FP32 or GDN_BF16                              */
    void *h;                    /* [B, T, D], dtype                                  */
    float *final_state;         /* [N, D], NULL = not written                        */
} gdn_linrec_fwd_args;

/* Backward:  e_t = dh_t + c_t;  c_{t-1} = exp(l_t) e_t;  c_{T-1} = d_final_state;
 *            dx_t = e_t;  dl_t = exp(l_t) h_{t-1} e_t;  d_initial_state = c_{-1}.
 * h is what the forward wrote.  dg is dl, or the gradient with respect to the
 * logits when gate_scale is given. */
typedef struct gdn_linrec_bwd_args {
    const void *d_h;            /* [B, T, D], dtype                                  */
    const void *g;              /* as in the forward                                 */
    const void *h;              /* [B, T, D], dtype                                  */
    const float *gate_scale;
    const float *initial_state;
    const int32_t *cu_seqlens;
    const float *d_final_state; /* [N, D], NULL = zeros                              */
    int32_t B, T, D, N;
    int32_t dtype;
    void *dx, *dg;              /* [B, T, D], dtype                                  */
    float *d_initial_state;     /* [N, D], NULL = not written                        */
    float *d_gate_scale;        /* [D], NULL = not written (ignored without gate_scale) */
} gdn_linrec_bwd_args;

/* One token for each of N sequences. */
typedef struct gdn_linrec_step_args {
    const void *x, *g;          /* [N, D], dtype                                     */
    const float *gate_scale;    /* NULL, or [D]                                      */
    const float *state;         /* [N, D]                                            */
    int32_t N, D;
    int32_t dtype;
    void *h;                    /* [N, D], dtype                                     */
    float *out_state;           /* [N, D]: may be `state` itself                     */
} gdn_linrec_step_args;

gdn_status gdn_linrec_fwd(const gdn_linrec_fwd_args *args, void *stream);
/* Bytes of workspace for these arguments: 256 at least, 0 when they are invalid. */
size_t gdn_linrec_bwd_workspace_size(const gdn_linrec_bwd_args *args);
gdn_status gdn_linrec_bwd(const gdn_linrec_bwd_args *args, void *workspace,
                          size_t workspace_bytes, void *stream);
gdn_status gdn_linrec_step(const gdn_linrec_step_args *args, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* GDN_LAYER_H_ */

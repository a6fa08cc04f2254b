/*
 * gdn_layer.h -- C ABI of libgdn.so for the operators a recurrent layer needs
 * around the gated delta rule of gdn.h: the residual addition with the RMS
 * norm, microscaled (MX) quantisation and products, a per-channel gated linear
 * recurrence, the short causal convolution, the selective state space scan, and the gated
 * feed-forward block.
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
    float *out_state;           /* [N, D]: may be `state` itself, not part of it     */
} gdn_linrec_step_args;

/* Bytes of workspace for these arguments: 256 (then none is read, and it may be NULL) or
 * more, 0 when the arguments are invalid. */
size_t gdn_linrec_fwd_workspace_size(const gdn_linrec_fwd_args *args);
gdn_status gdn_linrec_fwd(const gdn_linrec_fwd_args *args, void *workspace,
                          size_t workspace_bytes, void *stream);
size_t gdn_linrec_bwd_workspace_size(const gdn_linrec_bwd_args *args);
gdn_status gdn_linrec_bwd(const gdn_linrec_bwd_args *args, void *workspace,
                          size_t workspace_bytes, void *stream);
gdn_status gdn_linrec_step(const gdn_linrec_step_args *args, void *stream);

/* ------------------------------------------------------------------------
 * Microscaled (MX) tensors.  A matrix [rows, K], K a multiple of 32, is held as
 * elements of 8 or 4 bits and one scale for each row and 32 columns:
 * value = element * 2^(scale byte - 127); a scale byte of 255 stands for NaN.
 *
 *   GDN_MXFP8   e4m3 elements, a byte each, [rows, K]
 *   GDN_MXFP4   e2m1 elements, two to a byte (the first in the low half), [rows, K / 2]
 *
 * Scales are held in the order the product's tensor-core instructions read them:
 * tiles of 128 rows x 4 blocks (512 bytes), row-tile-major, ceil(rows / 128) x
 * ceil(K / 128) of them.  Inside a tile the byte of (row, block) is at
 * 16 (row % 32) + 4 (row / 32) + block.  Rows and blocks past the end of the
 * matrix hold zeros (2^-127).
 *
 * Quantisation takes, for each block, the least exponent that keeps the block's
 * largest magnitude within the element type (448 or 6), at least -127, and rounds
 * the scaled elements to nearest, ties to even: nothing saturates.  (The rounded-
 * down exponent that is the usual choice lets the largest element of a block
 * saturate, an error of up to 1/8 for e4m3 and 1/4 for e2m1 in the element that
 * matters most.)  A block that holds a NaN or an infinity gets a NaN scale.
 *
 * K, and M and N of a product, are at most 2^31 - 2^16. */
enum { GDN_MXFP8 = 0, GDN_MXFP4 = 1 };

/* Bytes of the scales of a [rows, K] matrix (0 for rows or K of none). */
size_t gdn_mx_scale_bytes(int32_t rows, int32_t K);

typedef struct gdn_mx_quantize_args {
    const void *x;              /* [rows, K], dtype                                  */
    int32_t rows, K;
    int32_t dtype;              /* GDN_FP32 or GDN_BF16                              */
    int32_t format;             /* GDN_MXFP8 or GDN_MXFP4                            */
    void *data;                 /* elements                                          */
    uint8_t *scales;            /* gdn_mx_scale_bytes(rows, K)                       */
} gdn_mx_quantize_args;
gdn_status gdn_mx_quantize(const gdn_mx_quantize_args *args, void *stream);

/* The values of an MX matrix: x [rows, K], dtype (the same struct, read the other way). */
typedef struct gdn_mx_dequantize_args {
    const void *data;
    const uint8_t *scales;
    int32_t rows, K;
    int32_t dtype, format;
    void *x;
} gdn_mx_dequantize_args;
gdn_status gdn_mx_dequantize(const gdn_mx_dequantize_args *args, void *stream);

/* C [M, N] = A B^T of MX matrices A [M, K] and B [N, K] of one format, summed in
 * fp32.  A block with a NaN scale makes its row's (column's) results NaN. */
typedef struct gdn_mx_matmul_args {
    const void *a;
    const uint8_t *a_scales;
    const void *b;
    const uint8_t *b_scales;
    int32_t M, N, K;            /* K a multiple of 32; 0 gives zeros                 */
    int32_t format;
    int32_t out_dtype;          /* GDN_FP32 or GDN_BF16                              */
    void *c;                    /* [M, N]                                            */
} gdn_mx_matmul_args;
gdn_status gdn_mx_matmul(const gdn_mx_matmul_args *args, void *stream);

/* C [M, N] = X W^T with X [M, K] quantised to W's format on the way, into the workspace:
 * the results of gdn_mx_quantize and gdn_mx_matmul.  Of large products only the first rows
 * are quantised ahead, the others under the product's own MMAs. */
typedef struct gdn_mx_linear_args {
    const void *x;              /* [M, K], dtype                                     */
    const void *w;              /* [N, K] MX matrix                                  */
    const uint8_t *w_scales;
    int32_t M, N, K;
    int32_t dtype;              /* of x: GDN_FP32 or GDN_BF16                        */
    int32_t format;
    int32_t out_dtype;
    void *c;                    /* [M, N]                                            */
} gdn_mx_linear_args;
size_t gdn_mx_linear_workspace_size(const gdn_mx_linear_args *args);
gdn_status gdn_mx_linear(const gdn_mx_linear_args *args, void *workspace, size_t workspace_bytes,
                         void *stream);

/* ------------------------------------------------------------------------
 * Residual addition and RMS norm, per row of D columns:
 *
 *     s = x + residual;  rstd = (mean(s^2) + eps)^-1/2;  y = s rstd weight
 *
 * in fp32 from the unrounded sum.  y has the input's type, or is an MXFP8 matrix
 * for gdn_mx_matmul. */
typedef struct gdn_rms_norm_fwd_args {
    const void *x;              /* [rows, D], dtype                                  */
    const void *residual;       /* [rows, D], dtype, NULL = none                     */
    const void *weight;         /* [D], dtype                                        */
    int32_t rows, D;            /* 1 <= D <= 16384; a multiple of 32 for MXFP8       */
    int32_t dtype;
    float eps;
    int32_t mx;                 /* 0: y in dtype; 1: y is MXFP8                      */
    void *y;                    /* [rows, D], dtype or e4m3                          */
    uint8_t *scales;            /* mx: gdn_mx_scale_bytes(rows, D)                   */
    void *sum;                  /* [rows, D], dtype: s; required with residual, else unused */
    float *rstd;                /* [rows], NULL = not written                        */
} gdn_rms_norm_fwd_args;
gdn_status gdn_rms_norm_fwd(const gdn_rms_norm_fwd_args *args, void *stream);

/* Backward, xh = s rstd:  ds = rstd (w dy - xh mean(w dy xh)) + d_sum;  dw = sum over rows of dy xh.
 * ds is the gradient of x and of the residual. */
typedef struct gdn_rms_norm_bwd_args {
    const void *dy;             /* [rows, D], dtype                                  */
    const void *sum;            /* [rows, D], dtype: s (x itself without a residual) */
    const void *weight;         /* [D], dtype                                        */
    const float *rstd;          /* [rows]                                            */
    const void *d_sum;          /* [rows, D], dtype: gradient that reaches s past the norm; NULL = none */
    int32_t rows, D;
    int32_t dtype;
    void *ds;                   /* [rows, D], dtype                                  */
    float *dweight;             /* [D]                                               */
} gdn_rms_norm_bwd_args;
size_t gdn_rms_norm_bwd_workspace_size(const gdn_rms_norm_bwd_args *args);
gdn_status gdn_rms_norm_bwd(const gdn_rms_norm_bwd_args *args, void *workspace,
                            size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Short causal convolution along the tokens, per channel, with its activation:
 *
 *     pre_t = bias + sum over k of weight[k] xp_{t + k},   y = act(pre)
 *
 * xp being the W - 1 inputs before the sequence (initial_state, or zeros) and then x.
 * The state after a sequence is the last W - 1 rows of xp, whatever its length. */
enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1, GDN_ACT_GELU = 2 };

typedef struct gdn_conv_fwd_args {
    const void *x;              /* [B, T, D], dtype                                  */
    const void *weight;         /* [D, W], dtype: the last tap is the token's own    */
    const void *bias;           /* [D], dtype, NULL = none                           */
    const void *initial_state;  /* [N, W - 1, D], dtype, oldest first; NULL = zeros  */
    const int32_t *cu_seqlens;  /* as in gdn_linrec_fwd_args                         */
    int32_t B, T, D, N, W;      /* W is 2, 3 or 4                                    */
    int32_t dtype;              /* GDN_FP32 or GDN_BF16                              */
    int32_t activation;         /* GDN_ACT_NONE or GDN_ACT_SILU                      */
    void *y;                    /* [B, T, D], dtype                                  */
    void *final_state;          /* [N, W - 1, D], dtype, NULL = not written          */
} gdn_conv_fwd_args;
gdn_status gdn_conv_fwd(const gdn_conv_fwd_args *args, void *stream);

/* Backward, dpre = dy act'(pre):  dxp_i = sum over k of weight[k] dpre_{i - k}, the last W - 1
 * rows with d_final_state added to them;  dweight[k] = sum over tokens of dpre_t xp_{t + k};
 * dbias = sum of dpre.  dx and d_initial_state are the two parts of dxp. */
typedef struct gdn_conv_bwd_args {
    const void *d_y;            /* [B, T, D], dtype                                  */
    const void *x, *weight, *bias, *initial_state;                 /* the forward's  */
    const int32_t *cu_seqlens;
    const void *d_final_state;  /* [N, W - 1, D], dtype, NULL = zeros                */
    int32_t B, T, D, N, W;
    int32_t dtype, activation;
    void *dx;                   /* [B, T, D], dtype                                  */
    float *dweight;             /* [D, W]                                            */
    float *dbias;               /* [D], NULL = not written                           */
    void *d_initial_state;      /* [N, W - 1, D], dtype, NULL = not written          */
} gdn_conv_bwd_args;
/* 256 or more, as gdn_linrec_bwd_workspace_size. */
size_t gdn_conv_bwd_workspace_size(const gdn_conv_bwd_args *args);
gdn_status gdn_conv_bwd(const gdn_conv_bwd_args *args, void *workspace, size_t workspace_bytes,
                        void *stream);

/* One token for each of N sequences. */
typedef struct gdn_conv_step_args {
    const void *x;              /* [N, D], dtype                                     */
    const void *weight, *bias;
    const void *state;          /* [N, W - 1, D], dtype                              */
    int32_t N, D, W;
    int32_t dtype, activation;
    void *y;                    /* [N, D], dtype                                     */
    void *out_state;            /* [N, W - 1, D], dtype: may be `state` itself, not
                                   part of it                                        */
} gdn_conv_step_args;
gdn_status gdn_conv_step(const gdn_conv_step_args *args, void *stream);

/* ------------------------------------------------------------------------
 * Selective state space scan: per channel d and state s,
 *
 *     h_t = exp(delta_t a) h_{t-1} + delta_t x_t b_t,   y_t = (<c_t, h_t> + skip x_t) silu(z_t)
 *
 * with the step delta = dt, or softplus(dt + dt_bias) when dt_bias is given; b_t and c_t belong to
 * the token, a and skip to the channel.  delta >= 0 and a <= 0 are expected (a step of 0 leaves the
 * state as it is): decays are multiplied together, and a product of growing factors can overflow
 * where the recurrence itself would not.  States are fp32. */
typedef struct gdn_ssm_fwd_args {
    const void *x;              /* [B, T, D], dtype                                  */
    const void *dt;             /* [B, T, D], dtype: steps, or their logits          */
    const float *a;             /* [D, S]                                            */
    const void *b, *c;          /* [B, T, S], dtype                                  */
    const float *skip;          /* [D], NULL = none                                  */
    const void *z;              /* [B, T, D], dtype, NULL = no gate                  */
    const float *dt_bias;       /* [D], or NULL                                      */
    const float *initial_state; /* [N, D, S], NULL = zeros                           */
    const int32_t *cu_seqlens;  /* as in gdn_linrec_fwd_args                         */
    int32_t B, T, D, S, N;      /* 1 <= S <= 64; at most 65535 sequences             */
    int32_t dtype;              /* GDN_FP32 or GDN_BF16                              */
    void *y;                    /* [B, T, D], dtype                                  */
    float *final_state;         /* [N, D, S], NULL = not written                     */
} gdn_ssm_fwd_args;

/* Backward, ds_t = dy_t silu(z_t) and e_t = c_t ds_t + exp(delta_{t+1} a) e_{t+1} (d_final_state
 * behind the last token), p_t = exp(delta_t a) h_{t-1}:
 *     db_t = sum over d of e delta x;  dc_t = sum over d of ds h;  dx = skip ds + delta <e, b>;
 *     ddelta = x <e, b> + <e, a p>;  da = sum over t of e delta p;  dskip = sum of ds x;
 *     dz = dy (<c, h> + skip x) silu'(z);  d_initial_state = exp(delta_0 a) e_0.
 * ddt is ddelta, or the logits' gradient when dt_bias is given. */
typedef struct gdn_ssm_bwd_args {
    const void *d_y;            /* [B, T, D], dtype                                  */
    const void *x, *dt;         /* the forward's                                     */
    const float *a;
    const void *b, *c;
    const float *skip;
    const void *z;
    const float *dt_bias, *initial_state;
    const int32_t *cu_seqlens;
    const float *d_final_state; /* [N, D, S], NULL = zeros                           */
    int32_t B, T, D, S, N;
    int32_t dtype;
    void *dx, *ddt;             /* [B, T, D], dtype                                  */
    float *da;                  /* [D, S]                                            */
    void *db, *dc;              /* [B, T, S], dtype                                  */
    float *dskip;               /* [D], NULL = not written (ignored without skip)    */
    void *dz;                   /* [B, T, D], dtype: required with z                 */
    float *ddt_bias;            /* [D], NULL = not written (ignored without dt_bias) */
    float *d_initial_state;     /* [N, D, S], NULL = not written                     */
} gdn_ssm_bwd_args;

/* One token for each of N sequences. */
typedef struct gdn_ssm_step_args {
    const void *x, *dt;         /* [N, D], dtype                                     */
    const float *a;
    const void *b, *c;          /* [N, S], dtype                                     */
    const float *skip;
    const void *z;              /* [N, D], dtype, NULL = no gate                     */
    const float *dt_bias;
    const float *state;         /* [N, D, S]                                         */
    int32_t N, D, S;
    int32_t dtype;
    void *y;                    /* [N, D], dtype                                     */
    float *out_state;           /* [N, D, S]: may be `state` itself, not part of it  */
} gdn_ssm_step_args;

/* Bytes of workspace, as gdn_linrec_fwd_workspace_size. */
size_t gdn_ssm_fwd_workspace_size(const gdn_ssm_fwd_args *args);
gdn_status gdn_ssm_fwd(const gdn_ssm_fwd_args *args, void *workspace, size_t workspace_bytes,
                       void *stream);
size_t gdn_ssm_bwd_workspace_size(const gdn_ssm_bwd_args *args);
gdn_status gdn_ssm_bwd(const gdn_ssm_bwd_args *args, void *workspace, size_t workspace_bytes,
                       void *stream);
gdn_status gdn_ssm_step(const gdn_ssm_step_args *args, void *stream);

/* ------------------------------------------------------------------------
 * Gated feed-forward block of M tokens of width K, F features wide inside:
 *
 *     g = x w_gate^T,  u = x w_up^T,  h = act(g) u,  y = h w_down^T
 *
 * act is silu, or gelu in its tanh form.  bf16 tensors, fp32 sums; h is rounded to bf16 between the
 * products (of up to 64 tokens to twice its bits).  K and F are multiples of 8. */
typedef struct gdn_ffn_fwd_args {
    const void *x;              /* [M, K], dtype                                     */
    const void *w_gate, *w_up;  /* [F, K], dtype                                     */
    const void *w_down;         /* [K, F], dtype                                     */
    int32_t M, K, F;
    int32_t dtype;              /* GDN_BF16                                          */
    int32_t activation;         /* GDN_ACT_SILU or GDN_ACT_GELU                      */
    void *y;                    /* [M, K], dtype                                     */
    void *gate, *up;            /* [M, F], dtype: g and u for the backward pass; NULL
                                   (both) = not written                              */
} gdn_ffn_fwd_args;

/* Backward, dh = dy w_down:  dg = dh u act'(g), du = dh act(g);  dx = dg w_gate + du w_up;
 * dw_gate = dg^T x, dw_up = du^T x, dw_down = dy^T h (h from gate and up once more).  dg, du and h
 * are rounded to bf16 between the products (of up to 8 tokens not at all). */
typedef struct gdn_ffn_bwd_args {
    const void *d_y;            /* [M, K], dtype                                     */
    const void *x, *w_gate, *w_up, *w_down;                        /* the forward's  */
    const void *gate, *up;      /* [M, F], dtype: what the forward wrote             */
    int32_t M, K, F;
    int32_t dtype, activation;
    void *dx;                   /* [M, K], dtype                                     */
    void *dw_gate, *dw_up;      /* [F, K], dtype                                     */
    void *dw_down;              /* [K, F], dtype                                     */
} gdn_ffn_bwd_args;

size_t gdn_ffn_fwd_workspace_size(const gdn_ffn_fwd_args *args);
gdn_status gdn_ffn_fwd(const gdn_ffn_fwd_args *args, void *workspace, size_t workspace_bytes,
                       void *stream);
size_t gdn_ffn_bwd_workspace_size(const gdn_ffn_bwd_args *args);
gdn_status gdn_ffn_bwd(const gdn_ffn_bwd_args *args, void *workspace, size_t workspace_bytes,
                       void *stream);

#ifdef __cplusplus
}
#endif
#endif /* GDN_LAYER_H_ */

/*
 * kda_layers.h -- the operators around a recurrent mixer: short convolution,
 * selective state space scan, block norm.  Same library and conventions as kda.h
 * (device pointers owned by the caller, work enqueued on `stream`, negative status on a
 * refusal, every check on the host before the first CUDA call, 16-byte aligned pointers,
 * kda_opts for the element type and the workspace).
 *
 * These operators stand next to the KDA entry points: kda_chunk_fwd_prologue has the
 * short convolution fused ahead of the KDA forward, kda_chunk_fwd_gated a gated RMSNorm
 * behind it, both without a gradient.  Here both are operators of their own, forward and
 * backward, with a second token mixer, the selective scan.
 *
 * kda_opts here: dtype is the type of the activations (bf16 or fp32); workspace, events
 * and n_events as in kda.h; scale is not used; of the flags only KDA_QK_L2NORM, which the
 * default options carry, is accepted, and it changes nothing (KDA_ERR_ARG otherwise).
 *
 * Sequences.  Rows are tokens.  Without cu_seqlens there are B sequences of T rows, B * T
 * rows in all.  With cu_seqlens (device, B + 1 int32, non-decreasing) there are B sequences
 * packed in T rows: sequence s has the rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1, possibly
 * none.  Bounds outside 0 .. T are clamped on the device.  Rows of no sequence are neither
 * read nor written, unless zero_rest is set: then the call's row outputs are zero there.
 *
 * At most 2^31 - 256 rows.  Row strides (ld_*) count elements, at most 2^27; 0 means the
 * row's own length (contiguous).  A tensor with a row stride may so be a column range of a
 * wider one, and unlike the others it may start at any element; rows at 16 bytes are read in
 * wider accesses.  Outputs must not overlap inputs or each other unless a comment says so
 * (KDA_ERR_ARG); column ranges of one wider tensor do not.
 *
 * Gradients of activations have the activation type, gradients of parameters and states
 * are FP32; all are written, not accumulated, and every sum has a fixed order.
 */
#ifndef KDA_B200_KDA_LAYERS_H
#define KDA_B200_KDA_LAYERS_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes and layout of the short convolution. */
typedef struct {
    int B, T, D, K;          /* sequences, rows (see above), channels, taps: 2, 3 or 4     */
    int silu;                /* 1: y = pre * sigmoid(pre), 0: y = pre                      */
    const int *cu_seqlens;   /* packed sequences, or NULL                                  */
    int zero_rest;           /* packed only: rows of no sequence are set to zero           */
    long long ld_x, ld_y, ld_dx;   /* rows of x; of y and dy; of dx                        */
} kda_conv_dims;

/*
 * kda_short_conv_fwd -- causal depthwise convolution over time, bias and SiLU.
 *
 *   pre[t, c] = bias[c] + sum_j w[c, j] x[t - (K-1) + j, c],  y = pre * sigmoid(pre)
 *
 *   x [rows, D], w [D, K] (tap K-1 on the current row), bias [D] or NULL, y [rows, D]
 *   state0  [B, K-1, D]  the K-1 rows ahead of each sequence, oldest first; NULL = zeros
 *   state_T [B, K-1, D]  the last K-1 rows of state0 and sequence together; NULL to skip
 * All of the activation type, sums in FP32.
 */
int kda_short_conv_fwd(const void *x, const void *w, const void *bias, const void *state0,
                       void *y, void *state_T, const kda_conv_dims *dims, const kda_opts *opts,
                       cudaStream_t stream);

/*
 * kda_short_conv_bwd -- gradients of <dy, y> + <dstate_T, state_T> of kda_short_conv_fwd.
 *
 *   dy [rows, D] (activation type: FP32 gradients, such as kda_chunk_bwd's, go into an FP32
 *   call as they are and into a bf16 one rounded); dstate_T [B, K-1, D] FP32 or NULL (zero)
 *   dx [rows, D] (activation type); dw [D, K] FP32; dbias [D] FP32 or NULL to skip;
 *   dstate0 [B, K-1, D] FP32 or NULL to skip
 * opts->workspace: kda_short_conv_bwd_workspace_bytes(dims, opts) bytes.
 */
int kda_short_conv_bwd(const void *x, const void *w, const void *bias, const void *state0,
                       const void *dy, const float *dstate_T, void *dx, float *dw, float *dbias,
                       float *dstate0, const kda_conv_dims *dims, const kda_opts *opts,
                       cudaStream_t stream);
size_t kda_short_conv_bwd_workspace_bytes(const kda_conv_dims *dims, const kda_opts *opts);

/*
 * kda_short_conv_step -- one row for each of dims->B sequences (decode); T and cu_seqlens
 * are not used.  x, y [B, D]; state [B, K-1, D] is read, the shifted state goes to
 * state_out, which may be state itself (in place).
 */
int kda_short_conv_step(const void *x, const void *w, const void *bias, const void *state,
                        void *state_out, void *y, const kda_conv_dims *dims,
                        const kda_opts *opts, cudaStream_t stream);

/* Sizes and layout of the selective scan. */
typedef struct {
    int B, T, D, N, G;       /* sequences, rows, channels, states a channel: 8, 16, 32 or 64;
                                groups: G divides D, channels d G / D share one B and C     */
    int dt_softplus;         /* 1: delta = softplus(dt + dt_bias), 0: delta = dt + dt_bias  */
    const int *cu_seqlens;
    int zero_rest;
    long long ld_u, ld_dt, ld_z, ld_B, ld_C, ld_out;   /* ld_out: rows of out and of dout   */
} kda_ssm_dims;

/*
 * kda_ssm_scan_fwd -- selective state space scan over sequences (training, prompts).
 *
 *   h_t[d, n] = exp(delta_t[d] A[d, n]) h_{t-1}[d, n] + delta_t[d] u_t[d] B_t[g(d), n]
 *   out_t[d]  = (sum_n C_t[g(d), n] h_t[d, n] + Dskip[d] u_t[d]) * z_t[d] sigmoid(z_t[d])
 *
 *   u, dt, z, out [rows, D], Bm, Cm [rows, G, N]   activation type (z NULL: no gate)
 *   A [D, N], Dskip [D] or NULL, dt_bias [D] or NULL   FP32
 *   h0 [B, D, N] FP32 or NULL (zero); h_T [B, D, N] FP32, the last states, NULL to skip
 * A <= 0 and delta >= 0 in earnest: long sequences take products of the factors exp(delta A) over
 * many tokens, here and in the backward, which have to stay finite in FP32 where factors exceed 1.
 * States and sums are FP32.  opts->workspace: kda_ssm_scan_fwd_workspace_bytes bytes (0 for
 * sizes whose sequences and channels alone fill the device).
 */
int kda_ssm_scan_fwd(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                     const float *Dskip, const void *z, const float *dt_bias, const float *h0,
                     void *out, float *h_T, const kda_ssm_dims *dims, const kda_opts *opts,
                     cudaStream_t stream);
size_t kda_ssm_scan_fwd_workspace_bytes(const kda_ssm_dims *dims, const kda_opts *opts);

/*
 * kda_ssm_scan_bwd -- gradients of <dout, out> + <dh_T, h_T> of kda_ssm_scan_fwd.
 *
 *   dout [rows, D] (rows ld_out apart); dh_T [B, D, N] FP32 or NULL (zero)
 *   du, ddt, dz [rows, D], dB, dC [rows, G, N]   contiguous, activation type (dz NULL
 *   exactly when z is)
 *   dA [D, N], dDskip [D], ddt_bias [D], dh0 [B, D, N]   FP32; the last three NULL to skip
 * opts->workspace: kda_ssm_scan_bwd_workspace_bytes bytes.
 */
int kda_ssm_scan_bwd(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                     const float *Dskip, const void *z, const float *dt_bias, const float *h0,
                     const void *dout, const float *dh_T, void *du, void *ddt, float *dA, void *dB,
                     void *dC, float *dDskip, void *dz, float *ddt_bias, float *dh0,
                     const kda_ssm_dims *dims, const kda_opts *opts, cudaStream_t stream);
size_t kda_ssm_scan_bwd_workspace_bytes(const kda_ssm_dims *dims, const kda_opts *opts);

/*
 * kda_ssm_step -- one token for each of dims->B sequences (decode); T and cu_seqlens are
 * not used.  u, dt, z, out [B, D], Bm, Cm [B, G, N]; h [B, D, N] FP32 is read, the new state
 * goes to h_out, which may be h itself (in place).  No workspace.
 */
int kda_ssm_step(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                 const float *Dskip, const void *z, const float *dt_bias, const float *h,
                 float *h_out, void *out, const kda_ssm_dims *dims, const kda_opts *opts,
                 cudaStream_t stream);

/* Sizes and layout of the block norm. */
typedef struct {
    int rows, D;             /* D from 1 to 16384                                          */
    float eps;               /* added to the mean square, finite and >= 0                  */
    long long ld_res, ld_block, ld_gate;   /* rows of residual; of block; of gate          */
} kda_norm_dims;

/*
 * kda_block_norm_fwd -- the norms behind one block and ahead of the next, with the block's
 * gate, its residual scale and the residual sum between them.
 *
 *   rms(v) = v / sqrt(mean(v^2) + eps)
 *   res_out = residual + scale * sigmoid(gate) * rms(block) * w_post
 *   x       = rms(res_out) * w_pre
 *
 *   residual, block, gate [rows, D]; res_out, x [rows, D] contiguous   activation type
 *   scale, w_post, w_pre [D] FP32, NULL = ones;  gate NULL = no gate
 * block NULL: res_out must be NULL too and x = rms(residual) * w_pre (ahead of the first
 * block).  x NULL: only res_out (behind the last block).  res_out may be residual itself
 * (in place, ld_res then D).  x is computed from the FP32 res_out, before its rounding.
 */
int kda_block_norm_fwd(const void *residual, const void *block, const void *gate,
                       const float *scale, const float *w_post, const float *w_pre, void *res_out,
                       void *x, const kda_norm_dims *dims, const kda_opts *opts,
                       cudaStream_t stream);

/*
 * kda_block_norm_bwd -- gradients of <dres, res_out> + <dx, x> of kda_block_norm_fwd.
 *
 * Takes res_out as the forward left it (rows ld_res apart) in place of residual; with
 * block NULL, that is the forward's residual.
 *   dres, dx [rows, D] contiguous, activation type; either may be NULL (zero), not both
 *   dresidual [rows, D], dblock [rows, D] (NULL exactly when block is), dgate [rows, D]
 *   (NULL exactly when gate is)   contiguous, activation type; dresidual may be dres itself
 *   dscale, dw_post, dw_pre [D] FP32, each NULL to skip
 * opts->workspace: kda_block_norm_bwd_workspace_bytes bytes.
 */
int kda_block_norm_bwd(const void *res_out, const void *block, const void *gate,
                       const float *scale, const float *w_post, const float *w_pre,
                       const void *dres, const void *dx, void *dresidual, void *dblock,
                       void *dgate, float *dscale, float *dw_post, float *dw_pre,
                       const kda_norm_dims *dims, const kda_opts *opts, cudaStream_t stream);
size_t kda_block_norm_bwd_workspace_bytes(const kda_norm_dims *dims, const kda_opts *opts);

#ifdef __cplusplus
}
#endif
#endif /* KDA_B200_KDA_LAYERS_H */

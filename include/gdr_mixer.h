/*
 * gdr_mixer.h — C ABI of the operators that stand next to the gated delta
 * rule in a sequence-mixing layer (AMD MI355X, gfx950):
 *
 *   short causal convolution   forward, one token per sequence, backward
 *   selective state space scan forward, one token per sequence, backward
 *   layer norm                 forward, backward
 *
 * Conventions are those of gdr.h: device pointers except cu_seqlens_host, the
 * caller owns every buffer, work is enqueued on `stream` and nothing is
 * synchronised, argument errors are found on the host before anything is
 * enqueued, statuses and gdr_last_error_message are shared. Differences:
 *
 * - Base addresses need the alignment of their element type only.
 * - Input rows may be strided: x_stride (and the other *_stride fields) is the
 *   distance in elements between consecutive tokens (or rows), the elements of
 *   one token being contiguous. Token t of batch row b is row b * seq_len + t.
 *   Outputs, states, gradients and parameters are dense.
 * - Variable-length batches: as in gdr.h, batch = 1, seq_len = total tokens and
 *   both copies of cu_seqlens. Sequences may be empty. If the two copies
 *   differ, the results are unspecified, but every access stays in its buffer.
 * - Every sum, state and statistic is fp32. A result in bf16 is rounded once,
 *   when it is stored. Sums over tokens, rows and channels run in a fixed
 *   order: the same call gives the same bits.
 * - Sequences do not touch each other: NaN or Inf in one stays in its outputs
 *   (gradients of parameters, which sum over all sequences, excepted).
 */
#ifndef GDR_MIXER_H
#define GDR_MIXER_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GDR_ACT_NONE = 0, GDR_ACT_SILU = 1 } gdr_activation_t;

/*
 * Short causal convolution, one filter per channel:
 *   p_t[d] = bias[d] + sum_{w < W} weight[d][w] u_{t-(W-1)+w}[d],   y = p or p / (1 + exp(-p))
 * where u is the sequence preceded by its W - 1 initial rows.
 *   x       [batch, seq_len, D] io_dtype, token stride x_stride
 *   weight  [D][W], bias [D] or NULL: param_dtype
 *   state   [num_seqs][W-1][D] io_dtype: the last W - 1 rows of u, oldest first
 */
typedef struct {
    int64_t batch, seq_len;
    int64_t x_stride;       /* elements between tokens of x, >= channels                 */
    int32_t num_seqs;       /* batch, or len(cu_seqlens) - 1                             */
    int32_t channels;       /* D: 1 to 2^30                                              */
    int32_t width;          /* W: 2, 3 or 4                                              */
    int32_t activation;     /* gdr_activation_t                                          */
    int32_t io_dtype;       /* x, y and states                                           */
    int32_t param_dtype;    /* weight and bias: io_dtype or GDR_F32                      */
    int32_t dy_dtype;       /* backward: d_y and d_final_state, io_dtype or GDR_F32      */
    int32_t grad_dtype;     /* backward: dx and d_initial_state, io_dtype or GDR_F32     */
} gdr_conv_problem_t;

/* initial_state NULL means zeros; final_state NULL is skipped (it may not
 * overlap initial_state). */
gdr_status_t gdr_conv_fwd(const gdr_conv_problem_t* problem, const void* x, const void* weight, const void* bias,
                          const void* initial_state, const int32_t* cu_seqlens_dev, const int32_t* cu_seqlens_host,
                          void* y, void* final_state, void* stream);

/* One token of every sequence: batch = num_seqs rows of x, seq_len = 1. `state`
 * is read and then overwritten by the state after the token. */
gdr_status_t gdr_conv_step(const gdr_conv_problem_t* problem, const void* x, const void* weight, const void* bias,
                           void* state, void* y, void* stream);

/* Gradients of gdr_conv_fwd for dL/dy (d_y, dense [batch, seq_len, D]) and
 * dL/dfinal_state (NULL: zeros); the pre-activation is formed again.
 * dx [batch, seq_len, D] dense; dweight [D][W] and dbias [D] fp32 (dbias NULL:
 * skipped); d_initial_state [num_seqs][W-1][D] (NULL: skipped). */
gdr_status_t gdr_conv_bwd_workspace_size(const gdr_conv_problem_t* problem, size_t* bytes);
gdr_status_t gdr_conv_bwd(const gdr_conv_problem_t* problem, const void* x, const void* weight, const void* bias,
                          const void* initial_state, const int32_t* cu_seqlens_dev, const int32_t* cu_seqlens_host,
                          const void* d_y, const void* d_final_state, void* dx, float* dweight, float* dbias,
                          void* d_initial_state, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Selective state space scan with a diagonal transition per channel:
 *   delta_t = dt_t + dt_bias, or softplus(dt_t + dt_bias) when dt_softplus is set
 *   h_t[d][n] = exp(delta_t[d] A[d][n]) h_{t-1}[d][n] + delta_t[d] B_t[g][n] x_t[d]
 *   s_t[d] = sum_n C_t[g][n] h_t[d][n] + D[d] x_t[d],   y = s or s z / (1 + exp(-z))
 * with group g = d / (channels / groups).
 *   x, dt, z [batch, seq_len, channels] io_dtype (z NULL: no gate)
 *   B, C     [batch, seq_len, groups, state_dim] io_dtype
 *   A        [channels][state_dim], D, dt_bias [channels] or NULL: fp32
 *   state    [num_seqs][channels][state_dim] fp32
 * exp(delta A) is meant to be at most one; a growing state may overflow where
 * pieces of a sequence are joined although its running value does not, and an
 * infinite one become NaN there. A may be -inf: a step size above zero then
 * forgets the state, one of zero keeps it. An infinite delta x may give NaN in
 * y where the sum over the state would be infinite.
 */
typedef struct {
    int64_t batch, seq_len;
    int64_t x_stride, dt_stride, z_stride, b_stride, c_stride;   /* elements between tokens; fwd, bwd: below 2^22 */
    int32_t num_seqs;
    int32_t channels;       /* 1 to 2^22 - 1                                             */
    int32_t groups;         /* >= 1, divides channels                                    */
    int32_t state_dim;      /* 1 to 64                                                   */
    int32_t dt_softplus;    /* 0 or 1                                                    */
    int32_t io_dtype;       /* x, dt, z, B, C                                            */
    int32_t out_dtype;      /* y: io_dtype or GDR_F32                                    */
    int32_t dy_dtype;       /* backward: d_y, io_dtype or GDR_F32                        */
    int32_t grad_dtype;     /* backward: dx, ddt, dz, dB and dC, io_dtype or GDR_F32     */
    int32_t reserved;       /* 0                                                         */
} gdr_scan_problem_t;

/* initial_state NULL means zeros; final_state NULL is skipped (it may not
 * overlap initial_state). workspace: at least gdr_scan_fwd_workspace_size bytes,
 * which may be 0 (then NULL is taken). */
gdr_status_t gdr_scan_fwd_workspace_size(const gdr_scan_problem_t* problem, size_t* bytes);
gdr_status_t gdr_scan_fwd(const gdr_scan_problem_t* problem, const void* x, const void* dt, const float* A,
                          const void* B, const void* C, const float* D, const void* z, const float* dt_bias,
                          const float* initial_state, const int32_t* cu_seqlens_dev, const int32_t* cu_seqlens_host,
                          void* y, float* final_state, void* workspace, size_t workspace_bytes, void* stream);

/* One token of every sequence: batch = num_seqs rows, seq_len = 1. `state` is
 * read and then overwritten by the state after the token. */
gdr_status_t gdr_scan_step(const gdr_scan_problem_t* problem, const void* x, const void* dt, const float* A,
                           const void* B, const void* C, const float* D, const void* z, const float* dt_bias,
                           float* state, void* y, void* stream);

/* Gradients of gdr_scan_fwd for dL/dy (d_y, dense) and dL/dfinal_state (NULL:
 * zeros); the states are formed again.
 *   dx, ddt, dz [batch, seq_len, channels], dB, dC [batch, seq_len, groups, state_dim]: grad_dtype, dense
 *   dA [channels][state_dim], dD, ddt_bias [channels], d_initial_state: fp32
 * dz is written when z is given; dD, ddt_bias and d_initial_state may be NULL. */
gdr_status_t gdr_scan_bwd_workspace_size(const gdr_scan_problem_t* problem, size_t* bytes);
gdr_status_t gdr_scan_bwd(const gdr_scan_problem_t* problem, const void* x, const void* dt, const float* A,
                          const void* B, const void* C, const float* D, const void* z, const float* dt_bias,
                          const float* initial_state, const int32_t* cu_seqlens_dev, const int32_t* cu_seqlens_host,
                          const void* d_y, const float* d_final_state, void* dx, void* ddt, float* dA, void* dB,
                          void* dC, float* dD, void* dz, float* ddt_bias, float* d_initial_state, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * Layer norm over the last axis:
 *   y = (x - mean) rstd weight + bias,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
 *   x [rows, cols] io_dtype, row stride x_stride; weight, bias [cols] param_dtype or NULL
 *   y [rows, cols] out_dtype; mean, rstd [rows] fp32 (forward: NULL to skip)
 */
typedef struct {
    int64_t rows, x_stride;
    int32_t cols;           /* 1 to 16384                                                */
    float eps;              /* >= 0                                                      */
    int32_t io_dtype, param_dtype;
    int32_t out_dtype;      /* y: io_dtype or GDR_F32                                    */
    int32_t dy_dtype;       /* backward: d_y (dense), io_dtype or GDR_F32                */
    int32_t grad_dtype;     /* backward: dx (dense), io_dtype or GDR_F32                 */
    int32_t reserved;       /* 0                                                         */
} gdr_norm_problem_t;

gdr_status_t gdr_layer_norm_fwd(const gdr_norm_problem_t* problem, const void* x, const void* weight,
                                const void* bias, void* y, float* mean, float* rstd, void* stream);

/* dx = rstd (c - mean(c) - xhat mean(c xhat)) with c = d_y weight; dweight =
 * sum over rows of d_y xhat, dbias = sum of d_y, fp32 [cols] (NULL: skipped). */
gdr_status_t gdr_layer_norm_bwd_workspace_size(const gdr_norm_problem_t* problem, size_t* bytes);
gdr_status_t gdr_layer_norm_bwd(const gdr_norm_problem_t* problem, const void* x, const void* d_y,
                                const void* weight, const float* mean, const float* rstd, void* dx, float* dweight,
                                float* dbias, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_MIXER_H */

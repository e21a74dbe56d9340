/*
 * gdr_attn.h — C ABI of attention with a sliding window and a few first tokens
 * that stay visible (AMD MI355X, gfx950): the mixer that stands between layers
 * of the gated delta rule, with a state of bounded size like theirs.
 *
 *   prompts   gdr_window_attn_fwd     packed or batched sequences, from empty or filled caches
 *   decoding  gdr_window_attn_step    one token of every sequence
 *   training  gdr_window_attn_bwd     gradients of gdr_window_attn_fwd from empty caches
 *
 * The token at position p of its sequence sees the tokens j <= p with
 * p - j < window or j < sinks. For query head h and key head h / (Nq / Nk):
 *   s_pj = scale (q_p . k_j),   lse_p = log sum_j exp(s_pj),   o_p = sum_j exp(s_pj - lse_p) v_j
 *
 * Conventions are those of gdr_mixer.h: addresses need the alignment of their
 * element type only, tokens of q, k and v may be strided (the heads of a token
 * contiguous), outputs and caches are dense, sequences are packed by cu_seqlens,
 * the caller owns every buffer, sums run in a fixed order and the same call
 * gives the same bits. Scores, weights' sums and outputs are summed in fp32.
 * For bf16 inputs the weights exp(s - max) are rounded once to bf16 for their
 * product with v, as are the weights and their gradients in the backward pass.
 *
 * Cache. One of the keys and one of the values, io_dtype, each
 * [num_seqs][sinks + window][num_kv_heads][head_dim]: the token at position t
 * lies in row t if t < sinks, else in row sinks + (t - sinks) % window. lens
 * [num_seqs] (device, int32) are the tokens of each sequence before the call;
 * they are read only, so that the layers of a stack can share them, and the
 * caller advances them. lens + seq_len has to stay below 2^31 - 64; a value out of
 * range gives unspecified results, but every access stays in its buffer. Rows of a
 * cache that hold no visible token are never read into a result: they may hold
 * anything, NaN among it.
 *
 * NaN and Inf: a token's k and v reach the outputs of the tokens that see it and
 * no others; an infinite or NaN element of v may reach them as NaN in all of the
 * head's elements. In the backward pass they may reach all gradients of their
 * sequence and key head. Sequences do not touch
 * each other. A row whose scores are all -inf gives NaN.
 */
#ifndef GDR_ATTN_H
#define GDR_ATTN_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t batch, seq_len;                     /* tokens: batch * seq_len, below 2^31 - 64                */
    int64_t q_stride, k_stride, v_stride;       /* elements between tokens, below 2^22 (step: 2^40)        */
    int32_t num_seqs;                           /* batch, or len(cu_seqlens) - 1                           */
    int32_t num_q_heads, num_kv_heads;          /* Nq a multiple of Nk                                     */
    int32_t head_dim_qk, head_dim_v;            /* 1 to 128                                                */
    int32_t window;                             /* >= 1: tokens that a token sees, itself among them       */
    int32_t sinks;                              /* >= 0; sinks + window below 2^31                         */
    float scale;                                /* positive and finite                                     */
    int32_t io_dtype;                           /* q, k, v and the caches                                  */
    int32_t out_dtype;                          /* o: io_dtype or GDR_F32                                  */
    int32_t do_dtype;                           /* backward: d_o, io_dtype or GDR_F32                      */
    int32_t grad_dtype;                         /* backward: dq, dk and dv, io_dtype or GDR_F32            */
} gdr_attn_problem_t;

/* q [batch, seq_len, Nq, dk], k [batch, seq_len, Nk, dk], v [batch, seq_len, Nk, dv];
 * o [batch, seq_len, Nq, dv] dense; lse [batch, seq_len, Nq] fp32, natural
 * logarithm, or NULL. k_cache and v_cache NULL: the sequences begin here and
 * nothing is kept. Otherwise the tokens go on behind the cached ones (lens NULL:
 * none) and the caches are changed in place to hold the new ones. workspace: at
 * least gdr_window_attn_fwd_workspace_size bytes, which may be 0 (then NULL is taken). */
gdr_status_t gdr_window_attn_fwd_workspace_size(const gdr_attn_problem_t* problem, size_t* bytes);
gdr_status_t gdr_window_attn_fwd(const gdr_attn_problem_t* problem, const void* q, const void* k, const void* v,
                                 void* k_cache, void* v_cache, const int32_t* lens, const int32_t* cu_seqlens_dev,
                                 const int32_t* cu_seqlens_host, void* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* One token of every sequence: batch = num_seqs rows, seq_len = 1. The token is
 * written into the caches. A sequence whose lens is negative is passed over: its
 * caches stay as they are and its row of o is zero. */
gdr_status_t gdr_window_attn_step_workspace_size(const gdr_attn_problem_t* problem, size_t* bytes);
gdr_status_t gdr_window_attn_step(const gdr_attn_problem_t* problem, const void* q, const void* k, const void* v,
                                  void* k_cache, void* v_cache, const int32_t* lens, void* o, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Gradients of gdr_window_attn_fwd from empty caches, for dL/do (d_o, dense) and
 * the forward's o (out_dtype) and lse: dq, dk and dv dense like q, k and v. The
 * weights are exp(s - lse); of rows with |lse| beyond 1,024 ln 2, which fp32 holds
 * too coarsely for that, they are formed again from the scores. Below, the
 * rounding of lse leaves a weight within 2^-12 of itself. A d_o in fp32 beside bf16
 * inputs is rounded to bf16 first. The workspace holds 12 bytes a token and query
 * head, that rounded d_o, and with sinks, where there are more tokens than the
 * window, up to tokens / 256 + 2 num_seqs + 1 partial sums of
 * min(sinks, seq_len) x num_kv_heads x (head_dim_qk + head_dim_v) floats: gigabytes
 * for thousands of sinks. */
gdr_status_t gdr_window_attn_bwd_workspace_size(const gdr_attn_problem_t* problem, size_t* bytes);
gdr_status_t gdr_window_attn_bwd(const gdr_attn_problem_t* problem, const void* q, const void* k, const void* v,
                                 const void* o, const float* lse, const void* d_o, const int32_t* cu_seqlens_dev,
                                 const int32_t* cu_seqlens_host, void* dq, void* dk, void* dv, void* workspace,
                                 size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_ATTN_H */

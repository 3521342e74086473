/*
 * gla_scan.h -- gated linear attention (GLA) over whole sequences, forward
 * and backward, in libmbd_operators.so; the one-token step is gla_decode.h's (same
 * handle, same status codes, gemv.h).
 *
 * Operation, for each head of each sequence (S is dk x dv, t = 1 .. tokens):
 *
 *     S_t = diag(exp(gk_t)) S_{t-1} + outer(k_t, v_t)
 *     o_t = scale * q_t^T S_t
 *
 * -- gla_decode_step's step for every token; a forward call leaves the state
 * that gla_decode_step goes on from.  The backward call returns the gradients
 * of  sum(o . dout) + sum(S_T . dST)  in q, k, v, gk and S_0.
 *
 * Types: q, k, v, o and their gradients share one 16-bit dtype; gk and its
 * gradient have that dtype or float32 (gate_f32); states and their gradients
 * are float32, dense (sequence, head, dk, dv), the layout of gla_decode_step.
 * States and all sums are held in float32; each 16-bit output is rounded once,
 * to nearest-even.  Decayed q, k and dout, scores and states enter the products
 * with 16 bits (within 2^-17) where the result is rounded to 16 bits, with 24
 * where it goes into a state or the gates' gradient, which is a running sum over
 * the tokens (bf16 gates of bf16 tensors: 16 bits, half a bf16 step after some
 * 10^5 tokens).  Any gate is taken: one of -inf clears the state, positive ones
 * let it grow; a token's exp(gk) is a float32 (0 below -104, infinite above
 * 88.7), as in gla_decode_step, the decay over many tokens is not.  A value that
 * is not finite reaches the outputs that depend on it and no earlier token's (o)
 * or later token's (gradients of k and v); a state that holds one makes every
 * output that reads its row NaN or infinite.
 *
 * Layout: element strides per tensor, so (batch, token, head, channel) and
 * (batch, head, token, channel) tensors and slices of fused projections are
 * taken as they are; channels are dense.  Token strides are 0 < stride <=
 * 2^24 elements and at least the channels (a single token's is not used); an
 * input's batch and head strides may be 0 (a broadcast input: its gradient is
 * returned per head, unsummed).  An output's elements must not overlap each
 * other, another output or an input; the exception is ST == S0 (the state
 * updated in place).  16-bit tensors need 2-byte alignment, float32 ones
 * 4-byte alignment.
 *
 * Packed sequences: with `offsets` (device memory, batch + 1 ascending int32),
 * sequence i is rows offsets[i] .. offsets[i+1] - 1 of tensors with `rows`
 * rows (batch strides are ignored), and `tokens` is the longest sequence's
 * length; tokens beyond it are not processed.  Rows in no sequence are
 * neither read nor written; offsets outside [0, rows] are clamped into it,
 * so no row outside the tensors is touched.  An empty sequence leaves its
 * state as it was (ST = S0, dS0 = dST).
 *
 * Like gla_decode_step: host validation, kernels enqueued on `stream`, no
 * allocation, no synchronisation; on any error nothing is launched.  With
 * enough tokens for the heads at hand a sequence is split into segments that
 * run side by side, for which the caller brings scratch:
 * gla_scan_workspace_bytes says how much (possibly 0), any contents, 16-byte
 * aligned, not shared by calls that can overlap on the GPU.  Results do not
 * depend on timing.
 *
 * Limits (GEMV_ERR_TOO_LARGE): dk <= 256; dv <= 65536 forward, 256 backward;
 * tokens, rows <= 2^30; batch * heads <= 2^20, and times ceil(dv / 128) <= 2^23
 * forward; batch * tokens <= 2^34 unless packed.  batch, heads, dk or dv of 0 is
 * a no-op, as is tokens == 0 without ST / dS0.
 */
#ifndef MBD_GLA_SCAN_H
#define MBD_GLA_SCAN_H

#include "gemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element strides of a (batch, token, head, channel) tensor. */
typedef struct {
  int64_t batch, token, head;
} gla_stride_t;

typedef struct {
  int64_t batch, tokens, heads, dk, dv;
  gemv_dtype_t dtype;
  int32_t gate_f32;         /* gk and dgk: 0 = dtype, 1 = float32 */
  float scale;
  gla_stride_t q, k, v, gk;
  gla_stride_t o;           /* of o (forward), of dout (backward) */
  const int32_t* offsets;   /* packed sequences, or NULL */
  int64_t rows;             /* packed: rows of every tensor */
} gla_scan_t;

/* Strides of the gradients. */
typedef struct {
  gla_stride_t dq, dk, dv, dgk;
} gla_scan_grad_t;

/* Scratch a call on these sizes needs; 0 for sizes that are refused. */
size_t gla_scan_workspace_bytes(const gla_scan_t* p, int32_t backward);

/* S0 may be NULL (zeros) and ST may be NULL (not wanted). */
gemv_status_t gla_scan_forward(gemv_handle_t h, const gla_scan_t* p, const void* q, const void* k,
                               const void* v, const void* gk, const float* S0, float* ST, void* o,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/* S0, dST and dS0 may be NULL (zeros; zeros; not wanted). */
gemv_status_t gla_scan_backward(gemv_handle_t h, const gla_scan_t* p, const gla_scan_grad_t* grad,
                                const void* q, const void* k, const void* v, const void* gk,
                                const float* S0, const void* dout, const float* dST, void* dq,
                                void* dk, void* dv, void* dgk, float* dS0, void* workspace,
                                size_t workspace_bytes, hipStream_t stream);

/* The host checks of the two calls, in their order (no handle, no GPU). */
gemv_status_t gla_scan_check_args(const gla_scan_t* p, const void* q, const void* k, const void* v,
                                  const void* gk, const float* S0, const float* ST, const void* o,
                                  const void* workspace, size_t workspace_bytes);
gemv_status_t gla_scan_grad_check_args(const gla_scan_t* p, const gla_scan_grad_t* grad,
                                       const void* q, const void* k, const void* v, const void* gk,
                                       const float* S0, const void* dout, const float* dST,
                                       const void* dq, const void* dk, const void* dv,
                                       const void* dgk, const float* dS0, const void* workspace,
                                       size_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* MBD_GLA_SCAN_H */

/*
 * gemm.h -- dense product of many rows with a fused epilogue, in
 * libmbd_operators.so, on the GEMV's handle and with its status codes (gemv.h).
 *
 * Operation, for A (m, k) -- a row per token -- and B (n, k), the weights in
 * the GEMV's layout:
 *
 *     C[i][j] = act( alpha * scale_a[i] * scale_b[j] * sum_x A[i][x] B[j][x]
 *                    + bias[j] ) + residual[i][j]
 *
 * Types: A and B share one type, GEMM_F16, GEMM_BF16 or GEMM_E4M3 (OCP 8-bit
 * float: 4 exponent bits, no infinity, 0x7f and 0xff NaN).  C, bias and
 * residual are 16-bit, of A's type, or of either 16-bit type when A and B are
 * e4m3.  Scales are float32 and may come with every type.  Products are summed
 * in fp32 in an order fixed by the sizes and by whether all rows of A and B lie
 * on 16-byte boundaries; the epilogue is fp32 and rounds once, to nearest-even.
 * IEEE special values propagate.  One exception: the 8-bit matrix instructions
 * align 8 neighbouring products to the largest exponent among them and drop
 * bits below 2^-13 of it before the fp32 sum.
 *
 * Activations: none; relu (max(y, 0), NaN kept); gelu, y/2 erfc(-y/sqrt 2);
 * gelu_tanh, y/2 (1 + tanh(sqrt(2/pi) (y + 0.044715 y^3))); silu,
 * y / (1 + e^-y).
 *
 * Layout: row-major with leading dimensions lda, ldb >= k, ldc, ldr >= n, in
 * elements (that of a single row is not used, nor limited below); every tensor
 * needs the alignment of its element only (16-byte aligned rows are faster).  C
 * must not overlap anything else, except that residual may be C itself with
 * ldr == ldc.
 *
 * Like gemv_run: host validation, kernels enqueued on `stream`, no allocation,
 * no synchronisation; on any error nothing is launched.  m == 0 or n == 0 is a
 * no-op; with k == 0 the sum is 0 and A and B are not read.  Products of few
 * tiles with a long k split k over workgroups, for which the caller brings
 * scratch: gemm_workspace_bytes says how much (possibly 0), any contents,
 * 16-byte aligned, not shared by calls that can overlap on the GPU.
 *
 * Limits (GEMV_ERR_TOO_LARGE): m, n, k <= 2^30, m n <= 2^38, and n <= 2^28 for
 * up to 64 tokens; lda and ldb at most 2^23 bytes, ldc and ldr at most 2^30
 * elements; also where the tiles that are picked are more than a launch takes
 * (beyond 2^36 outputs at the least).
 */
#ifndef MBD_GEMM_H
#define MBD_GEMM_H

#include "gemv.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { GEMM_F16 = 0, GEMM_BF16 = 1, GEMM_E4M3 = 2 };
enum { GEMM_ACT_NONE = 0, GEMM_ACT_RELU = 1, GEMM_ACT_GELU = 2, GEMM_ACT_GELU_TANH = 3, GEMM_ACT_SILU = 4 };

typedef struct {
  int64_t m, n, k;
  int64_t lda, ldb, ldc, ldr;
  int32_t in_type;         /* GEMM_F16, GEMM_BF16, GEMM_E4M3: A and B */
  gemv_dtype_t dtype;      /* C, bias, residual */
  int32_t act;             /* GEMM_ACT_* */
  float alpha;
  const float* scale_a;    /* m values, or NULL */
  const float* scale_b;    /* n values, or NULL */
  const void* bias;        /* n values, or NULL */
  const void* residual;    /* (m, n), or NULL */
} gemm_t;

/* Scratch a call on these sizes needs; 0 for sizes that are refused. */
size_t gemm_workspace_bytes(const gemm_t* p);

gemv_status_t gemm_run(gemv_handle_t h, const gemm_t* p, const void* A, const void* B, void* C,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/* What gemm_run picks for a call, worked out on the host alone (no handle, no GPU);
 * of A and B only the alignment is looked at.  GEMV_ERR_INVALID_ARG without p or
 * out, gemm_run's statuses for sizes that it refuses, zeros where it does nothing. */
typedef struct {
  int32_t rows, tokens;    /* outputs per workgroup: rows of B x tokens */
  int32_t kind;            /* 0 few tokens, 1 tiles through registers, 2 tiles by loads into LDS */
  int32_t splits;          /* of k over workgroups */
} gemm_config_t;
gemv_status_t gemm_plan_config(const gemm_t* p, const void* A, const void* B, gemm_config_t* out);

/* The host checks of gemm_run, in its order (no handle, no GPU). */
gemv_status_t gemm_check_args(const gemm_t* p, const void* A, const void* B, const void* C,
                              const void* workspace, size_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* MBD_GEMM_H */

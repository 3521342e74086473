/*
 * rmsnorm.h -- root-mean-square norm with the residual's addition, in 16 bits
 * or in 8 bits with a scale per row, in libmbd_operators.so, on the GEMV's
 * handle and with its status codes (gemv.h).  Its 8-bit output and scales are the A
 * and scale_a of gemm_run (gemm.h).
 *
 * Operation, per row i of n channels:
 *
 *     s_ij = x_ij + residual_ij, rounded to the dtype (s = x without residual)
 *     y_ij = s_ij * rsqrt(mean_j(s_ij^2) + eps) * w_j
 *     16 bits:  out_ij = y_ij, rounded once
 *     8 bits:   scale_i = max_j |y_ij| / 448,  out_ij = e4m3(y_ij / scale_i)
 *
 * x, residual, w, s and a 16-bit y share one 16-bit dtype; sums and scales are
 * float32; roundings are to nearest-even.  e4m3 is the OCP 8-bit float with 448
 * its largest value.  A row of zeros has scale 0 and codes 0.  In 8 bits a row
 * with a NaN gets a NaN scale; elements that are infinite, whose y is NaN, get
 * the code NaN, and the maximum is taken over the others.
 *
 * Layout: rows of leading dimension >= n (that of a single row is not used),
 * channels dense; 2-byte alignment
 * (scales 4-byte) is enough, 16-byte aligned rows are faster.  sum_out may be
 * x or residual, a 16-bit y may be x, each with the same leading dimension;
 * other overlaps with an output are refused.
 *
 * Like gemv_run: host validation, one kernel enqueued on `stream`, no
 * allocation, no synchronisation; on any error nothing is launched.  m == 0
 * or n == 0 is a no-op.  Limits (GEMV_ERR_TOO_LARGE): m <= 2^21, n <= 2^24,
 * leading dimensions <= 2^30.
 */
#ifndef MBD_RMSNORM_H
#define MBD_RMSNORM_H

#include "gemv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t m, n;
  int64_t ldx, ldres, ldsum, ldy;
  gemv_dtype_t dtype;
  int32_t out_e4m3;    /* y: 0 = dtype, 1 = e4m3 with scales */
  float eps;
} rmsnorm_t;

/* residual, sum_out: NULL or (m, n); sum_out needs a residual.  scales: m
 * values with out_e4m3, else NULL. */
gemv_status_t rmsnorm_run(gemv_handle_t h, const rmsnorm_t* p, const void* x, const void* residual,
                          const void* w, void* sum_out, void* y, float* scales, hipStream_t stream);

/* The host checks of rmsnorm_run, in its order (no handle, no GPU). */
gemv_status_t rmsnorm_check_args(const rmsnorm_t* p, const void* x, const void* residual,
                                 const void* w, const void* sum_out, const void* y,
                                 const float* scales);

#ifdef __cplusplus
}
#endif

#endif /* MBD_RMSNORM_H */

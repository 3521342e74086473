/*
 * operators.h -- libmbd_operators.so: operators of gated-linear-attention
 * models around the GEMV and the one-token GLA step of libgemv.so.
 *
 *   gla_scan.h   the recurrence over whole sequences, forward and backward
 *   gemm.h       the dense product of many tokens with its epilogue
 *   rmsnorm.h    root-mean-square norm with the residual's addition, 16 or 8 bits
 *
 * They run on the handles that gemv_create (gemv.h, libgemv.so) makes, and
 * return its status codes.
 */
#ifndef MBD_OPERATORS_H
#define MBD_OPERATORS_H

#include "gemm.h"
#include "gla_scan.h"
#include "rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Set the kernels up on the handle's device (which must be current): what the
 * first call of an operator on a device otherwise does, some milliseconds.
 * Threads may call it, and operators, at once. */
gemv_status_t operators_prepare(gemv_handle_t h);

#ifdef __cplusplus
}
#endif

#endif /* MBD_OPERATORS_H */

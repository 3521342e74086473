"""MI355X-native dense GEMV, c = B @ a (fp16/bf16 in, fp32 sum).

The compute lives in libgemv.so (HIP kernels for gfx950 behind a C ABI,
include/gemv.h) and libmbd_operators.so (the operators around it,
include/operators.h); this package is their ctypes binding.
"""
from ._lib import (EXPORTS, GEMV_BF16, GEMV_F16, GEMV_OK, Gemv, GemvError, GlaDecode,
                   gemv_check_args, gla_check_args, gla_decode_step,
                   gemv_check_args_ex, gemv_create, gemv_destroy, gemv_force_config,
                   gemv_num_variants, gemv_plan_config, gemv_query_config, gemv_run,
                   gemv_run_ex, gemv_run_noalloc, gemv_run_ws, gemv_status_string, gemv_variant_info, load)
from ._operators import (GEMM_ACTS, GEMM_BF16, GEMM_E4M3, GEMM_F16, OPERATOR_EXPORTS, Gemm, GlaScan,
                         RmsNorm, gemm_check_args, gemm_config_t, gemm_plan_config, gemm_run, gemm_t, gemm_workspace_bytes,
                         gla_scan_backward, gla_scan_check_args, gla_scan_forward,
                         gla_scan_grad_check_args, gla_scan_grad_t, gla_scan_t,
                         gla_scan_workspace_bytes, gla_stride_t, operators_prepare, rmsnorm_check_args, rmsnorm_run,
                         rmsnorm_t)

__all__ = ["EXPORTS", "GEMV_BF16", "GEMV_F16", "GEMV_OK", "Gemv", "GemvError", "GlaDecode",
           "gla_check_args", "gla_decode_step", "gemv_check_args",
           "gemv_check_args_ex", "gemv_create", "gemv_destroy", "gemv_force_config",
           "gemv_num_variants", "gemv_plan_config", "gemv_query_config", "gemv_run", "gemv_run_ex",
           "gemv_run_noalloc", "gemv_run_ws",
           "gemv_status_string", "gemv_variant_info", "load",
           "GEMM_ACTS", "GEMM_BF16", "GEMM_E4M3", "GEMM_F16", "Gemm", "RmsNorm",
           "gemm_check_args", "gemm_config_t", "gemm_plan_config", "gemm_run", "gemm_t", "gemm_workspace_bytes", "rmsnorm_check_args",
           "rmsnorm_run", "rmsnorm_t", "OPERATOR_EXPORTS", "GlaScan", "gla_scan_backward", "gla_scan_check_args",
           "gla_scan_forward", "gla_scan_grad_check_args", "gla_scan_grad_t", "gla_scan_t",
           "gla_scan_workspace_bytes", "gla_stride_t", "operators_prepare"]

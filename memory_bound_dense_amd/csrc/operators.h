// Internal to libmbd_operators.so: what its operators share on the host.
#pragma once

#include "handle.h"

namespace mbd_host {

// Kernel attributes on the current device (kernels with more than the default
// 64 KiB of dynamic LDS).
bool scan_set_attributes();
bool gemm_set_attributes();

// The handle's device is current and its kernels are set up (once per device).
gemv_status_t ready(gemv_handle_t h, const char* what);

}  // namespace mbd_host

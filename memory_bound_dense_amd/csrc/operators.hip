// libmbd_operators.so: set-up shared by its operators (include/operators.h).
#include "../../include/operators.h"

#include <mutex>

#include "operators.h"

namespace {

constexpr int kMaxDevices = 64;
std::once_flag once[kMaxDevices];
bool good[kMaxDevices];

}  // namespace

gemv_status_t mbd_host::ready(gemv_handle_t h, const char* what) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return report(h, GEMV_ERR_HIP, "hipGetDevice");
  if (dev != h->device) return report(h, GEMV_ERR_WRONG_DEVICE, what);
  if (dev < 0 || dev >= kMaxDevices) return report(h, GEMV_ERR_UNSUPPORTED, what);
  std::call_once(once[dev], [dev] { good[dev] = scan_set_attributes() && gemm_set_attributes(); });
  return good[dev] ? GEMV_OK : report(h, GEMV_ERR_HIP, "hipFuncSetAttribute(max dynamic LDS)");
}

extern "C" gemv_status_t operators_prepare(gemv_handle_t h) {
  if (!h || h->magic != mbd_host::kMagic) return report(nullptr, GEMV_ERR_NULL_HANDLE, "operators_prepare");
  return mbd_host::ready(h, "operators_prepare");
}

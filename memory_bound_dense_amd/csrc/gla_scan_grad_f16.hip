// libmbd_operators.so: the f16 forms of scan_grad_kernel.
#include "gla_scan_table.h"

namespace mbd {

#define FORM(G32, N, REV) {&scan_grad_kernel<DT_F16, G32, N, 2, REV>, &scan_grad_kernel<DT_F16, G32, N, 4, REV>}
#define FORMS(G32, REV) {FORM(G32, 2, REV), FORM(G32, 4, REV), FORM(G32, 8, REV)}
extern const ScanForms kScanGradF16 = {{FORMS(false, false), FORMS(false, true)}, {FORMS(true, false), FORMS(true, true)}};

}  // namespace mbd

// libgemv.so, continued: the compiled forms of scan_grad_kernel for a segment's own state.
#include "gla_scan_table.h"

namespace mbd {

#define FORM(DT, N, REV) {&scan_grad_kernel<DT, N, 2, REV, false>, &scan_grad_kernel<DT, N, 4, REV, false>}
#define FORMS(DT, REV) {FORM(DT, 2, REV), FORM(DT, 4, REV), FORM(DT, 8, REV)}
const ScanFn kScanState[2][2][3][2] = {{FORMS(0, false), FORMS(0, true)}, {FORMS(1, false), FORMS(1, true)}};

}  // namespace mbd

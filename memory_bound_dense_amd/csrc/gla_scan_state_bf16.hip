// libmbd_operators.so: the bf16 forms of scan_grad_kernel that leave a segment's own state.
#include "gla_scan_table.h"

namespace mbd {

#define FORM(G32, N, REV) {&scan_grad_kernel<DT_BF16, G32, N, 2, REV, false>, &scan_grad_kernel<DT_BF16, G32, N, 4, REV, false>}
#define FORMS(G32, REV) {FORM(G32, 2, REV), FORM(G32, 4, REV), FORM(G32, 8, REV)}
extern const ScanForms kScanStateBf16 = {{FORMS(false, false), FORMS(false, true)}, {FORMS(true, false), FORMS(true, true)}};

}  // namespace mbd

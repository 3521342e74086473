// libmbd_operators.so: the f16 forms of scan_state_kernel.
#include "gla_scan_table.h"

namespace mbd {

#define FORM(G32, N) {&scan_state_kernel<DT_F16, G32, N, 2>, &scan_state_kernel<DT_F16, G32, N, 4>}
extern const StateForms kScanStateF16 = {{FORM(false, 2), FORM(false, 4), FORM(false, 8)},
                                         {FORM(true, 2), FORM(true, 4), FORM(true, 8)}};

}  // namespace mbd

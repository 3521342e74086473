// libgemv.so, continued: the compiled forms of scan_out_kernel.
#include "gla_scan_table.h"

namespace mbd {

#define FORM(DT, N, REV) {&scan_out_kernel<DT, N, 2, REV>, &scan_out_kernel<DT, N, 4, REV>}
#define FORMS(DT, REV) {FORM(DT, 2, REV), FORM(DT, 4, REV), FORM(DT, 8, REV)}
const ScanFn kScanOut[2][2][3][2] = {{FORMS(0, false), FORMS(0, true)}, {FORMS(1, false), FORMS(1, true)}};

}  // namespace mbd

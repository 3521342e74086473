// The compiled forms of the scan kernels, the table of each kernel and dtype in
// a source file of its own: [float32 gates][reversed][64, 128 or 256 channels]
// [2 or 4 waves].
#pragma once

#include "gla_scan_kernel.h"

namespace mbd {

using ScanFn = void (*)(const ScanArgs);
using ScanForms = ScanFn[2][2][3][2];
using StateFn = void (*)(const StateArgs);   // both directions in one
using StateForms = StateFn[2][3][2];
extern const ScanForms kScanOutF16, kScanOutBf16;       // channels: DK
extern const ScanForms kScanGradF16, kScanGradBf16;     // channels: DV
extern const StateForms kScanStateF16, kScanStateBf16;   // channels: DV

}  // namespace mbd

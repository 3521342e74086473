// The compiled forms of the scan kernels, each table in a source file of its
// own: [dtype][reversed][64, 128 or 256 channels][2 or 4 waves].
#pragma once

#include "gla_scan_kernel.h"

namespace mbd {

using ScanFn = void (*)(const ScanArgs);
extern const ScanFn kScanOut[2][2][3][2];     // channels: DK
extern const ScanFn kScanGrad[2][2][3][2];    // channels: DV
extern const ScanFn kScanState[2][2][3][2];   // channels: DV

}  // namespace mbd

// scan_f16.hip -- the gated linear recurrence, fp16 data.
#include "scan_kernels.h"
#include "scan_launch.h"

namespace lcv {
hipError_t launch_scan_fwd_f16(const ScanArgs& a, hipStream_t stream) { return scan_fwd<CT_F16>(a, stream); }
}  // namespace lcv

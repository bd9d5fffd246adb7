// scan_f32.hip -- the gated linear recurrence, fp32 data.
#include "scan_kernels.h"
#include "scan_launch.h"

namespace lcv {
hipError_t launch_scan_fwd_f32(const ScanArgs& a, hipStream_t stream) { return scan_fwd<CT_F32>(a, stream); }
}  // namespace lcv

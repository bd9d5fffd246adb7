// scan_f16.hip -- the gated linear recurrence and its gradients, fp16 data.
#include "scan_kernels.h"
#include "scan_launch.h"

namespace lcv {
hipError_t launch_scan_fwd_f16(const ScanArgs& a, hipStream_t stream) { return scan_fwd<CT_F16>(a, stream); }
hipError_t launch_scan_bwd_f16(const ScanArgs& a, hipStream_t stream) { return scan_bwd<CT_F16>(a, stream); }
}  // namespace lcv

// scan_grad_f32.hip -- the gradients of the gated linear recurrence, fp32 data.
#include "scan_kernels.h"
#include "scan_launch.h"

namespace lcv {
hipError_t launch_scan_bwd_f32(const ScanArgs& a, hipStream_t stream) { return scan_bwd<CT_F32>(a, stream); }
}  // namespace lcv

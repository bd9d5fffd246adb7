// scan_grad_bf16.hip -- the gradients of the gated linear recurrence, bf16 data.
#include "scan_kernels.h"
#include "scan_launch.h"

namespace lcv {
hipError_t launch_scan_bwd_bf16(const ScanArgs& a, hipStream_t stream) { return scan_bwd<CT_BF16>(a, stream); }
}  // namespace lcv

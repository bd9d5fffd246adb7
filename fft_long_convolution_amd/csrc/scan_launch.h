// scan_launch.h -- the recurrence's launchers by dtype, one source file each (scan_f32.hip, scan_f16.hip, scan_bf16.hip).
#pragma once
#include "block_kernels.h"

namespace lcv {

hipError_t launch_scan_fwd_f32(const ScanArgs& a, hipStream_t stream);
hipError_t launch_scan_fwd_f16(const ScanArgs& a, hipStream_t stream);
hipError_t launch_scan_fwd_bf16(const ScanArgs& a, hipStream_t stream);
hipError_t launch_scan_bwd_f32(const ScanArgs& a, hipStream_t stream);
hipError_t launch_scan_bwd_f16(const ScanArgs& a, hipStream_t stream);
hipError_t launch_scan_bwd_bf16(const ScanArgs& a, hipStream_t stream);

}  // namespace lcv

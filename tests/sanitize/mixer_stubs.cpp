// Host-only stand-ins for the mixer operators' launchers (see stubs.cpp): each returns an error.
#include "mixer_kernels.h"

namespace lcv {
#define LCV_STUB(sig) sig { return hipErrorInvalidValue; }
LCV_STUB(hipError_t launch_linattn(int, const LinJob&, hipStream_t))
LCV_STUB(hipError_t launch_linattn_step(int, const LinStepArgs&, hipStream_t))
LCV_STUB(hipError_t launch_linattn_tan(int, const LinTanArgs&, float*, hipStream_t))
LCV_STUB(hipError_t launch_head_sum(int, const HeadSumArgs&, hipStream_t))
LCV_STUB(hipError_t launch_copy_state(const float*, float*, int64_t, hipStream_t))
LCV_STUB(hipError_t launch_rotary(int, const RotaryArgs&, hipStream_t))
LCV_STUB(hipError_t launch_layernorm_fwd(int, const NormArgs&, hipStream_t))
LCV_STUB(hipError_t launch_layernorm_bwd(int, const NormArgs&, hipStream_t))
#undef LCV_STUB
}  // namespace lcv

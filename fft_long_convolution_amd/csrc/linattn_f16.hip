// linattn_f16.hip -- the chunk kernels of linear attention for f16 data.
#include "linattn_chunk.h"

namespace lcv {

hipError_t launch_linattn_f16(const LinJob& a, hipStream_t stream) { return launch_chunk_io<CT_F16>(a, stream); }

}  // namespace lcv

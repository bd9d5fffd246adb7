// linattn_f32.hip -- the chunk kernels of linear attention for f32 data.
#include "linattn_chunk.h"

namespace lcv {

hipError_t launch_linattn_f32(const LinJob& a, hipStream_t stream) { return launch_chunk_io<CT_F32>(a, stream); }

}  // namespace lcv

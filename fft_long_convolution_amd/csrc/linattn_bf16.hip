// linattn_bf16.hip -- the chunk kernels of linear attention for bf16 data.
#include "linattn_chunk.h"

namespace lcv {

hipError_t launch_linattn_bf16(const LinJob& a, hipStream_t stream) { return launch_chunk_io<CT_BF16>(a, stream); }

}  // namespace lcv

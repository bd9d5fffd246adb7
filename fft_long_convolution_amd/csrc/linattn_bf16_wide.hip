// linattn_bf16_wide.hip -- the chunk kernels of linear attention for bf16 data, 128 columns to a workgroup.
#include "linattn_chunk.h"

namespace lcv {

hipError_t launch_linattn_bf16_wide(const LinJob& a, hipStream_t stream) { return launch_chunk_nw<CT_BF16, 2>(a, stream); }

}  // namespace lcv

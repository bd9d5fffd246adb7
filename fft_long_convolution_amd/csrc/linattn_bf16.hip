// linattn_bf16.hip -- the chunk kernels of linear attention for bf16 data, 64 columns to a workgroup
// (128 in linattn_bf16_wide.hip: apart for the compiler's time only).
#include "linattn_chunk.h"

namespace lcv {

hipError_t launch_linattn_bf16(const LinJob& a, hipStream_t stream) {
    return a.nw == 1 ? launch_chunk_nw<CT_BF16, 1>(a, stream) : launch_linattn_bf16_wide(a, stream);
}

}  // namespace lcv

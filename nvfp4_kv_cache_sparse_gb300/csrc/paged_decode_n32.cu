// paged_decode_n32.cu -- the paged attention kernel for row tiles of 32 (a translation unit of its own,
// so that the row tile sizes compile side by side).
#include "paged_decode.cuh"

namespace nvfp4mla {

cudaError_t launch_paged_decode_n32(const PagedDecodeArgs& d, cudaStream_t stream) { return paged::launch_rows<32>(d, stream); }

}  // namespace nvfp4mla

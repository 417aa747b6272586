// paged_decode_n16.cu -- the paged attention kernel for row tiles of 16 (a translation unit of its own,
// so that the row tile sizes compile side by side).
#include "paged_decode.cuh"

namespace nvfp4mla {

cudaError_t launch_paged_decode_n16(const PagedDecodeArgs& d, cudaStream_t stream) { return paged::launch_rows<16>(d, stream); }

}  // namespace nvfp4mla

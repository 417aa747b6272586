// paged_decode_n64.cu -- the paged attention kernel for row tiles of 64 (a translation unit of its own,
// so that the row tile sizes compile side by side).
#include "paged_decode.cuh"

namespace nvfp4mla {

cudaError_t launch_paged_decode_n64(const PagedDecodeArgs& d, cudaStream_t stream) { return paged::launch_rows<64>(d, stream); }

}  // namespace nvfp4mla

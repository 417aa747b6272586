// paged_decode_pair.cu -- host side of attention over whole sequences for jobs of up to 128 query rows on a
// CTA pair (decode_pair.cuh with kPaged).
#include <cuda_runtime.h>

#include <cstdint>

#include "decode_pair.cuh"
#include "launch.h"

namespace nvfp4mla {

cudaError_t launch_paged_decode_pair(const PagedDecodeArgs& d, cudaStream_t stream) {
    using namespace pairdec;
    KernelArgs a = {};
    if (!encode_q_map(&a.qmap, d.q, static_cast<int64_t>(d.jobs.batch) * d.jobs.rows_per_seq)) return cudaErrorInvalidValue;
    a.cache = d.cache;
    a.splits = 1;
    a.sm_scale = d.sm_scale;
    a.sink = d.attn_sink;
    a.out = static_cast<__nv_bfloat16*>(d.out);
    a.lse = d.lse;
    a.part_out = d.part_out;
    a.part_lse = d.part_lse;
    a.status = d.dev_status;
    a.jobs = d.jobs;
    a.jobs.row_tiles = (a.jobs.rows_per_seq + 127) / 128;
    a.hdr = reinterpret_cast<int4*>(d.hdr);
    a.runs = d.ctas;
    const auto kernel = d.record_bytes == 432 ? decode_pair_kernel<432, false, true>
                        : d.block_scales      ? decode_pair_kernel<352, true, true>
                                              : decode_pair_kernel<352, false, true>;
    cudaError_t err = d.record_bytes == 432 ? prepare_kernel<432, false, true>()
                      : d.block_scales      ? prepare_kernel<352, true, true>()
                                            : prepare_kernel<352, false, true>();
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    // a pair per segment: at most one for each job and each cut (those behind the last one leave at once)
    cfg.gridDim = dim3(2u * (static_cast<unsigned>(d.jobs.batch) * static_cast<unsigned>(a.jobs.row_tiles) + static_cast<unsigned>(d.ctas)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = d.record_bytes == 432 ? kSmemAlloc<432> : kSmemAlloc<352>;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddepcontrol.wait
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, kernel, a);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace nvfp4mla

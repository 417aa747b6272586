// sparse_decode_pair.cu -- host side of the sparse MLA decode for 128 query heads on a CTA pair
// (decode_pair.cuh).
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "decode_pair.cuh"
#include "launch.h"

namespace nvfp4mla {

bool decode_pair_supported(const DecodeArgs& d) { return d.h_q == 128 && (d.record_bytes == 352 || d.record_bytes == 432); }

int decode_pair_keys_per_split(int topk, int splits) {
    const int per = (topk + splits - 1) / splits;
    return (per + pairdec::kTile - 1) / pairdec::kTile * pairdec::kTile;
}

// How many clusters of 2 * splits CTAs of this kernel variant fit on the current device at once
// (0: none), asked once per variant, split count and device.
int pair_clusters_fit(int record_bytes, bool block_scales, int splits) {
    using namespace pairdec;
    if (splits < 1 || splits > kMaxClusterSplits) return 0;
    static std::atomic<int> fits[3][kMaxClusterSplits + 1][8];   // 0 unknown, else 1 + clusters
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    const int variant = record_bytes == 432 ? 2 : block_scales ? 1 : 0;
    std::atomic<int>& known = fits[variant][splits][dev & 7];
    int state = known.load(std::memory_order_relaxed);
    if (state == 0) {
        const auto kernel = record_bytes == 432 ? decode_pair_kernel<432, false, false>
                            : block_scales      ? decode_pair_kernel<352, true, false>
                                                : decode_pair_kernel<352, false, false>;
        const cudaError_t err = record_bytes == 432 ? prepare_kernel<432, false, false>()
                                : block_scales      ? prepare_kernel<352, true, false>()
                                                    : prepare_kernel<352, false, false>();
        int clusters = 0;
        if (err == cudaSuccess) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2u * static_cast<unsigned>(splits));
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = record_bytes == 432 ? kSmemAlloc<432> : kSmemAlloc<352>;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2u * static_cast<unsigned>(splits);
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) clusters = 0;
        }
        (void)cudaGetLastError();
        state = 1 + (clusters > 0 ? clusters : 0);
        known.store(state, std::memory_order_relaxed);
    }
    return state - 1;
}

// All splits of a row in one cluster when there are 2-4 of them and such clusters fit on this
// GPU all at once (a second wave of large clusters would leave SMs idle): the kernel then merges
// them itself and no merge grid follows.
bool decode_pair_merges(const DecodeArgs& d) {
    if (!decode_pair_supported(d) || d.splits < 2 || d.splits > pairdec::kMaxClusterSplits) return false;
    return static_cast<int64_t>(pair_clusters_fit(d.record_bytes, d.block_scales, d.splits)) >= d.rows;
}

cudaError_t launch_decode_pair(const DecodeArgs& d, cudaStream_t stream, bool* merged) {
    using namespace pairdec;
    KernelArgs a;
    if (!encode_q_map(&a.qmap, d.q, static_cast<int64_t>(d.rows) * 128)) return cudaErrorInvalidValue;
    a.cache = d.cache;
    a.num_slots = d.num_slots;
    a.indices = d.indices;
    a.topk = d.topk;
    a.splits = d.splits;
    a.keys_per_split = decode_pair_keys_per_split(d.topk, d.splits);
    a.sm_scale = d.sm_scale;
    a.sink = d.attn_sink;
    a.out = static_cast<__nv_bfloat16*>(d.out);
    a.lse = d.lse;
    a.part_out = d.part_out;
    a.part_lse = d.part_lse;
    a.status = d.dev_status;
    const auto kernel = d.record_bytes == 432 ? decode_pair_kernel<432, false, false>
                        : d.block_scales      ? decode_pair_kernel<352, true, false>
                                              : decode_pair_kernel<352, false, false>;
    cudaError_t err = d.record_bytes == 432 ? prepare_kernel<432, false, false>()
                      : d.block_scales      ? prepare_kernel<352, true, false>()
                                            : prepare_kernel<352, false, false>();
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(d.rows) * static_cast<unsigned>(d.splits) * 2u);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = d.record_bytes == 432 ? kSmemAlloc<432> : kSmemAlloc<352>;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddepcontrol.wait
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    // All splits of a row in one cluster when there are 2-4 of them and such clusters fit on this
    // GPU: the kernel then merges them itself and no merge grid follows.
    a.merge = decode_pair_merges(d) ? 1 : 0;
    attr[1].val.clusterDim.x = a.merge ? 2u * static_cast<unsigned>(d.splits) : 2u;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    *merged = a.merge != 0;
    err = cudaLaunchKernelEx(&cfg, kernel, a);
    if (err == cudaSuccess) err = cudaGetLastError();
    return err;
}

}  // namespace nvfp4mla

// head_tiles.cuh -- what the kernels around the latent attention share (head_products.cu, paged_expand.cu,
// ragged_attention.cu): TMA tiles of [tokens, heads, dims] tensors, bounded waits with one abort flag per CTA,
// and stores of whole 32-byte sectors.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "dequant.cuh"
#include "sm103_ptx.cuh"

namespace nvfp4mla {
namespace tiles {

constexpr int kBox = 128 * 128;    // bytes of a box of 128 rows x 64 bf16 values, 128B swizzle

// TMA 3-D tiled load of the box at element coordinates (x, y, z); completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst_saddr, const void* tmap, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst_saddr),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// The same in a kernel whose tcgen05 instructions work on a CTA pair: `bar_cluster` is a barrier of either CTA, in the
// shared::cluster window.
__device__ __forceinline__ void tma_load_3d_cg2(uint32_t dst_saddr, const void* tmap, int32_t x, int32_t y, int32_t z, uint32_t bar_cluster) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst_saddr),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const void* tmap) { asm volatile("prefetch.tensormap [%0];" ::"l"(tmap) : "memory"); }

// TMA 3-D tiled store of a box from shared memory; rows outside the tensor are not written. One bulk group per call.
__device__ __forceinline__ void tma_store_3d(const void* tmap, int32_t x, int32_t y, int32_t z, uint32_t src_saddr) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(tmap), "r"(x), "r"(y), "r"(z),
                 "r"(src_saddr)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the latest kPending stores of this thread have read their shared memory / have been written.
template <int kPending>
__device__ __forceinline__ void tma_store_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A warp's 32 rows of 64 accumulator columns as a bf16 box with the 128B swizzle (4 KB, 1024-byte aligned).
__device__ __forceinline__ void stage_box(uint32_t tmem_addr, uint32_t saddr, int lane) {
    uint32_t v[64];
    tmem_ld32(tmem_addr, *reinterpret_cast<uint32_t(*)[32]>(v));
    tmem_ld32(tmem_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(__uint_as_float(v[8 * c + 2 * e]), __uint_as_float(v[8 * c + 2 * e + 1]));
        sts_u128(saddr + swz(lane, c), make_uint4(w[0], w[1], w[2], w[3]));
    }
}

// 32 bytes (a whole sector) to a 32-byte aligned address.
__device__ __forceinline__ void st_sector(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Sixteen fp32 values times f as bf16, one sector.
__device__ __forceinline__ void st_bf16x16(void* p, const uint32_t* v, float f) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(__uint_as_float(v[2 * e]) * f, __uint_as_float(v[2 * e + 1]) * f);
    st_sector(p, w);
}

__device__ __forceinline__ void give_up(uint32_t* abort, uint32_t* status) {
    if (atomicExch(abort, 1u) == 0u && status != nullptr) atomicOr(status, 0x4u);
}

// Bounded wait, for one thread or a whole warp; false after the limit, and soon after another warp gave up. kCluster: acquire at
// cluster scope, for barriers that the peer CTA arrives on.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_or_give_up(uint64_t* bar, uint32_t parity, uint32_t* abort, uint32_t* status) {
    auto poll = [&] { return kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (poll()) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
#pragma unroll 1
        for (int k = 0; k < 64; ++k)
            if (poll()) return true;
        if (*reinterpret_cast<volatile uint32_t*>(abort) != 0u) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            give_up(abort, status);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint32_t* abort, uint32_t* status) {
    return __all_sync(0xffffffffu, wait_or_give_up(bar, parity, abort, status));
}

// After a wait that gave up: time for the copies and products in flight before the CTA leaves.
__device__ __forceinline__ void let_copies_land() {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 5000000ull) __nanosleep(1000);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                   const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link).
inline EncodeTiledFn encode_tiled() {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// bf16 [outer, mid, inner] with the given strides (elements, multiples of 8), boxes of box_outer x box_mid x 64 values with the
// 128B swizzle. Places outside read zeros.
inline bool encode_map(CUtensorMap* map, const void* base, int64_t inner, int64_t mid, int64_t outer, int64_t mid_stride,
                       int64_t outer_stride, int box_mid, int box_outer) {
    const EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(mid), static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(mid_stride) * 2u, static_cast<cuuint64_t>(outer_stride) * 2u};
    const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_mid), static_cast<cuuint32_t>(box_outer)};
    const cuuint32_t steps[3] = {1u, 1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, steps,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Raises a kernel's dynamic shared memory limit once per device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit != 0 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    err = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

// Launch as a programmatic dependent of the work before it on the stream, in clusters of `cluster` CTAs.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, int smem, int cluster, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args...);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace tiles
}  // namespace nvfp4mla

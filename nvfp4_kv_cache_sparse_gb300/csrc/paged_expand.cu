// paged_expand.cu -- per-head keys and values of whole sequences from their NVFP4 records in pages.
//
//   kv[t, h, 0:256] = kv_b[h] c[t],   k_pe[t] = the record's RoPE dims
// c[t] being the dequantized latent (512) of token t of the batch, its sequences lying one behind the other. An e2m1 code times its
// e4m3 scale has six significant bits, so c is exact in bf16; the sums run in fp32 in tensor memory and are rounded to bf16 once.
//
// This is one product [tokens, 512] x [512, 256 heads] whose left side is gathered and dequantized on the way: 512 FLOP per
// byte written: the tensor cores bound it (1.91 PFLOP/s; whole lines written one behind the other reach 7.7 TB/s, half of that time). A CTA pair holds the latents of 256 tokens in shared memory (128 KB a CTA, dequantized
// once) and runs over heads: each CTA streams half of a head's weights (CTA 0 the key's 128 rows, CTA 1 the value's)
// through a ring, and every tcgen05.mma of M = 256, N = 256 works on both halves, which halves what a CTA has to
// read of the weights through L2 (one CTA alone: 32 MB for every 128 tokens at 128 heads, 15 TB/s). Accumulators of two heads alternate in
// tensor memory. Pairs take equal runs of (tile of 256 tokens, head), heads innermost, so that all work to the
// end, and the records of the next tile are loaded into registers while the last heads of this one still run.
// 30,626 tokens x 128 heads: 765 to 791 us, 1.30 to 1.34 PFLOP/s; 454 without the writes, 592 with all of them into 64 MB that stay in L2, the same with
// half the loads: the writes bound it, 512 bytes of a token 64 KB from the next one's (2.6 TB/s). 80,232 tokens x 16 heads: 216 to 235 us, 1.43 to
// 1.56 PFLOP/s.
#include "head_tiles.cuh"
#include "launch.h"

namespace nvfp4mla {
namespace {

using namespace tiles;

constexpr int kStages = 4;             // ring of weight boxes: 128 rows x 64 k
constexpr int kChunks = 8;             // K = 512 in steps of 64
constexpr int kOffA = 1024;
constexpr int kOffRing = kOffA + kChunks * kBox;
constexpr int kStage = 4096;           // a warp's 32 tokens x 64 columns on the way out, two of them a warp
constexpr int kOffStage = kOffRing + kStages * kBox;
constexpr int kSmem = kOffStage + 8 * kStage + 1024;
static_assert(kSmem <= 232448, "shared memory");
constexpr int kWarpLoad = 4, kWarpMma = 5, kWarpConvert = 6, kConvertWarps = 8;   // warps 0-3 read the accumulators out
constexpr int kThreads = 32 * (kWarpConvert + kConvertWarps);
constexpr int kTokens = 128 / (4 * kConvertWarps);   // tokens of a lane: eight lanes hold one, four a warp at a time
constexpr int kTmemCols = 512;

struct Ctl {
    uint64_t full[kStages];            // CTA 0: both CTAs' boxes landed
    uint64_t empty[kStages];           // multicast: the products have read both boxes
    uint64_t a_full;                   // CTA 0: 16 warps (8 a CTA) wrote a tile's latents
    uint64_t a_free;                   // multicast: no product reads the tile's latents any more
    uint64_t acc_full[2];              // multicast
    uint64_t acc_empty[2];             // CTA 0: 8 warps (4 a CTA)
    uint64_t drain;
    uint32_t tmem_base, abort;
};

struct KernelArgs {
    CUtensorMap w_map;                 // kv_b [heads, 256, 512], box 1 x 128 x 64
    CUtensorMap kv_map;                // kv [rows, heads, 256], box 32 x 1 x 64
    ExpandArgs p;
};

// What a lane holds of a token's record: word j of each 64-dim chunk and the scales of those words' blocks.
template <int R, bool kBlk>
struct Piece {
    uint32_t codes[8];
    uint4 scales[kBlk || R == 432 ? 2 : 1];
    uint4 rope;
    bool valid, outside;
};

template <int R, bool kBlk>
__device__ __forceinline__ Piece<R, kBlk> load_piece(const ExpandArgs& p, int64_t t, int64_t total, int j, bool rope) {
    Piece<R, kBlk> x;
    x.valid = t < total;
    x.outside = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.codes[i] = 0u;
#pragma unroll
    for (auto& s : x.scales) s = make_uint4(0u, 0u, 0u, 0u);
    x.rope = make_uint4(0u, 0u, 0u, 0u);
    if (!x.valid) return x;
    int lo = 0, hi = p.batch;          // starts[lo] <= t < starts[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.starts + mid) <= t) lo = mid;
        else hi = mid;
    }
    const int64_t pos = t - __ldg(p.starts + lo);
    int page = -1;
    if (pos >= 0 && (pos >> p.page_shift) < p.width) page = __ldg(p.page_table + lo * p.table_stride + (pos >> p.page_shift));
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
        x.outside = true;
        return x;
    }
    const int64_t slot = (static_cast<int64_t>(page) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
    const uint8_t* rec = p.cache + slot * R;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.codes[i] = __ldg(reinterpret_cast<const uint32_t*>(rec + 32 * i + 4 * j));
    if constexpr (R == 432 || kBlk) {
        const uint4* s = reinterpret_cast<const uint4*>(rec + (R == 432 ? 256 : 320));
        x.scales[0] = __ldg(s);
        x.scales[1] = __ldg(s + 1);
    } else {
        const uint2 s = __ldg(reinterpret_cast<const uint2*>(rec + 320 + 8 * (j >> 1)));
        x.scales[0].x = s.x;
        x.scales[0].y = s.y;
    }
    if (rope) {
        if constexpr (R == 432) {
            x.rope = __ldg(reinterpret_cast<const uint4*>(rec + 304 + 16 * j));
        } else {
            const uint2 r = __ldg(reinterpret_cast<const uint2*>(rec + 256 + 8 * j));
            x.rope.x = r.x;
            x.rope.y = r.y;
        }
    }
    return x;
}

// f16x2 -> bf16x2 (exact for the values that occur)
__device__ __forceinline__ uint32_t to_bf16x2(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_bf16x2(f.x, f.y);
}

// The lane's eight words as bf16 rows of the K-major tile: word j of chunk i is the 16-byte chunk j of row `row` in box i
// (the eight lanes of a token write eight different chunks: no bank conflicts).
template <int R, bool kBlk>
__device__ __forceinline__ void store_piece(const Piece<R, kBlk>& x, uint32_t a_base, int row, int j) {
    uint32_t sw[2];                    // byte i: the scale of word j of chunk i
    if constexpr (R == 432 || kBlk) {
        sw[0] = gather_byte4(x.scales[0], j >> 1);
        sw[1] = gather_byte4(x.scales[1], j >> 1);
    } else {
        sw[0] = x.scales[0].x;
        sw[1] = x.scales[0].y;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4 h = dq8(x.codes[i], scale_half2((sw[i >> 2] >> (8 * (i & 3))) & 0xFFu));
        sts_u128(a_base + i * kBox + swz(row, j), make_uint4(to_bf16x2(h.x), to_bf16x2(h.y), to_bf16x2(h.z), to_bf16x2(h.w)));
    }
}

template <int R, bool kBlk>
__global__ void __launch_bounds__(kThreads, 1) paged_expand_kernel(const __grid_constant__ KernelArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    Ctl* ctl = reinterpret_cast<Ctl*>(smem);
    const uint32_t sbase = smem_addr(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const ExpandArgs& p = a.p;
    if (warp == kWarpLoad && lane == 0) {
        prefetch_map(&a.w_map);
        prefetch_map(&a.kv_map);
        for (int i = 0; i < kStages; ++i) mbar_init(&ctl->full[i], 1), mbar_init(&ctl->empty[i], 1);
        mbar_init(&ctl->a_full, 2 * kConvertWarps), mbar_init(&ctl->a_free, 1);
        for (int i = 0; i < 2; ++i) mbar_init(&ctl->acc_full[i], 1), mbar_init(&ctl->acc_empty[i], 8);
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0u;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc_cg2(&ctl->tmem_base, kTmemCols);
        tmem_relinquish_cg2();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();                    // the peer's barriers are ready
    tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int64_t last = p.batch > 0 ? __ldg(p.starts + p.batch) : 0;
    const int64_t total = last < 0 ? 0 : last > p.rows ? p.rows : last;
    const int64_t units = ((total + 255) >> 8) * p.heads;
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int64_t u0 = units * pair / pairs;
    const int n_units = static_cast<int>(units * (pair + 1) / pairs - u0);
    int64_t tile = u0 / p.heads;
    int head = static_cast<int>(u0 - tile * p.heads);
    uint32_t* abort = &ctl->abort;
    uint32_t* status = p.status;

    if (warp == kWarpLoad) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int i = 0; i < n_units && ok; ++i) {
                for (int c = 0; c < kChunks; ++c) {
                    ok = wait_or_give_up(&ctl->empty[stage], phase, abort, status);
                    if (!ok) break;
                    if (rank == 0) mbar_arrive_expect_tx(&ctl->full[stage], 2 * kBox);
                    tma_load_3d_cg2(sbase + kOffRing + stage * kBox, &a.w_map, 64 * c, 128 * rank, head, mapa_shared(smem_addr(&ctl->full[stage]), 0));
                    if (++stage == kStages) stage = 0, phase ^= 1;
                }
                if (++head == p.heads) head = 0;
            }
            // The last boxes' arrivals: no barrier of the cluster orders what a commit sends to the other CTA, and it must not reach
            // this CTA's shared memory after the CTA has left. (They come with products that the epilogue waits for anyway.)
            bool landed = ok;
            for (int c = 0; c < kStages && landed; ++c) {
                landed = wait_or_give_up(&ctl->empty[stage], phase, abort, status);
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        if (rank == 0 && elect_one_in_warp()) {
            constexpr uint32_t idesc = idesc_bf16_f32(256, 256, false, false);
            const uint64_t a0 = sdesc_sw128(sbase + kOffA, 16, 1024), w0 = sdesc_sw128(sbase + kOffRing, 16, 1024);
            int stage = 0, tiles_seen = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int i = 0; i < n_units && ok; ++i) {
                if (i == 0 || head == 0) ok = wait_or_give_up<true>(&ctl->a_full, tiles_seen++ & 1, abort, status);
                const int buf = i & 1;
                if (ok) ok = wait_or_give_up<true>(&ctl->acc_empty[buf], ((i >> 1) & 1) ^ 1, abort, status);
                for (int c = 0; c < kChunks && ok; ++c) {
                    ok = wait_or_give_up<true>(&ctl->full[stage], phase, abort, status);
                    if (!ok) break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_ss_cg2(tmem + 256 * buf, a0 + static_cast<uint64_t>((c * kBox + ks * 32) >> 4),
                                   w0 + static_cast<uint64_t>((stage * kBox + ks * 32) >> 4), idesc, c > 0 || ks > 0 ? 1u : 0u);
                    mma_commit_cg2(&ctl->empty[stage], 0x3u);
                    if (++stage == kStages) stage = 0, phase ^= 1;
                }
                if (ok) mma_commit_cg2(&ctl->acc_full[buf], 0x3u);
                if (++head == p.heads) {
                    head = 0;
                    if (ok && i + 1 < n_units) mma_commit_cg2(&ctl->a_free, 0x3u);
                }
            }
            mma_commit_cg2(&ctl->drain, 0x1u);
            wait_or_give_up(&ctl->drain, 0, abort, status);
        }
        __syncwarp();
    } else if (warp < 4) {
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * warp) << 16);
        const uint32_t stage = sbase + kOffStage + 2 * warp * kStage;
        bool ok = true;
        for (int i = 0; i < n_units && ok; ++i) {
            const int buf = i & 1;
            const int64_t t0 = tile * 256 + 128 * rank + 32 * warp, t = t0 + lane;
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.kv) + (t * p.heads + head) * 256;
            ok = wait_warp(&ctl->acc_full[buf], (i >> 1) & 1, abort, status);
            if (!ok) break;
            tc_fence_after_sync();
            if (t0 + 32 <= total) {    // (the same for the whole warp)
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    const uint32_t box = stage + (c & 1) * kStage;
                    if (lane == 0) tma_store_wait_read<1>();     // the box before the last one has left
                    __syncwarp();
                    stage_box(lanes + 256 * buf + 64 * c, box, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) tma_store_3d(&a.kv_map, 64 * c, head, static_cast<int32_t>(t0), box);
                }
            } else if (t0 < total) {   // rows behind the last sequence stay as they were
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint32_t v[32];
                    tmem_ld32_wait(lanes + 256 * buf + 32 * c, v);
                    if (t < total) {
                        st_bf16x16(dst + 32 * c, v, 1.0f);
                        st_bf16x16(dst + 32 * c + 16, v + 16, 1.0f);
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_addr(&ctl->acc_empty[buf]), 0));
            if (++head == p.heads) head = 0, ++tile;
        }
        if (lane == 0) tma_store_wait();
        __syncwarp();
    } else {
        const int w = warp - kWarpConvert, j = lane & 7;
        bool ok = true;
        int done = 0;
        for (int k = 0; done < n_units && ok; ++k, ++tile) {
            const int here = min(p.heads - head, n_units - done);
            const bool rope = head == 0;   // the pair that has the tile's first head writes k_pe
            Piece<R, kBlk> x[kTokens];
            const int64_t t0 = tile * 256 + 128 * rank + 4 * kTokens * w + (lane >> 3);
            bool outside = false;
#pragma unroll
            for (int e = 0; e < kTokens; ++e) {
                x[e] = load_piece<R, kBlk>(p, t0 + 4 * e, total, j, rope);
                outside |= x[e].outside;
            }
            if (outside && rope && status != nullptr && j == 0) atomicOr(status, 0x2u);
            if (k > 0) ok = wait_warp(&ctl->a_free, (k - 1) & 1, abort, status);
            if (!ok) break;
#pragma unroll
            for (int e = 0; e < kTokens; ++e) store_piece<R, kBlk>(x[e], sbase + kOffA, 4 * kTokens * w + 4 * e + (lane >> 3), j);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_addr(&ctl->a_full), 0));
            if (rope) {
#pragma unroll
                for (int e = 0; e < kTokens; ++e) {
                    if (!x[e].valid) continue;
                    uint4 v = x[e].rope;
                    if constexpr (R == 352) {
                        const uint2 lo = e4m3x4_to_f16(v.x), hi = e4m3x4_to_f16(v.y);
                        v = make_uint4(to_bf16x2(lo.x), to_bf16x2(lo.y), to_bf16x2(hi.x), to_bf16x2(hi.y));
                    }
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k_pe) + (t0 + 4 * e) * 64 + 8 * j) = v;
                }
            }
            done += here;
            head = 0;
        }
    }
    tc_fence_before_sync();
    __syncwarp();
    if (*reinterpret_cast<volatile uint32_t*>(abort) != 0u) let_copies_land();
    cluster_sync();                    // no CTA leaves while the other's products may read its shared or tensor memory
    if (warp == kWarpMma) {
        tc_fence_after_sync();
        tmem_dealloc_cg2(tmem, kTmemCols);
    }
}

template <int R, bool kBlk>
cudaError_t launch_records(const KernelArgs& a, int sms, cudaStream_t stream) {
    const cudaError_t err = allow_smem<paged_expand_kernel<R, kBlk>>(kSmem);
    if (err != cudaSuccess) return err;
    const int64_t units = ((a.p.rows + 255) / 256) * a.p.heads;
    const int pairs = static_cast<int>(units < sms / 2 ? units : sms / 2);
    return launch_dependent(paged_expand_kernel<R, kBlk>, dim3(2 * pairs), kThreads, kSmem, 2, stream, a);
}

}  // namespace

cudaError_t launch_paged_expand(const ExpandArgs& p, int sms, cudaStream_t stream) {
    KernelArgs a;
    a.p = p;
    if (!encode_map(&a.w_map, p.kv_b, 512, 256, p.heads, p.w_row_stride, p.w_head_stride, 128, 1) ||
        !encode_map(&a.kv_map, p.kv, 256, p.heads, p.rows, 256, static_cast<int64_t>(p.heads) * 256, 1, 32))
        return cudaErrorInvalidValue;
    if (p.record_bytes == 432) return launch_records<432, false>(a, sms, stream);
    return p.block_scales ? launch_records<352, true>(a, sms, stream) : launch_records<352, false>(a, sms, stream);
}

}  // namespace nvfp4mla

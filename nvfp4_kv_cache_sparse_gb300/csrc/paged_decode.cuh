// paged_decode.cuh -- attention of each query over all tokens of its own sequence, read from NVFP4
// records (352 or 432 bytes) through a page table.
//
// What is computed. Sequence b has n = seq_lens[b] tokens; token p lies in slot
// page_table[b, p / page_size] * page_size + p % page_size. Its s_q queries are its last s_q tokens:
// query i has position n - s_q + i and attends the tokens j <= its position:
//     z_j = sm_scale * q[b,i,h,:] . K_j,   out = sum_j e^{z_j} V_j / (sum_j e^{z_j} + e^{sink_h}),
//     lse = ln sum_j e^{z_j},              V_j = K_j[0:512]
//
// Work split. The s_q * h_q query rows of a sequence lie one behind the other in q; N of them (16, 32
// or 64: the kernel's row tile) share every key that is dequantized, so a job is (sequence, row tile)
// and costs ceil(keys / 128) tiles of 128 keys. The tiles of all jobs, one job behind the other, are
// cut into as many equal runs as there are CTAs (one per SM), whatever the lengths are: the lengths
// are read on the device, so a captured call follows them. A job that lies in one run is finished by
// its CTA; the parts of a job that was cut go to the workspace (at most two per CTA, f16 outputs
// divided by their own sums, fp32 log-sum-exps) and a second kernel joins them.
//
// Contractions. As keys outnumber rows, both products have the keys or the value dims on the MMA's M
// side: S^T [128 keys x N] = K Q^T and O^T [512 dims x N] += V^T P^T (four M = 128 MMAs per 16
// keys). A record is dequantized once, into f16 (exact: an e2m1 x e4m3 product has few bits), and
// read twice: K-major as K, MN-major as V^T. The 64 RoPE dims of K come from tensor memory. Queries
// are f16 times a power of two per row (exact within 2^28 of the row's largest), scores fp32, P f16.
//
// Pipeline. Shared memory holds a ring of kRing blocks (128 keys x 128 dims, 32 KB); a block is
// filled by the converters, read by the QK MMAs, and freed by the PV MMAs of its tile. With a ring
// of more than four blocks the first blocks of tile i + 1 are converted and multiplied (into the
// other of two score buffers) while tile i is in its softmax.
//
// Softmax. A lazy reference maximum per row (log2 domain): P = 2^(z - m); a tile moves m only where
// some score exceeds m + 8. A softmax thread holds one key's scores of 16 or 32 rows; it writes P
// against the current references at once, the warps vote, and only where a reference has to move is
// O^T rescaled and the pass redone. Row sums stay in fp32 registers (a key lane's share each) and
// are added up across lanes at the end of a job.
//
// Masks. A key behind the sequence's end, in a page outside the pool, or with a NaN scale gets a zero
// row in shared memory (V and K share it, and 0 x NaN in PV would reach rows that do not see the
// key); P is 0 for a key that a row does not see and NaN for a NaN key that it sees.
//
// Every wait is bounded by time; on timeout the CTA sets NVFP4_MLA_DEV_TIMEOUT, stops issuing work,
// drains what it issued and returns.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "dequant.cuh"
#include "launch.h"
#include "sm103_ptx.cuh"

namespace nvfp4mla {
namespace paged {

constexpr int kTile = 128;                 // keys per tile (M of the QK MMAs)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <int N>
struct Shape {
    static constexpr int kSoft = N == 16 ? 4 : 8;        // softmax warps
    static constexpr int kConv = N == 64 ? 8 : 16;       // converter warps
    static constexpr int kKeys = 16 / kConv;             // keys of a converter thread
    static constexpr int kThreads = 32 * (kSoft + kConv + 1);
    static constexpr int kRpt = 4 * N / kSoft;           // rows of a softmax thread (it has one key)
    static constexpr int kRopeDims = 256 / kSoft;        // RoPE dims a softmax thread converts
    static constexpr int kRing = N == 16 ? 6 : N == 32 ? 5 : 4;
    static constexpr int kEarly = kRing - 4;             // blocks of the next tile that fit beside a whole tile
    // tensor memory columns: O^T four blocks, two score buffers, the RoPE rows of K
    static constexpr uint32_t kColO = 0, kColS = 4 * N, kColR = 6 * N;
    static constexpr int kTmemCols = N == 16 ? 128 : N == 32 ? 256 : 512;
    static_assert(6 * N + 32 <= kTmemCols, "tensor memory");
    // shared memory (offsets from a 1024-byte aligned base)
    static constexpr int kQBlk = N * 128;                // N rows x 64 dims
    static constexpr int kOffQ = 4096;
    static constexpr int kOffK = kOffQ + 9 * kQBlk;
    static constexpr int kOffP = kOffK + kRing * 32768;
    static constexpr int kSmemBytes = kOffP + N * 256;
    static constexpr int kSmemAlloc = kSmemBytes + 1024;
    static_assert(kSmemAlloc <= 232448, "shared memory");
    static_assert(kOffK % 1024 == 0 && kOffP % 1024 == 0, "operand alignment");
};
constexpr int kSubBlk = 16384;             // 128 keys x 64 dims
constexpr int kBlk = 32768;
constexpr int kOffCM = 256;                // float [N/2][4]: per row pair {ch_a, ch_b, -m_a, -m_b}
constexpr int kOffAlpha = 768;             // float [N]: rescale factors, then 1 / l
constexpr int kOffXmax = 1024;             // float [N][4]: per-row values of the four key quadrants
constexpr int kOffPos = 2048;              // int [N]: each row's position (its last visible key)
constexpr int kOffNan = 2304;              // uint8 [2][128]: keys with a NaN scale, by tile parity
constexpr int kOffScan = 2560;             // int64 [32]

struct __align__(8) Ctl {
    uint64_t qload;           // q boxes landed (TMA, tx-counted)
    uint64_t qready;          // softmax warps: q converted in shared memory
    uint64_t kfull[6];        // converter warps: a ring block is written
    uint64_t kfree[6];        // PV commit: a ring block has been read
    uint64_t ropefull;        // softmax warps: RoPE rows of the tile in tensor memory
    uint64_t sfull;           // QK commit: S^T ready (every earlier MMA completed too)
    uint64_t pfull;           // softmax warps: P^T written (and O^T rescaled)
    uint64_t drain;           // every MMA issued completed
    int64_t total;            // tiles of all jobs
    uint32_t tmem_base;
    uint32_t abort;
    int32_t job0, tile0;      // where this CTA's run begins
};
static_assert(sizeof(Ctl) <= kOffCM, "control block");

struct KernelArgs {
    CUtensorMap qmap;         // q as bf16 [batch * s_q * h_q, 576], box 64 dims x N rows, 128B swizzle
    const uint8_t* cache;
    const int32_t* page_table;
    int64_t table_stride;
    const int32_t* seq_lens;
    int num_pages;            // pages of the pool
    int page_shift;
    int capacity;             // tokens that a page table row can name
    int batch, s_q, h_q;
    int rows_per_seq;         // s_q * h_q
    int row_tiles;            // ceil(rows_per_seq / N)
    float sm_scale;
    const float* sink;
    __nv_bfloat16* out;       // [batch * rows_per_seq, 512]
    float* lse;
    uint16_t* part_out;       // f16 [2 * CTAs, N, 512]
    float* part_lse;          // [2 * CTAs, N], log2 domain
    int4* hdr;                // [CTAs]: the cut job that begins in the CTA's run: first output row, rows,
                              // last CTA with a part of it, first head; rows 0: none
    uint32_t* status;
};

struct Job {
    int seq, row0, rows;      // rows row0 .. row0 + rows - 1 of sequence seq
    int keys;                 // keys that some of them sees
    int tiles;
    int first_pos, first_tok; // position and token of row row0
};

template <int N>
__device__ __forceinline__ Job job_info(const KernelArgs& a, int job) {
    Job j;
    j.seq = job / a.row_tiles;
    j.row0 = (job - j.seq * a.row_tiles) * N;
    j.rows = min(N, a.rows_per_seq - j.row0);
    const int len = min(max(__ldg(a.seq_lens + j.seq), 0), a.capacity);
    const int last_tok = (j.row0 + j.rows - 1) / a.h_q;
    j.first_tok = j.row0 / a.h_q;
    j.keys = max(0, len - a.s_q + last_tok + 1);
    j.tiles = (j.keys + kTile - 1) / kTile;
    j.first_pos = len - a.s_q + j.first_tok;
    return j;
}

// A position in the run of tiles of a CTA.
template <int N>
struct Walk {
    Job j;
    int job, t, left;         // tile t of the job; tiles left in the run, this one included
    __device__ __forceinline__ void start(const KernelArgs& a, int job0, int tile0, int count) {
        job = job0;
        t = tile0;
        left = count;
        j = job_info<N>(a, job);
    }
    __device__ __forceinline__ void next(const KernelArgs& a) {
        if (left <= 1) {
            left = 0;
            return;
        }
        --left;
        if (++t < j.tiles) return;
        do j = job_info<N>(a, ++job);
        while (j.tiles == 0);
        t = 0;
    }
    __device__ __forceinline__ bool last_of_segment() const { return left == 1 || t == j.tiles - 1; }
    // byte offset of the record of key `key` (0..127) of the tile; -1: none, -2: its page is outside the pool
    template <int R>
    __device__ __forceinline__ int64_t record(const KernelArgs& a, int key) const {
        const int pos = kTile * t + key;
        if (left <= 0 || pos >= j.keys) return -1;
        const int page = __ldg(a.page_table + j.seq * a.table_stride + (pos >> a.page_shift));
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.num_pages)) return -2;
        return ((static_cast<int64_t>(page) << a.page_shift) + (pos & ((1 << a.page_shift) - 1))) * R;
    }
};

__device__ __forceinline__ void set_abort(Ctl* ctl, uint32_t* status) {
    if (atomicExch(&ctl->abort, 1u) == 0u && status != nullptr) atomicOr(status, 0x4u);
}
__device__ __forceinline__ bool aborted(Ctl* ctl) { return *reinterpret_cast<volatile uint32_t*>(&ctl->abort) != 0u; }

// Bounded wait, one answer per warp.
__device__ __forceinline__ bool wait_warp(Ctl* ctl, uint64_t* bar, uint32_t parity, uint32_t* status) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok && !aborted(ctl)) {
        ok = mbar_wait(bar, parity);
        if (!ok) set_abort(ctl, status);
    }
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float lds_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts_f32(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ void sts_u16(uint32_t a, uint16_t v) { asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v) : "memory"); }
__device__ __forceinline__ void sts_u8(uint32_t a, uint32_t v) { asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// Starts bringing `bytes` (a multiple of 16, from a 16-byte boundary) into L2.
__device__ __forceinline__ void prefetch_l2_bulk(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// Whether one of the four bytes is an e4m3 NaN (0x7F or 0xFF).
__device__ __forceinline__ bool has_nan_e4m3(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u; }

template <int R, bool kBlkOrder, int N>
__global__ void __launch_bounds__(Shape<N>::kThreads, 1) paged_decode_kernel(const __grid_constant__ KernelArgs a) {
    using S = Shape<N>;
    constexpr int kSoftThreads = 32 * S::kSoft;
    constexpr int kWarpMma = S::kSoft + S::kConv;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    Ctl* ctl = reinterpret_cast<Ctl*>(smem);
    const uint32_t sbase = smem_addr(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(&ctl->qload, 1);
        mbar_init(&ctl->qready, S::kSoft);
        for (int s = 0; s < S::kRing; ++s) {
            mbar_init(&ctl->kfull[s], S::kConv);
            mbar_init(&ctl->kfree[s], 1);
        }
        mbar_init(&ctl->ropefull, S::kSoft);
        mbar_init(&ctl->sfull, 1);
        mbar_init(&ctl->pfull, S::kSoft);
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0u;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(&ctl->tmem_base, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;
    // Launched as a programmatic dependent of the preceding kernel: nothing is read before that grid
    // has completed and its writes are visible.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    // ---- the run of this CTA: a prefix sum over the jobs' tiles, a contiguous piece of the jobs per thread
    const int jobs = a.batch * a.row_tiles;
    int count = 0;
    {
        const int per = (jobs + S::kThreads - 1) / S::kThreads;
        const int ja = min(jobs, static_cast<int>(threadIdx.x) * per), jb = min(jobs, ja + per);
        int64_t mine = 0;
        for (int j = ja; j < jb; ++j) mine += job_info<N>(a, j).tiles;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        int64_t* scan = reinterpret_cast<int64_t*>(smem + kOffScan);
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        int64_t total = 0, before = incl - mine;
        for (int w = 0; w < S::kThreads / 32; ++w) {
            const int64_t v = scan[w];
            if (w < warp) before += v;
            total += v;
        }
        const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
        const int64_t c = blockIdx.x;
        if (c < ctas) {
            const int64_t g0 = total * c / ctas;
            count = static_cast<int>(total * (c + 1) / ctas - g0);
            if (before <= g0 && g0 < before + mine) {
                int64_t at = before;
                int j = ja;
                for (;; ++j) {
                    const int nt = job_info<N>(a, j).tiles;
                    if (g0 < at + nt) break;
                    at += nt;
                }
                ctl->job0 = j;
                ctl->tile0 = static_cast<int>(g0 - at);
            }
        }
        if (threadIdx.x == 0) ctl->total = total;
        __syncthreads();
    }
    // ---- jobs without a visible key: out = 0, lse = -inf
    for (int job = blockIdx.x; job < jobs; job += gridDim.x) {
        const Job j = job_info<N>(a, job);
        if (j.tiles > 0) continue;
        const int64_t row = static_cast<int64_t>(j.seq) * a.rows_per_seq + j.row0;
        uint4* o = reinterpret_cast<uint4*>(a.out + row * 512);
        for (int e = threadIdx.x; e < j.rows * 64; e += S::kThreads) o[e] = make_uint4(0u, 0u, 0u, 0u);
        for (int e = threadIdx.x; e < j.rows; e += S::kThreads) a.lse[row + e] = -INFINITY;
    }
    if (blockIdx.x == 0 && a.status != nullptr)
        for (int b = threadIdx.x; b < a.batch; b += S::kThreads)
            if (__ldg(a.seq_lens + b) > a.capacity) atomicOr(a.status, 0x2u);
    if (threadIdx.x == 0 && count == 0) a.hdr[blockIdx.x] = make_int4(0, 0, 0, 0);

    if (count == 0) {
        // nothing to do in this CTA
    } else if (warp < S::kSoft) {
        // ======================= softmax warps =======================
        const int qd = warp & 3;              // TMEM lane quadrant: keys 32 qd.. of a tile
        const int h2 = warp >> 2;
        const int key = 32 * qd + lane;
        const int rb = S::kRpt * h2;          // rows rb .. rb + kRpt - 1
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * qd) << 16);
        const uint32_t cm_s = sbase + kOffCM;
        const uint32_t alpha_s = sbase + kOffAlpha;
        const uint32_t xmax_s = sbase + kOffXmax;
        const uint32_t pos_s = sbase + kOffPos;
        auto ch_addr = [&](int r) { return cm_s + 16 * (r >> 1) + 4 * (r & 1); };
        auto negm_addr = [&](int r) { return cm_s + 16 * (r >> 1) + 8 + 4 * (r & 1); };

        constexpr int kRopeVec = S::kRopeDims * (R == 352 ? 1 : 2) / 16;
        uint4 rope[kRopeVec];
        auto load_rope = [&](int64_t off) {
            if (off >= 0) {
                const uint8_t* src = a.cache + off + (R == 352 ? 256 : 304) + h2 * (16 * kRopeVec);
#pragma unroll
                for (int e = 0; e < kRopeVec; ++e) rope[e] = ldg_stream16(src + 16 * e);
            }
        };
        // the RoPE dims of this key into tensor memory; zero for a key that is not there
        auto store_rope = [&](bool there) {
#pragma unroll
            for (int part = 0; part < S::kRopeDims / 32; ++part) {
                uint32_t v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = 0u;
                if (there) {
                    if constexpr (R == 352) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint4 x = rope[2 * part + e];
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const uint2 f = e4m3x4_to_f16(w[m]);
                                v[8 * e + 2 * m] = f.x;
                                v[8 * e + 2 * m + 1] = f.y;
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint4 x = rope[4 * part + e];
                            v[4 * e] = x.x;
                            v[4 * e + 1] = x.y;
                            v[4 * e + 2] = x.z;
                            v[4 * e + 3] = x.w;
                        }
                    }
                }
                tmem_st16(lane_base + S::kColR + (S::kRopeDims / 2) * h2 + 16 * part, v);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->ropefull);
        };

        bool ok = true;
        // q of a job's rows into shared memory (TMA); rows behind the sequence's last one are those of the
        // next sequence or zeros, and reach columns that nothing reads
        auto load_q = [&](const Job& j) {
            if (threadIdx.x == 0) {
                mbar_arrive_expect_tx(&ctl->qload, 9u * S::kQBlk);
                for (int bx = 0; bx < 9; ++bx)
                    tma_load_2d(sbase + S::kOffQ + bx * S::kQBlk, &a.qmap, 64 * bx, j.seq * a.rows_per_seq + j.row0, &ctl->qload);
            }
        };
        // per-row prescale and f16 (bf16 RoPE for 432-byte records) in place; the rows' scales and positions
        auto stage_q = [&](const Job& j, int seg) {
            constexpr int kTpr = kSoftThreads / N, kChunks = 72 / kTpr;   // threads of a row, chunks of 8 dims of a thread
            if (ok) ok = wait_warp(ctl, &ctl->qload, seg & 1, a.status);
            const int r = threadIdx.x / kTpr, part = threadIdx.x % kTpr;
            float qmax = 0.0f;
            if (ok) {
#pragma unroll 3
                for (int k = kChunks * part; k < kChunks * part + kChunks; ++k) {
                    const uint4 x = lds_u128(sbase + S::kOffQ + (k >> 3) * S::kQBlk + swz(r, k & 7));
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        qmax = fmax3(qmax, fabsf(__uint_as_float(w[m] << 16)), fabsf(__uint_as_float(w[m] & 0xFFFF0000u)));
                }
            }
#pragma unroll
            for (int o = 1; o < kTpr; o <<= 1) qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, o));
            int pre = 0;
            if (qmax > 0.0f) {
                const int e = static_cast<int>(__float_as_uint(qmax) >> 23) - 126;   // qmax < 2^e
                pre = min(113, max(-113, 15 - e));
            }
            const float fpre = __int_as_float((127 + pre) << 23);
            if (part == 0) {
                // S' = 2^pre S and z = ch S'; a row that does not exist scores 0 throughout
                sts_f32(ch_addr(r), r < j.rows ? a.sm_scale * kLog2e * __int_as_float((127 - pre) << 23) : 0.0f);
                sts_f32(negm_addr(r), INFINITY);   // reference maximum -inf
                const int tok = (j.row0 + min(r, j.rows - 1)) / a.h_q;
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(pos_s + 4 * r), "r"(j.first_pos + tok - j.first_tok) : "memory");
            }
            if (ok) {
#pragma unroll 3
                for (int k = kChunks * part; k < kChunks * part + kChunks; ++k) {
                    const bool bf = R == 432 && k >= 64;   // bf16 RoPE of 432-byte records
                    const uint32_t addr = sbase + S::kOffQ + (k >> 3) * S::kQBlk + swz(r, k & 7);
                    const uint4 x = lds_u128(addr);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    uint32_t y[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const float lo = __uint_as_float(w[m] << 16) * fpre, hi = __uint_as_float(w[m] & 0xFFFF0000u) * fpre;
                        y[m] = bf ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
                    }
                    sts_u128(addr, make_uint4(y[0], y[1], y[2], y[3]));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->qready);
            named_bar_sync(1, kSoftThreads);   // the rows' scales, references and positions are written
        };

        Walk<N> cur, ahead;
        cur.start(a, ctl->job0, ctl->tile0, count);
        ahead = cur;
        load_q(cur.j);
        int64_t off = ahead.template record<R>(a, key);
        load_rope(off);
        ahead.next(a);
        int64_t off_n = ahead.template record<R>(a, key);
        int seg = 0;
        stage_q(cur.j, seg);
        store_rope(off >= 0);
        bool seg_first = true;
        int seg_tile = cur.t;                  // the segment's first tile
        float l[S::kRpt];                      // this key lane's share of each row's sum of 2^(z - m)
#pragma unroll
        for (int e = 0; e < S::kRpt; ++e) l[e] = 0.0f;
        int4 hdr = make_int4(0, 0, 0, 0);

        // P^T in shared memory. N = 64: row = key, 64 rows of the tile across (MN-major B operand); N = 16, 32:
        // row = query row, 64 keys across, twice (K-major B operand)
        const uint32_t p_key = N == 64 ? sbase + S::kOffP + (key >> 3) * 1024 + (key & 7) * 128
                                       : sbase + S::kOffP + (key >> 6) * (N * 128) + (key & 7) * 2;
        const uint32_t p_chunk = static_cast<uint32_t>((key & 63) >> 3) << 4;

        // Every softmax warp takes part in every named barrier below, also after a wait ran out (then it only
        // passes the barriers), so no warp can be left waiting on a missing one. Tensor-memory loads and stores
        // are warp-collective: masks change values only.
        for (int it = 0; it < count; ++it) {
            if (it + 1 < count) load_rope(off_n);   // in flight while this tile is scored
            ahead.next(a);
            const int64_t off_n2 = ahead.template record<R>(a, key);
            const bool there = off >= 0;
            const int pos = kTile * cur.t + key;
            const bool full = kTile * cur.t + kTile - 1 <= cur.j.first_pos;   // every row sees every key of the tile
            const uint32_t s_col = lane_base + S::kColS + N * (it & 1) + rb;
            float ln[S::kRpt];
            float nan_add = 0.0f;
            // one pass over this key's scores: P (against the current references), the sums, the largest z - m
            auto score = [&]() -> float {
                float tmax = -INFINITY;
#pragma unroll
                for (int part = 0; part < S::kRpt / 16; ++part) {
                    uint32_t sv[16];
                    tmem_ld16(s_col + 16 * part, sv);
                    tmem_wait_ld();
#pragma unroll
                    for (int c2 = 0; c2 < 2; ++c2) {
                        uint32_t pw[4];
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const int e = 8 * c2 + 2 * g, r = 16 * part + e;   // rows rb + r, rb + r + 1
                            const uint4 c = lds_u128(cm_s + 8 * (rb + r));
                            uint64_t z2 = f32x2_fma(f32x2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])),
                                                    f32x2_pack(__uint_as_float(c.x), __uint_as_float(c.y)),
                                                    f32x2_pack(__uint_as_float(c.z), __uint_as_float(c.w)));
                            z2 = f32x2_add(z2, f32x2_pack(nan_add, nan_add));
                            const float2 z = f32x2_unpack(z2);
                            bool v0 = there, v1 = there;
                            if (!full) {
                                const uint2 qp = lds_u64(pos_s + 4 * (rb + r));
                                v0 = there && pos <= static_cast<int>(qp.x);
                                v1 = there && pos <= static_cast<int>(qp.y);
                            }
                            tmax = fmax3(tmax, v0 ? z.x : -INFINITY, v1 ? z.y : -INFINITY);
                            const float p0 = v0 ? ex2_approx(z.x) : 0.0f, p1 = v1 ? ex2_approx(z.y) : 0.0f;
                            ln[r] = l[r] + p0;
                            ln[r + 1] = l[r + 1] + p1;
                            pw[g] = pack_f16x2(p0, p1);
                            if constexpr (N != 64) {
                                const int rr = S::kRpt * h2 + r;
                                const uint32_t base = p_key + static_cast<uint32_t>((rr >> 3) * 1024 + (rr & 7) * 128);
                                sts_u16(base + (p_chunk ^ ((rr & 7) << 4)), static_cast<uint16_t>(pw[g]));
                                sts_u16(base + 128 + (p_chunk ^ (((rr & 7) + 1) << 4)), static_cast<uint16_t>(pw[g] >> 16));
                            }
                        }
                        if constexpr (N == 64)
                            sts_u128(p_key + (((4 * h2 + 2 * part + c2) ^ (key & 7)) << 4), make_uint4(pw[0], pw[1], pw[2], pw[3]));
                    }
                }
                return tmax;
            };
            float tmax = -INFINITY;
            if (ok) ok = wait_warp(ctl, &ctl->kfull[(4 * it) % S::kRing], (4 * it / S::kRing) & 1, a.status);
            if (ok) ok = wait_warp(ctl, &ctl->sfull, it & 1, a.status);
            if (ok) {
                tc_fence_after_sync();
                if (lds_u8(sbase + kOffNan + 128 * (it & 1) + key) != 0u) nan_add = NAN;
                tmax = score();
            }
            // ---- does any row need a new reference? (one barrier reduction)
            if (bar_red_or(1, kSoftThreads, tmax > kRescaleThreshold)) {
                // per row: the tile's largest z over the 128 keys (warp maximum, then the four quadrants)
                float mine = -INFINITY;
#pragma unroll
                for (int part = 0; part < S::kRpt / 16; ++part) {
                    uint32_t sv[16];
                    if (ok) {
                        tmem_ld16(s_col + 16 * part, sv);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int r = rb + 16 * part + e;
                        bool v = ok && there;
                        if (!full) v = v && pos <= static_cast<int>(lds_u32(pos_s + 4 * r));
                        const float wm = warp_max(v ? __uint_as_float(sv[e]) * lds_f32(ch_addr(r)) : -INFINITY);
                        if (lane == 16 * part + e) mine = wm;
                    }
                }
                if (lane < S::kRpt) sts_f32(xmax_s + 16 * (rb + lane) + 4 * qd, mine);
                named_bar_sync(1, kSoftThreads);
                if (qd == 0 && lane < S::kRpt) {   // one thread per row: the new reference and the rescale factor
                    const uint4 x = lds_u128(xmax_s + 16 * (rb + lane));
                    const float zt = fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)),
                                           fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
                    const float mo = -lds_f32(negm_addr(rb + lane));
                    float al = 1.0f;
                    if (zt > mo + kRescaleThreshold) {
                        al = mo == -INFINITY ? 0.0f : ex2_approx(mo - zt);
                        sts_f32(negm_addr(rb + lane), -zt);
                    }
                    sts_f32(alpha_s + 4 * (rb + lane), al);
                }
                named_bar_sync(1, kSoftThreads);
                if (ok) {
                    if (!seg_first) {
                        // O^T (dims 128b + key lane, this warp's rows) *= alpha; PV of the previous tile has
                        // completed (it was issued before the QK whose commit was just waited for)
#pragma unroll 1
                        for (int c = 0; c < 4 * (S::kRpt / 16); ++c) {
                            const int r0 = rb + 16 * (c % (S::kRpt / 16));
                            const uint32_t col = lane_base + S::kColO + N * (c / (S::kRpt / 16)) + r0;
                            uint32_t o[16];
                            tmem_ld16(col, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * lds_f32(alpha_s + 4 * (r0 + e)));
                            tmem_st16(col, o);
                        }
                        tmem_wait_st();
                    }
#pragma unroll
                    for (int e = 0; e < S::kRpt; ++e) l[e] *= lds_f32(alpha_s + 4 * (rb + e));
                    (void)score();   // P and the sums again against the moved references
                }
            }
            if (ok) {
#pragma unroll
                for (int e = 0; e < S::kRpt; ++e) l[e] = ln[e];
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->pfull);
                // RoPE rows of the next tile (this tile's QK, which read the current ones, is done)
                if (it + 1 < count) store_rope(off_n >= 0);
            }
            off = off_n;
            off_n = off_n2;
            seg_first = false;

            if (cur.last_of_segment()) {
                const Job j = cur.j;
                const int t_end = cur.t;
                Walk<N> nxt = cur;
                nxt.next(a);
                const bool more = it + 1 < count;
                if (more && ok) load_q(nxt.j);   // every QK of this segment has completed
                // ---- row sums, O^T / l, out (or the job's part) and lse
                bool have_o = false;
                if (ok) {
                    const int g = 4 * it + 3;
                    have_o = wait_warp(ctl, &ctl->kfree[g % S::kRing], (g / S::kRing) & 1, a.status);
                    ok = have_o;
                    if (have_o) tc_fence_after_sync();
                }
                const bool whole = seg_tile == 0 && t_end == j.tiles - 1;
                const int slot = 2 * blockIdx.x + (seg_tile == 0 ? 1 : 0);
                const int64_t row = static_cast<int64_t>(j.seq) * a.rows_per_seq + j.row0;
                float sums = 0.0f;
#pragma unroll
                for (int e = 0; e < S::kRpt; ++e) {
                    float v = l[e];
                    l[e] = 0.0f;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    if (lane == e) sums = v;
                }
                if (lane < S::kRpt) sts_f32(xmax_s + 16 * (rb + lane) + 4 * qd, sums);
                named_bar_sync(1, kSoftThreads);
                if (qd == 0 && lane < S::kRpt) {
                    const int r = rb + lane;
                    const uint4 x = lds_u128(xmax_s + 16 * r);
                    const float sum = (__uint_as_float(x.x) + __uint_as_float(x.y)) + (__uint_as_float(x.z) + __uint_as_float(x.w));
                    const float mref = -lds_f32(negm_addr(r));
                    const bool empty = sum == 0.0f;   // the row sees no key of this segment
                    const float lse2 = empty ? -INFINITY : mref + log2f(sum);
                    float factor = 0.0f;
                    if (!empty) {
                        float denom = sum;
                        if (whole && a.sink != nullptr && r < j.rows) denom += exp2f(__ldg(a.sink + (j.row0 + r) % a.h_q) * kLog2e - mref);
                        factor = 1.0f / denom;
                    }
                    sts_f32(alpha_s + 4 * r, factor);
                    if (r < j.rows) {
                        if (whole)
                            a.lse[row + r] = lse2 * kLn2;
                        else
                            a.part_lse[static_cast<int64_t>(slot) * N + r] = lse2;
                    }
                }
                named_bar_sync(1, kSoftThreads);
                // O^T block b: this thread's lane is dim 128b + 32qd + lane; a warp store covers 32 consecutive
                // dims of one row (64 bytes)
                uint16_t* dst = whole ? reinterpret_cast<uint16_t*>(a.out) + row * 512
                                      : a.part_out + static_cast<int64_t>(slot) * N * 512;
#pragma unroll 1
                for (int c = 0; c < 4 * (S::kRpt / 16); ++c) {
                    const int b = c / (S::kRpt / 16), r0 = rb + 16 * (c % (S::kRpt / 16));
                    uint32_t o[16];
                    if (have_o) {
                        tmem_ld16(lane_base + S::kColO + N * b + r0, o);
                        tmem_wait_ld();
                    }
                    uint16_t* p = dst + static_cast<int64_t>(r0) * 512 + 128 * b + 32 * qd + lane;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        if (r0 + e < j.rows) {
                            const float f = lds_f32(alpha_s + 4 * (r0 + e));
                            const float v = have_o && f != 0.0f ? __uint_as_float(o[e]) * f : 0.0f;
                            p[e * 512] = whole ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
                        }
                    }
                }
                tc_fence_before_sync();
                if (!whole && seg_tile == 0) {
                    // the first part of a cut job: CTA c holds tile T of the run iff c = ((T + 1) CTAs - 1) / total
                    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), ctl->total);
                    const int64_t end = ctl->total * (static_cast<int64_t>(blockIdx.x) + 1) / ctas;   // behind this CTA's run
                    const int64_t last = end - (t_end + 1) + j.tiles - 1;
                    hdr = make_int4(static_cast<int>(row), j.rows, static_cast<int>(((last + 1) * ctas - 1) / ctl->total), j.row0 % a.h_q);
                }
                named_bar_sync(1, kSoftThreads);   // the factors and references have been read
                if (more) {
                    ++seg;
                    stage_q(nxt.j, seg);
                    seg_first = true;
                    seg_tile = nxt.t;
                }
            }
            cur.next(a);
        }
        if (threadIdx.x == 0) a.hdr[blockIdx.x] = hdr;
    } else if (warp < kWarpMma) {
        // ============ converters: K dims 0-511, 16-dim blocks 8c + 2q, 8c + 2q + 1 of each key ============
        const int t = threadIdx.x - 32 * S::kSoft;
        // lane l of converter warp w: key 8w + (l & 7) (and 64 more), quarter q = l >> 3: the eight lanes of a
        // quarter-warp store to eight bank slots, and the four quarters of a key load one 64-byte run
        const int q = (t >> 3) & 3;
        const int j = (t & 7) + 8 * (t >> 5);
        const uint32_t k_s = sbase + S::kOffK;
        bool ok = true;
        KeyRaw<R, kBlkOrder> raw[S::kKeys];
        int64_t o[S::kKeys], n[S::kKeys], m[S::kKeys];   // records of this tile, the next, the one behind
        Walk<N> ahead;
        ahead.start(a, ctl->job0, ctl->tile0, count);
#pragma unroll
        for (int u = 0; u < S::kKeys; ++u) {
            o[u] = ahead.template record<R>(a, j + 64 * u);
            if (o[u] >= 0) raw[u].load(a.cache + o[u], q);
        }
        // records that will be loaded later go into L2: eight keys of a warp are one run of a page (of eight
        // records or more), else each record by itself
        auto prefetch = [&](const int64_t (&r)[S::kKeys]) {
#pragma unroll
            for (int u = 0; u < S::kKeys; ++u) {
                if (a.page_shift >= 3) {
                    if (lane == 0 && r[u] >= 0) prefetch_l2_bulk(a.cache + r[u], 8u * R);
                } else if (q == 0 && r[u] >= 0) {
                    prefetch_l2_bulk(a.cache + r[u], R);
                }
            }
        };
        ahead.next(a);
#pragma unroll
        for (int u = 0; u < S::kKeys; ++u) n[u] = ahead.template record<R>(a, j + 64 * u);
        prefetch(n);
        ahead.next(a);
#pragma unroll
        for (int u = 0; u < S::kKeys; ++u) m[u] = ahead.template record<R>(a, j + 64 * u);
        prefetch(m);
        int slot = 0, round = 0;                          // ring slot of the next block, times around the ring
        for (int k = 0; k < count; ++k) {
            bool v[S::kKeys];
            uint32_t sp[S::kKeys][2];
#pragma unroll
            for (int u = 0; u < S::kKeys; ++u) {
                if (q == 0 && o[u] == -2 && a.status != nullptr) atomicOr(a.status, 0x2u);
                v[u] = o[u] >= 0;
                raw[u].scale_pairs(q, sp[u]);
                // a key with a NaN scale becomes a zero row, and its scores NaN
                const uint32_t nan = __ballot_sync(0xffffffffu, v[u] && (has_nan_e4m3(sp[u][0]) || has_nan_e4m3(sp[u][1])));
                const bool bad = ((nan >> (lane & 7)) & 0x01010101u) != 0u;
                if (bad) v[u] = false;
                if (q == 0) sts_u8(sbase + kOffNan + 128 * (k & 1) + j + 64 * u, bad ? 1u : 0u);
                if (n[u] >= 0) raw[u].load_scales(a.cache + n[u], q);
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (round > 0) ok = wait_warp(ctl, &ctl->kfree[slot], (round - 1) & 1, a.status);
                if (!ok) break;
                const uint32_t blk = k_s + slot * kBlk + (q >> 1) * kSubBlk;
                const int ch0 = 4 * (q & 1);
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int u = 0; u < S::kKeys; ++u) {
                    const uint32_t s2 = sp[u][b >> 1] >> (16 * (b & 1));
                    const __half2 sa = scale_half2(s2 & 0xFFu), sb = scale_half2((s2 >> 8) & 0xFFu);
                    const int row = j + 64 * u;
                    sts_u128(blk + swz(row, ch0), v[u] ? dq8(raw[u].codes[b].x, sa) : z);
                    sts_u128(blk + swz(row, ch0 + 1), v[u] ? dq8(raw[u].codes[b].y, sa) : z);
                    sts_u128(blk + swz(row, ch0 + 2), v[u] ? dq8(raw[u].codes[b].z, sb) : z);
                    sts_u128(blk + swz(row, ch0 + 3), v[u] ? dq8(raw[u].codes[b].w, sb) : z);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->kfull[slot]);
#pragma unroll
                for (int u = 0; u < S::kKeys; ++u)
                    if (n[u] >= 0) raw[u].load_codes(a.cache + n[u], q, b);
                if (++slot == S::kRing) {
                    slot = 0;
                    ++round;
                }
            }
            if (!ok) break;
            ahead.next(a);
#pragma unroll
            for (int u = 0; u < S::kKeys; ++u) {
                o[u] = n[u];
                n[u] = m[u];
                m[u] = ahead.template record<R>(a, j + 64 * u);
            }
            prefetch(m);
        }
    } else {
        // ======================= MMA issuer =======================
        const uint32_t idesc_qk = idesc_f16_f32(128, N, false, false);
        const uint32_t idesc_rope = R == 432 ? idesc_bf16_f32(128, N, false, false) : idesc_qk;
        const uint32_t idesc_pv = idesc_f16_f32(128, N, true, N == 64);
        const uint64_t kdesc0 = sdesc_sw128(sbase + S::kOffK, 16, 1024);          // K-major: keys x dims
        const uint64_t qdesc0 = sdesc_sw128(sbase + S::kOffQ, 16, 1024);          // K-major: rows x dims
        const uint64_t vdesc0 = sdesc_sw128(sbase + S::kOffK, kSubBlk, 1024);     // MN-major: dims x keys
        // P^T: MN-major rows x keys (N = 64), K-major rows x keys (N = 16, 32)
        const uint64_t pdesc0 = N == 64 ? sdesc_sw128(sbase + S::kOffP, kTile * 128, 1024) : sdesc_sw128(sbase + S::kOffP, 16, 1024);
        const bool leader = elect_one_in_warp();
        bool ok = true;
        Walk<N> w;
        w.start(a, ctl->job0, ctl->tile0, count);
        int qk_slot = 0, qk_round = 0, pv_slot = 0, seg = 0;
        bool first = true, prev_first = true;
        auto qk_block = [&](int b, uint32_t d) {   // dims 128b .. 128b + 127 as soon as they are converted
            ok = wait_warp(ctl, &ctl->kfull[qk_slot], qk_round & 1, a.status);
            if (!ok) return;
            tc_fence_after_sync();
            if (leader) {
                const uint64_t kd = kdesc0 + static_cast<uint64_t>((qk_slot * kBlk) >> 4);
                const uint64_t qd = qdesc0 + static_cast<uint64_t>((2 * b * S::kQBlk) >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss(d, kd + static_cast<uint64_t>(((kk >> 2) * kSubBlk + (kk & 3) * 32) >> 4),
                           qd + static_cast<uint64_t>(((kk >> 2) * S::kQBlk + (kk & 3) * 32) >> 4), idesc_qk,
                           (b > 0 || kk > 0) ? 1u : 0u);
            }
            __syncwarp();
            if (++qk_slot == S::kRing) {
                qk_slot = 0;
                ++qk_round;
            }
        };
        auto pv = [&](int tile, bool fresh) {      // O^T += V^T P^T of a tile; its ring blocks are free then
            ok = wait_warp(ctl, &ctl->pfull, tile & 1, a.status);
            if (!ok) return;
            tc_fence_after_sync();
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                if (leader) {
                    const uint64_t vd = vdesc0 + static_cast<uint64_t>((pv_slot * kBlk) >> 4);
#pragma unroll
                    for (int s = 0; s < 8; ++s)    // keys 16s .. 16s + 15
                        mma_ss(tmem + S::kColO + N * b, vd + static_cast<uint64_t>((s * 2048) >> 4),
                               pdesc0 + static_cast<uint64_t>((N == 64 ? s * 2048 : (s >> 2) * (N * 128) + (s & 3) * 32) >> 4), idesc_pv,
                               (!fresh || s > 0) ? 1u : 0u);
                    mma_commit(&ctl->kfree[pv_slot]);
                }
                __syncwarp();
                if (++pv_slot == S::kRing) pv_slot = 0;
            }
        };
        for (int it = 0; it < count && ok; ++it) {
            const uint32_t d = tmem + S::kColS + N * (it & 1);
            if (first) {
                // (the new queries are staged behind the epilogue of the old ones, which waits for this PV)
                if (it > 0) pv(it - 1, prev_first);
                if (ok) ok = wait_warp(ctl, &ctl->qready, seg & 1, a.status);
                ++seg;
            }
#pragma unroll 1
            for (int b = 0; b < S::kEarly && ok; ++b) qk_block(b, d);
            if (ok && !first) pv(it - 1, prev_first);
#pragma unroll 1
            for (int b = S::kEarly; b < 4 && ok; ++b) qk_block(b, d);
            if (ok) ok = wait_warp(ctl, &ctl->ropefull, it & 1, a.status);
            if (!ok) break;
            tc_fence_after_sync();
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)   // dims 512-575: K rows from tensor memory
                    mma_ts(d, tmem + S::kColR + 8 * kk, qdesc0 + static_cast<uint64_t>((8 * S::kQBlk + kk * 32) >> 4), idesc_rope, 1u);
                mma_commit(&ctl->sfull);
            }
            __syncwarp();
            prev_first = first;
            first = w.last_of_segment();
            w.next(a);
        }
        if (ok) pv(count - 1, prev_first);
        if (leader) mma_commit(&ctl->drain);
        __syncwarp();
        if (!mbar_wait(&ctl->drain, 0)) set_abort(ctl, a.status);
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, S::kTmemCols);
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// q as bf16 [rows, 576], box 64 dims x N rows, 128B swizzle.
template <int N>
bool encode_q_map(CUtensorMap* map, const void* q, int64_t rows) {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    if (fn == nullptr || rows < 1 || rows > 0x7FFFFFFF) return false;
    const cuuint64_t dims[2] = {576u, static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {576u * 2u};
    const cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(N)};
    const cuuint32_t elem_strides[2] = {1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(q), dims, strides, box, elem_strides,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int R, bool kBlkOrder, int N>
cudaError_t prepare_kernel() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit != 0 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    err = cudaFuncSetAttribute(paged_decode_kernel<R, kBlkOrder, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<N>::kSmemAlloc);
    if (err == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

// The attention grid of one row tile size (the join of cut jobs is a launch of its own).
template <int N>
cudaError_t launch_rows(const PagedDecodeArgs& d, cudaStream_t stream) {
    KernelArgs a;
    const int64_t rows = static_cast<int64_t>(d.batch) * d.s_q * d.h_q;
    if (!encode_q_map<N>(&a.qmap, d.q, rows)) return cudaErrorInvalidValue;
    a.cache = d.cache;
    a.page_table = d.page_table;
    a.table_stride = d.table_stride;
    a.seq_lens = d.seq_lens;
    a.num_pages = d.num_pages;
    a.page_shift = d.page_shift;
    a.capacity = d.capacity;
    a.batch = d.batch;
    a.s_q = d.s_q;
    a.h_q = d.h_q;
    a.rows_per_seq = d.s_q * d.h_q;
    a.row_tiles = (a.rows_per_seq + N - 1) / N;
    a.sm_scale = d.sm_scale;
    a.sink = d.attn_sink;
    a.out = static_cast<__nv_bfloat16*>(d.out);
    a.lse = d.lse;
    a.part_out = d.part_out;
    a.part_lse = d.part_lse;
    a.hdr = reinterpret_cast<int4*>(d.hdr);
    a.status = d.dev_status;
    const auto kernel = d.record_bytes == 432 ? paged_decode_kernel<432, false, N>
                        : d.block_scales      ? paged_decode_kernel<352, true, N>
                                              : paged_decode_kernel<352, false, N>;
    cudaError_t err = d.record_bytes == 432 ? prepare_kernel<432, false, N>()
                      : d.block_scales      ? prepare_kernel<352, true, N>()
                                            : prepare_kernel<352, false, N>();
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(d.ctas));
    cfg.blockDim = dim3(Shape<N>::kThreads);
    cfg.dynamicSmemBytes = Shape<N>::kSmemAlloc;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddepcontrol.wait
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel, a);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace paged
}  // namespace nvfp4mla

// paged_decode_few.cu -- attention of each query over all tokens of its own sequence, read from NVFP4
// records (352 or 432 bytes) through a page table, for up to 16 query rows (tokens x heads) of a sequence.
//
// What is computed. Sequence b has n = seq_lens[b] tokens; token p lies in slot
// page_table[b, p / page_size] * page_size + p % page_size. Its s_q queries are its last s_q tokens:
// query i has position n - s_q + i and attends the tokens j <= its position:
//     z_j = sm_scale * q[b,i,h,:] . K_j,   out = sum_j e^{z_j} V_j / (sum_j e^{z_j} + e^{sink_h}),
//     lse = ln sum_j e^{z_j},              V_j = K_j[0:512]
//
// Work split. The rows of a sequence (a job) share every key that is dequantized; the tiles of 64 keys of all
// jobs are cut into equal runs, one per CTA (one CTA per SM; paged_jobs.cuh). A job that lies in one run is
// finished by its CTA; the parts of a job that was cut go to the workspace (at most two per CTA, f16
// outputs divided by their own sums, times kPartScale, and fp32 log-sum-exps) and a second kernel joins them.
//
// Contractions. As keys outnumber rows, both products have the keys or the value dims on the MMA's M
// side: S^T [64 keys x 16] = K Q^T and O^T [512 dims x 16] += V^T P^T (four M = 128 MMAs per 16
// keys). A record is dequantized once, into f16 (exact: an e2m1 x e4m3 product has few bits), and
// read twice: K-major as K, MN-major as V^T. Queries are f16 times a power of two per row (exact
// within 2^28 of the row's largest), scores fp32, P f16.
//
// Pipeline. Shared memory holds a ring of kRing blocks (64 keys x 128 dims, 16 KB), two tiles and more:
// a block is filled by the converters, read by the QK MMAs, and freed by the PV MMAs of its tile.
// The conversion of one tile, the softmax of two others and the MMAs of all run side by side (two
// score buffers, two P buffers; QK and PV are issued by a thread each). Tiles of 64 keys, not 128: what a
// CTA can have in flight is bounded by shared memory, and a tile of 128 keys (128 KB) left the ring half
// empty while its softmax ran (3.5 us per 128 keys with a ring of 1.5 such tiles).
//
// Softmax. A lazy reference per row (log2 domain): P = 2^(z - m) in f16; a tile moves m only where some
// score exceeds m + 15.9, to a little below its largest score (new_reference in paged_jobs.cuh): the
// warps vote once per tile, and only then is O^T rescaled. A tile's softmax
// is a chain of short waits (2900 to 3800 clk from its scores to the next tile's, against 1500 of MMAs), so
// two groups of four warps take the even and the odd tiles; only the vote, from reading m to having moved
// it, goes in the tiles' order (242 -> 223 us for 64 sequences x 16 heads). The scores of an M = 64 MMA lie in
// 16 lanes of each lane quadrant; 16x256b loads spread them over the warp, two keys and four rows a thread.
// Row sums stay in fp32 registers (a thread's share of its rows) and are added up at the end of a job.
//
// Masks. A key behind the sequence's end or in a page outside the pool gets a zero row in shared memory
// (V and K share it, and 0 x NaN in PV would reach rows that do not see the key), a block of dims
// with a NaN scale likewise; P is 0 for a key that a row does not see and NaN for a NaN key that it
// sees.
//
// What bounds it. 64 sequences of 1024 to 32768 tokens, 16 heads, 352-byte records (382 MB): 166 to 172 us, 2.3 TB/s, where
// the records alone take 56 us. A tile takes about 1.5 us: its converters' chain (barrier, scales, two blocks of
// conversion and stores, fence: 2600 clk) and the ring, whose blocks live through the QK, the softmax and the PV of
// their tile (ring of 10 blocks 197 us, of 11 192). Of the shared memory's cycles the threads' accesses take 67% and
// the MMAs' operands 46% (two pipes, side by side in part), issue slots 55%, DRAM 31%: one f16 tile for both
// products, 64 KB written and read twice for 22 KB of records, is what keeps it from the memory's rate. One sequence
// of 1500 tokens: 17 us on the device, a chain of latencies (lengths, page table, records, products, join).
//
// Every wait is bounded by time; on timeout the CTA sets NVFP4_MLA_DEV_TIMEOUT, stops issuing work,
// drains what it issued and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "dequant.cuh"
#include "launch.h"
#include "paged_jobs.cuh"
#include "sm103_ptx.cuh"

namespace nvfp4mla {
namespace paged {

constexpr int kRows = 16;                  // query rows of a job (N of both products)
constexpr int kTile = 64;                  // keys per tile (M of the QK MMAs)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kSubBlk = 8192;              // 64 keys x 64 dims
constexpr int kBlk = 16384;                // 64 keys x 128 dims
constexpr int kAhead = 8;                  // tiles whose keys' slots are looked up ahead
constexpr int kLook = 2;                   // of them at a time
// Shared memory (offsets from a 1024-byte aligned base)
constexpr int kOffCM = 512;                // float [8][4]: per row pair {ch_a, ch_b, -m_a, -m_b}: the score scale
                                           // sm_scale log2(e) 2^-pre and the negated reference maximum
constexpr int kOffAlpha = 640;             // float [kRows]: rescale factors, then 1 / l
constexpr int kOffPos = 704;               // int [kRows]: each row's position (its last visible key)
constexpr int kOffXmax = 768;              // float [kRows][8]: per-row values of the four key quadrants, of two groups
constexpr int kOffNan = 1280;              // uint8 [4][2][64]: keys with a NaN scale, by tile and converter group
constexpr int kOffTile = 1792;             // int4 [kAhead]: first key position, row 0's position, 2 x (tiles left of the
                                           // segment) + (its first one), job
constexpr int kOffSlot = 1920;             // int [kAhead][64]: the keys' slots; -1: no key, -2: its page is outside the pool
constexpr int kOffScan = kOffSlot;         // int64 [35], while the CTA's run is looked for
constexpr int kOffQ = 4096;
static_assert(kOffSlot + kAhead * kTile * 4 <= kOffQ, "control area");

constexpr int kSoft = 8;                   // softmax warps: two groups of four, even and odd tiles
constexpr int kConv = 16;                  // converter warps: two groups, even and odd blocks
constexpr int kThreads = 32 * (kSoft + kConv + 3);   // and two MMA issuers and the look-up warp
constexpr int kRing = 11;
constexpr int kRopeRing = 3;               // tiles whose RoPE dims are held (see the converters)
// tensor memory columns: O^T four blocks, two score buffers
constexpr uint32_t kColO = 0, kColS = 4 * kRows;
constexpr int kTmemCols = 128;
static_assert(6 * kRows <= kTmemCols, "tensor memory");
constexpr int kQBlk = kRows * 128;         // rows x 64 dims
constexpr int kOffK = kOffQ + 9 * kQBlk;
constexpr int kOffRope = kOffK + kRing * kBlk;
constexpr int kOffP = kOffRope + kRopeRing * kSubBlk;
constexpr int kPBytes = kRows * 128;       // P of a tile: 64 keys x rows
constexpr int kSmemAlloc = kOffP + 2 * kPBytes + 1024;
static_assert(kSmemAlloc <= 232448, "shared memory");
static_assert(kOffQ % 1024 == 0 && kOffK % 1024 == 0 && kOffP % 1024 == 0, "operand alignment");

struct __align__(8) Ctl {
    uint64_t qload;           // q boxes landed (TMA, tx-counted)
    uint64_t qready;          // four softmax warps: q converted in shared memory
    uint64_t kfull[4];        // converter warps, by tile mod 4: the tile's blocks and RoPE dims are written
    uint64_t kfree[kRing];    // PV commit: a ring block has been read
    uint64_t sfull[2];        // QK commit, by tile parity: S^T ready
    uint64_t pfull[2];        // softmax warps, by tile parity: P^T written (and O^T rescaled)
    uint64_t voted[2];        // softmax warps, by tile parity: the references are those of the next tile
    uint64_t tfull[kAhead];   // look-up warp: slots and description of a tile
    uint64_t tfree[kAhead];   // converters and softmax warps have taken them
    uint64_t drain;           // every MMA issued completed
    uint32_t pfirst[2];       // by tile parity, behind pfull: the tile is the first one of its segment
    uint32_t tmem_base;
    uint32_t abort;
};
static_assert(sizeof(Ctl) <= kOffCM, "control block");

struct KernelArgs {
    CUtensorMap qmap;         // q as bf16 [batch * s_q * h_q, 576], box 64 dims x kRows rows, 128B swizzle
    const uint8_t* cache;
    Jobs jobs;
    float sm_scale;
    const float* sink;
    __nv_bfloat16* out;       // [batch * rows_per_seq, 512]
    float* lse;
    uint16_t* part_out;       // f16 [2 * CTAs, kRows, 512]
    float* part_lse;          // [2 * CTAs, kRows], log2 domain
    int4* hdr;                // [CTAs]: the cut job that begins in the CTA's run: first output row, rows
                              // (0: none), parts, slot of the first part (the others: 2 (CTA + 1), 2 (CTA + 2), ...)
    uint32_t* status;
};

// The next sequence from `from` on that has a token, or the last one. 32 lengths at a time (a call with 10^6 empty
// sequences in a row: 12 ms, of which other warps' work is the most): one by one that took 120 ms, and 2^23 of them, half of
// what a batch may hold, more than the second after which the pipeline's waits give up. Warp-collective.
__device__ __noinline__ int next_with_tokens(const Jobs& a, int from) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int b = from; b < a.batch; b += 32) {
        const uint32_t some = __ballot_sync(0xffffffffu, b + lane < a.batch && __ldg(a.seq_lens + b + lane) > 0);
        if (some != 0u) return b + __ffs(some) - 1;
    }
    return a.batch - 1;
}

// A position in the run of tiles of a CTA (whole warps call it).
struct Walk {
    Job j;
    int job, t, left;         // tile t of the job; tiles left in the run, this one included
    __device__ __forceinline__ void start(const Jobs& a, int job0, int tile0, int count) {
        job = job0;
        t = tile0;
        left = count;
        j = job_info<kRows, kTile>(a, job);
    }
    __device__ __forceinline__ void next(const Jobs& a) {
        if (left <= 1) {
            left = 0;
            return;
        }
        --left;
        if (++t < j.tiles) return;
        job = next_with_tokens(a, job + 1);   // (a tile is left, so there is one)
        j = job_info<kRows, kTile>(a, job);
        t = 0;
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

// The same for one thread.
__device__ __forceinline__ bool wait_one(Ctl* ctl, uint64_t* bar, uint32_t parity, uint32_t* status) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok && !aborted(ctl)) {
        ok = mbar_wait(bar, parity);
        if (!ok) set_abort(ctl, status);
    }
    return ok;
}

// Which of three phases have completed, without waiting for them (bits 0, 1, 2; the tests are in flight together).
__device__ __forceinline__ uint32_t test_three(uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, uint64_t* b2, uint32_t p2) {
    uint32_t r;
    asm volatile(
        "{\n"
        "  .reg .pred p, q, r;\n"
        "  .reg .b32 x, y;\n"
        "  mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
        "  mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 q, [%3], %4;\n"
        "  mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 r, [%5], %6;\n"
        "  selp.b32 %0, 1, 0, p;\n"
        "  selp.b32 x, 2, 0, q;\n"
        "  selp.b32 y, 4, 0, r;\n"
        "  or.b32 %0, %0, x;\n"
        "  or.b32 %0, %0, y;\n"
        "}\n"
        : "=&r"(r)
        : "r"(smem_addr(b0)), "r"(p0), "r"(smem_addr(b1)), "r"(p1), "r"(smem_addr(b2)), "r"(p2)
        : "memory");
    return r;
}

__device__ __forceinline__ float lds_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts_f32(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ void sts_u8(uint32_t a, uint32_t v) { asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts_u32(uint32_t a, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
// 16 lanes x 16 consecutive 32-bit columns over the warp: thread t gets, for each group of eight
// columns, columns 2 (t & 3), 2 (t & 3) + 1 of lane t >> 2 and of lane (t >> 2) + 8.
__device__ __forceinline__ void tmem_ld_16x256_x2(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ uint32_t ldg_stream2(const void* p) {
    uint16_t r;
    asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(r) : "l"(p));
    return r;
}
__device__ __forceinline__ uint4 ldg_stream16(const void* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// What a converter thread reads of one key: of the two 128-dim blocks c = group, group + 2 the record
// bytes 64c + 16q .. + 15 (the codes of 16-dim blocks 8c + 2q and 8c + 2q + 1) and their scales, and, for half of the
// keys, RoPE dims 16q .. 16q + 15.
template <int R, bool kBlkOrder>
struct HalfRecord {
    // 352-byte records place block s's scale at 320 + 8 (s & 3) + (s >> 2): the thread's four scales lie in
    // one 16-byte half of the field; otherwise block s's scale is at byte s, two pairs
    static constexpr bool kPermuted = R == 352 && !kBlkOrder;
    uint4 codes[2];
    uint32_t sc[kPermuted ? 4 : 2];
    uint32_t rope[R == 352 ? 4 : 8];

    __device__ __forceinline__ void load_codes(const uint8_t* rec, int q, int group, int i) { codes[i] = ldg_stream16(rec + 64 * (group + 2 * i) + 16 * q); }
    __device__ __forceinline__ void load_scales(const uint8_t* rec, int q, int group) {
        if constexpr (kPermuted) {
            const uint4 x = ldg_stream16(rec + 320 + 16 * (q & 1));
            sc[0] = x.x; sc[1] = x.y; sc[2] = x.z; sc[3] = x.w;
        } else {
            const uint8_t* p = rec + (R == 352 ? 320 : 256) + 8 * group + 2 * q;
            sc[0] = ldg_stream2(p);
            sc[1] = ldg_stream2(p + 16);
        }
    }
    __device__ __forceinline__ void load_rope(const uint8_t* rec, int q) {
#pragma unroll
        for (int e = 0; e < (R == 352 ? 1 : 2); ++e) {
            const uint4 x = ldg_stream16(rec + (R == 352 ? 256 + 16 * q : 304 + 32 * q + 16 * e));
            rope[4 * e] = x.x; rope[4 * e + 1] = x.y; rope[4 * e + 2] = x.z; rope[4 * e + 3] = x.w;
        }
    }
    // the scales of the 16-dim blocks of 128-dim block group + 2i: low byte 8c + 2q, next byte 8c + 2q + 1
    __device__ __forceinline__ uint32_t scale_pair(int q, int group, int i) const {
        if constexpr (kPermuted) {
            const uint32_t bi = static_cast<uint32_t>(2 * group + (q >> 1)) & 3u;   // byte 16 (q & 1) + 2c + (q >> 1)
            return __byte_perm(i == 0 ? sc[0] : sc[1], i == 0 ? sc[2] : sc[3], bi | ((bi + 4u) << 4)) & 0xFFFFu;
        } else {
            return sc[i];
        }
    }
    // RoPE dims 16q + 8e .. + 7 as 16-bit values (f16; the bf16 of 432-byte records as they are)
    __device__ __forceinline__ uint4 rope_values(int e) const {
        if constexpr (R == 352) {
            const uint2 a = e4m3x4_to_f16(rope[2 * e]), b = e4m3x4_to_f16(rope[2 * e + 1]);
            return make_uint4(a.x, a.y, b.x, b.y);
        } else {
            return make_uint4(rope[4 * e], rope[4 * e + 1], rope[4 * e + 2], rope[4 * e + 3]);
        }
    }
};
// Brings a tensor map near ahead of its first copy.
__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* map) { asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory"); }
// Starts bringing `bytes` (a multiple of 16, from a 16-byte boundary) into L2.
__device__ __forceinline__ void prefetch_l2_bulk(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// Whether one of the four bytes is an e4m3 NaN (0x7F or 0xFF).
__device__ __forceinline__ bool has_nan_e4m3(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u; }

template <int R, bool kBlkOrder>
__global__ void __launch_bounds__(kThreads, 1) paged_decode_kernel(const __grid_constant__ KernelArgs a) {
    constexpr int kSoftThreads = 32 * kSoft, kGroupWarps = 4, kGroupThreads = 128;
    constexpr int kWarpQk = kSoft + kConv, kWarpLook = kWarpQk + 2;   // the PV issuer between them
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    Ctl* ctl = reinterpret_cast<Ctl*>(smem);
    const uint32_t sbase = smem_addr(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        prefetch_tensormap(&a.qmap);
        mbar_init(&ctl->qload, 1);
        mbar_init(&ctl->qready, kGroupWarps);
        for (int s = 0; s < 4; ++s) mbar_init(&ctl->kfull[s], kConv);
        for (int s = 0; s < kRing; ++s) mbar_init(&ctl->kfree[s], 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ctl->sfull[s], 1);
            mbar_init(&ctl->pfull[s], kGroupWarps);
            mbar_init(&ctl->voted[s], kGroupWarps);
        }
        for (int s = 0; s < kAhead; ++s) {
            mbar_init(&ctl->tfull[s], 1);
            mbar_init(&ctl->tfree[s], kGroupWarps + kConv);
        }
        mbar_init(&ctl->drain, 2);
        ctl->abort = 0u;
        fence_barrier_init();
    }
    if (warp == kWarpQk) {
        tmem_alloc(&ctl->tmem_base, kTmemCols);
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

    const Run run = find_run<kRows, kTile, kThreads>(a.jobs, reinterpret_cast<int64_t*>(smem + kOffScan), static_cast<int>(gridDim.x), static_cast<int>(blockIdx.x));
    __syncthreads();   // every thread has its run: the scratch becomes the table of slots
    const int count = run.count;
    write_empty_jobs<kRows, kTile, kThreads>(a.jobs, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), a.out, a.lse);
    if (blockIdx.x == 0) check_lengths(a.jobs, static_cast<int>(threadIdx.x), kThreads, a.status);
    if (threadIdx.x == 0 && count == 0) a.hdr[blockIdx.x] = make_int4(0, 0, 0, 0);

    if (count == 0) {
        // nothing to do in this CTA
    } else if (warp < kSoft) {
        // ======================= softmax warps: two groups of four, group g the tiles of parity g =======================
        constexpr int kGroups = kRows / 8;        // groups of eight rows
        const int grp = warp >> 2;
        const int qd = warp & 3;              // TMEM lane quadrant: keys 16 qd .. 16 qd + 15 of a tile, and 128 dims' share of O^T
        const int k0 = 16 * qd + (lane >> 2); // this thread's keys: k0 and k0 + 8; its rows: c0 + 8g, c0 + 8g + 1
        const int c0 = 2 * (lane & 3);
        const uint32_t bar_grp = 1u + static_cast<uint32_t>(grp), bar_all = 3u;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * qd) << 16);
        const uint32_t s_col = lane_base + kColS + kRows * grp;
        const uint32_t p_s = sbase + kOffP + kPBytes * grp;
        const uint32_t cm_s = sbase + kOffCM;
        const uint32_t alpha_s = sbase + kOffAlpha;
        const uint32_t xmax_s = sbase + kOffXmax;
        const uint32_t pos_s = sbase + kOffPos;
        auto ch_addr = [&](int r) { return cm_s + 16 * (r >> 1) + 4 * (r & 1); };
        auto negm_addr = [&](int r) { return cm_s + 16 * (r >> 1) + 8 + 4 * (r & 1); };

        bool ok = true;
        // q of a job: rows row0 .. row0 + kRows - 1 of its sequence (thread 0); rows behind the job's last one are the
        // next sequence or zeros, and reach columns that nothing reads
        auto load_q = [&](const Job& j) {
            mbar_arrive_expect_tx(&ctl->qload, 9u * kQBlk);
            for (int bx = 0; bx < 9; ++bx)
                tma_load_2d(sbase + kOffQ + bx * kQBlk, &a.qmap, 64 * bx, j.seq * a.jobs.rows_per_seq + j.row0, &ctl->qload);
        };
        // group 0: per-row prescale and f16 (bf16 RoPE for 432-byte records) in place; the rows' scales and positions
        auto stage_q = [&](const Job& j, int seg) {
            constexpr int kTpr = kGroupThreads / kRows;   // threads of a row: each a block of 64 dims and a chunk of 8 RoPE dims
            static_assert(kTpr == 8, "a thread per block");
            if (ok) ok = wait_warp(ctl, &ctl->qload, seg & 1, a.status);
            const int r = threadIdx.x / kTpr, part = threadIdx.x % kTpr;
            auto chunk_at = [&](int bx, int c) { return sbase + kOffQ + bx * kQBlk + swz(r, c); };
            float qmax = 0.0f;
            auto take_max = [&](uint4 x) {
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    qmax = fmax3(qmax, fabsf(__uint_as_float(w[m] << 16)), fabsf(__uint_as_float(w[m] & 0xFFFF0000u)));
            };
            if (ok) {
#pragma unroll 4
                for (int i = 0; i < 8; ++i) take_max(lds_u128(chunk_at(part, (i + part) & 7)));
                take_max(lds_u128(chunk_at(8, part)));
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
                const int tok = (j.row0 + min(r, j.rows - 1)) / a.jobs.h_q;
                sts_u32(pos_s + 4 * r, static_cast<uint32_t>(j.first_pos + tok - j.first_tok));
            }
            auto scaled = [&](uint4 x, bool bf) {
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                uint32_t y[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float lo = __uint_as_float(w[m] << 16) * fpre, hi = __uint_as_float(w[m] & 0xFFFF0000u) * fpre;
                    y[m] = bf ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
                }
                return make_uint4(y[0], y[1], y[2], y[3]);
            };
            if (ok) {
                // (odd blocks with the chunks of each pair swapped, as the converters store K)
#pragma unroll 2
                for (int i = 0; i < 4; ++i) {
                    const int c = 2 * ((i + part) & 3);
                    const uint4 x = lds_u128(chunk_at(part, c)), y = lds_u128(chunk_at(part, c + 1));
                    sts_u128(chunk_at(part, c ^ (part & 1)), scaled(x, false));
                    sts_u128(chunk_at(part, (c + 1) ^ (part & 1)), scaled(y, false));
                }
                // RoPE chunks 1 and 2 of four are swapped (the threads of a row lie in one warp); bf16 for 432-byte records
                const uint4 x = scaled(lds_u128(chunk_at(8, part)), R == 432);
                __syncwarp();
                sts_u128(chunk_at(8, (part & 4) | ((part & 1) << 1) | ((part >> 1) & 1)), x);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->qready);
        };

        if (threadIdx.x == 0) load_q(job_info<kRows, kTile>(a.jobs, run.job));
        float l[kGroups][2] = {}, lnm[kGroups][2] = {};  // this thread's share of its rows' sums of 2^(z - m), and the -m that they are for
        int4 hdr = make_int4(0, 0, 0, 0);
        int seg = 0;
        // the sums for references that have moved since (also by the other group)
        auto move_sum = [&](int g, float nm0, float nm1) {
            if (nm0 != lnm[g][0]) {
                l[g][0] *= ex2_approx(nm0 - lnm[g][0]);
                lnm[g][0] = nm0;
            }
            if (nm1 != lnm[g][1]) {
                l[g][1] *= ex2_approx(nm1 - lnm[g][1]);
                lnm[g][1] = nm1;
            }
        };

        // Every warp of a group takes part in each of the group's barriers below, also after a wait ran out in it,
        // until the next vote, where the group leaves its tiles together; both groups then meet at the segment's end,
        // and leave together. No warp is left waiting on a missing one. Tensor-memory loads and stores are
        // warp-collective: masks change values only.
        for (int s0 = 0; s0 < count; ++seg) {
            if (ok) ok = wait_warp(ctl, &ctl->tfull[s0 % kAhead], (s0 / kAhead) & 1, a.status);
            const uint4 head = ok ? lds_u128(sbase + kOffTile + 16 * (s0 % kAhead)) : make_uint4(0u, 0u, 2u, static_cast<uint32_t>(run.job));
            const Job j = job_info<kRows, kTile>(a.jobs, static_cast<int>(head.w));
            const int s1 = s0 + static_cast<int>(head.z >> 1);
            const int seg_tile = static_cast<int>(head.x) / kTile;
            if (grp == 0) stage_q(j, seg);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                l[g][0] = l[g][1] = 0.0f;
                lnm[g][0] = lnm[g][1] = INFINITY;
            }
            if (bar_red_or(bar_all, kSoftThreads, !ok)) break;   // the rows' scales, references and positions are written

            for (int it = s0 + ((s0 ^ grp) & 1); it < s1; it += 2) {
                const int at = it % kAhead;
                if (ok) ok = wait_warp(ctl, &ctl->tfull[at], (it / kAhead) & 1, a.status);
                const uint32_t slot_s = sbase + kOffSlot + 4 * kTile * at;
                const bool there0 = ok && static_cast<int>(lds_u32(slot_s + 4 * k0)) >= 0;
                const bool there1 = ok && static_cast<int>(lds_u32(slot_s + 4 * k0 + 32)) >= 0;
                const int pos0 = kTile * (seg_tile + it - s0), pos = pos0 + k0;
                const bool full = pos0 + kTile - 1 <= j.first_pos;   // every row sees every key of the tile
                uint32_t sv[4 * kGroups];
                float z[kGroups][4];
                uint4 rows[kGroups];   // score scales and references of this thread's rows
                auto load_rows = [&]() {
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        rows[g] = lds_u128(cm_s + 8 * (c0 + 8 * g));
                        move_sum(g, __uint_as_float(rows[g].z), __uint_as_float(rows[g].w));
                    }
                };
                // z - m of this thread's scores (-inf for a row that does not see the key); returns the largest
                auto load_z = [&]() -> float {
                    float tmax = -INFINITY;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const uint4 c = rows[g];
                        const uint64_t ch = f32x2_pack(__uint_as_float(c.x), __uint_as_float(c.y));
                        const uint64_t nm = f32x2_pack(__uint_as_float(c.z), __uint_as_float(c.w));
                        const float2 a0 = f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(sv[4 * g]), __uint_as_float(sv[4 * g + 1])), ch, nm));
                        const float2 a1 = f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(sv[4 * g + 2]), __uint_as_float(sv[4 * g + 3])), ch, nm));
                        z[g][0] = a0.x;
                        z[g][1] = a0.y;
                        z[g][2] = a1.x;
                        z[g][3] = a1.y;
                    }
                    if (!full) {
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) {
                            const uint2 qp = lds_u64(pos_s + 4 * (c0 + 8 * g));
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (pos + 8 * (e >> 1) > static_cast<int>((e & 1) ? qp.y : qp.x)) z[g][e] = -INFINITY;
                        }
                    }
                    if (!there0 || !there1) {
#pragma unroll
                        for (int g = 0; g < kGroups; ++g)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!(e < 2 ? there0 : there1)) z[g][e] = -INFINITY;
                    }
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) tmax = fmax3(fmax3(tmax, z[g][0], z[g][1]), z[g][2], z[g][3]);
                    return tmax;
                };
                float tmax = -INFINITY;
                uint32_t nan0 = 0u, nan1 = 0u;
                if (ok && it >= 2) {   // the PV that read this P buffer
                    const int g = 4 * it - 5;
                    ok = wait_warp(ctl, &ctl->kfree[g % kRing], (g / kRing) & 1, a.status);
                }
                // the other group's tile before this one has its references
                if (ok && it > s0) ok = wait_warp(ctl, &ctl->voted[grp ^ 1], ((it - 1) >> 1) & 1, a.status);
                if (ok) load_rows();
                if (ok) ok = wait_warp(ctl, &ctl->sfull[grp], (it >> 1) & 1, a.status);
                if (ok) {
                    if (lane == 0) mbar_arrive(&ctl->tfree[at]);   // (the wait's vote put every lane's reads before)
                    tc_fence_after_sync();
                    tmem_ld_16x256_x2(s_col, sv);
                    // (the scores' MMAs were issued behind the waits for the blocks that the flags were written before)
                    const uint32_t nan_s = sbase + kOffNan + 128 * (it & 3) + k0;
                    nan0 = lds_u8(nan_s) | lds_u8(nan_s + 64);
                    nan1 = lds_u8(nan_s + 8) | lds_u8(nan_s + 72);
                    tmem_wait_ld();
                }
                if (ok) tmax = load_z();
                // ---- does any row need a new reference? (one barrier reduction; also entered where a wait ran out,
                // and then left by the whole group at once)
                if (bar_red_or(bar_grp, kGroupThreads, tmax > kMaxWeightLog2 || !ok)) {
                    // O^T stands still once the PV of the tile before has completed
                    if (ok && it > s0) {
                        const int g = 4 * it - 1;
                        ok = wait_warp(ctl, &ctl->kfree[g % kRing], (g / kRing) & 1, a.status);
                        tc_fence_after_sync();
                    }
                    if (bar_red_or(bar_grp, kGroupThreads, !ok)) {
                        ok = false;
                        break;
                    }
                    // per row: the tile's largest z over the 64 keys (a thread's two, the warp's, then the four quadrants)
#pragma unroll
                    for (int g = 0; g < kGroups; ++g)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int r = c0 + 8 * g + e;
                            const int last = static_cast<int>(lds_u32(pos_s + 4 * r));
                            const float ch = lds_f32(ch_addr(r));
                            float m = -INFINITY;
                            if (there0 && pos <= last) m = __uint_as_float(sv[4 * g + e]) * ch;
                            if (there1 && pos + 8 <= last) m = fmaxf(m, __uint_as_float(sv[4 * g + 2 + e]) * ch);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                            if (lane < 4) sts_f32(xmax_s + 32 * r + 4 * qd, m);
                        }
                    named_bar_sync(bar_grp, kGroupThreads);
                    if (qd == 0 && lane < kRows) {   // one thread per row: the new reference and the rescale factor
                        const uint4 x = lds_u128(xmax_s + 32 * lane);
                        const float zt = fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)),
                                               fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
                        const float mo = -lds_f32(negm_addr(lane));
                        float al = 1.0f;
                        if (zt > mo + kMaxWeightLog2) {
                            const float m = new_reference(zt, fminf(fminf(__uint_as_float(x.x), __uint_as_float(x.y)),
                                                                    fminf(__uint_as_float(x.z), __uint_as_float(x.w))));
                            al = mo == -INFINITY ? 0.0f : ex2_approx(mo - m);
                            sts_f32(negm_addr(lane), -m);
                        }
                        sts_f32(alpha_s + 4 * lane, al);
                    }
                    named_bar_sync(bar_grp, kGroupThreads);
                    if (it > s0) {
                        // O^T (this warp's 32 lanes of each block of dims) *= alpha
#pragma unroll 1
                        for (int b = 0; b < 4; ++b) {
                            uint32_t o[kRows];
                            tmem_ld16(lane_base + kColO + kRows * b, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < kRows; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * lds_f32(alpha_s + 4 * e));
                            tmem_st16(lane_base + kColO + kRows * b, o);
                        }
                        tmem_wait_st();
                    }
                    load_rows();
                    (void)load_z();   // against the moved references
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&ctl->voted[grp]);   // (the barrier's vote put every lane's reads before)
                if ((nan0 | nan1) != 0u) {   // a NaN key: NaN for the rows that see it
#pragma unroll
                    for (int g = 0; g < kGroups; ++g)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if ((e < 2 ? nan0 : nan1) != 0u && z[g][e] != -INFINITY) z[g][e] = NAN;
                }
                // P^T in shared memory: row = query row, 64 keys across (K-major B operand). Lanes of neighbouring keys
                // exchange a row each, so that a store is one wavefront of whole words.
                const bool odd_key = (lane & 4) != 0;
                const uint32_t perm = odd_key ? 0x3276u : 0x5410u;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int c = c0 + 8 * g;
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = ex2_approx(z[g][e]);
                    l[g][0] += p[0] + p[2];
                    l[g][1] += p[1] + p[3];
                    const uint32_t w0 = pack_f16x2(p[0], p[1]), w1 = pack_f16x2(p[2], p[3]);
                    const uint32_t v0 = __byte_perm(w0, __shfl_xor_sync(0xffffffffu, w0, 4), perm);
                    const uint32_t v1 = __byte_perm(w1, __shfl_xor_sync(0xffffffffu, w1, 4), perm);
                    const int r = c + (odd_key ? 1 : 0);
                    sts_u32(p_s + 4 * ((k0 & 7) >> 1) + swz(r, k0 >> 3), v0);
                    sts_u32(p_s + 4 * ((k0 & 7) >> 1) + swz(r, (k0 >> 3) + 1), v1);
                }
                if (qd == 0 && lane == 0) ctl->pfirst[grp] = it == s0 ? 1u : 0u;
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->pfull[grp]);
            }

            // ---- the segment's end: row sums, O^T / l, out (or the job's part) and lse
            const int t_end = seg_tile + s1 - s0 - 1;
            if (ok) {
                const int g = 4 * s1 - 1;
                ok = wait_warp(ctl, &ctl->kfree[g % kRing], (g / kRing) & 1, a.status);
                tc_fence_after_sync();
            }
            if (bar_red_or(bar_all, kSoftThreads, !ok)) break;   // the references are final, every QK of the segment has completed
            if (warp == 0 && s1 < count) {
                ok = wait_warp(ctl, &ctl->tfull[s1 % kAhead], (s1 / kAhead) & 1, a.status);
                if (ok && lane == 0) load_q(job_info<kRows, kTile>(a.jobs, static_cast<int>(lds_u32(sbase + kOffTile + 16 * (s1 % kAhead) + 12))));
                __syncwarp();
            }
            const bool whole = seg_tile == 0 && t_end == j.tiles - 1;
            const int slot = 2 * blockIdx.x + (seg_tile == 0 ? 1 : 0);
            const int64_t row = static_cast<int64_t>(j.seq) * a.jobs.rows_per_seq + j.row0;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const uint4 c = lds_u128(cm_s + 8 * (c0 + 8 * g));
                move_sum(g, __uint_as_float(c.z), __uint_as_float(c.w));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = l[g][e];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    if (lane < 4) sts_f32(xmax_s + 32 * (c0 + 8 * g + e) + 16 * grp + 4 * qd, v);
                }
            }
            named_bar_sync(bar_all, kSoftThreads);
            if (warp == 0 && lane < kRows) {
                const int r = lane;
                const uint4 x = lds_u128(xmax_s + 32 * r), y = lds_u128(xmax_s + 32 * r + 16);
                const float sum = ((__uint_as_float(x.x) + __uint_as_float(x.y)) + (__uint_as_float(x.z) + __uint_as_float(x.w))) +
                                  ((__uint_as_float(y.x) + __uint_as_float(y.y)) + (__uint_as_float(y.z) + __uint_as_float(y.w)));
                const float mref = -lds_f32(negm_addr(r));
                const bool empty = sum == 0.0f;   // the row sees no key of this segment
                const float lse2 = empty ? -INFINITY : mref + log2f(sum);
                float factor = 0.0f;
                if (!empty) {
                    float denom = sum;
                    if (whole && a.sink != nullptr && r < j.rows) denom += exp2f(__ldg(a.sink + (j.row0 + r) % a.jobs.h_q) * kLog2e - mref);
                    factor = (whole ? 1.0f : kPartScale) / denom;
                }
                sts_f32(alpha_s + 4 * r, factor);
                if (r < j.rows) {
                    if (whole)
                        a.lse[row + r] = lse2 * kLn2;
                    else
                        a.part_lse[static_cast<int64_t>(slot) * kRows + r] = lse2;
                }
            }
            named_bar_sync(bar_all, kSoftThreads);
            // O^T blocks 2 grp, 2 grp + 1: this thread's lane is dim 128b + 32qd + lane (in the second half of a block with
            // the chunks of each pair swapped); a warp store covers 32 consecutive dims of one row (64 bytes)
            const int dim = 32 * qd + (qd >= 2 ? lane ^ 8 : lane);
            uint16_t* dst = whole ? reinterpret_cast<uint16_t*>(a.out) + row * 512
                                  : a.part_out + static_cast<int64_t>(slot) * kRows * 512;
            float factor[kRows];
#pragma unroll
            for (int e = 0; e < kRows; e += 4) {
                const uint4 f = lds_u128(alpha_s + 4 * e);
                factor[e] = __uint_as_float(f.x);
                factor[e + 1] = __uint_as_float(f.y);
                factor[e + 2] = __uint_as_float(f.z);
                factor[e + 3] = __uint_as_float(f.w);
            }
#pragma unroll 1
            for (int b = 2 * grp; b < 2 * grp + 2; ++b) {
                uint32_t o[kRows];
                tmem_ld16(lane_base + kColO + kRows * b, o);
                tmem_wait_ld();
                // neighbouring lanes (dims) exchange a row each: 32-bit stores, the even lane's of row e, the odd lane's of row e + 1
                uint16_t* p = dst + 128 * b + (dim & ~1);
#pragma unroll
                for (int e = 0; e < kRows; e += 2) {
                    const float v0 = factor[e] != 0.0f ? __uint_as_float(o[e]) * factor[e] : 0.0f;
                    const float v1 = factor[e + 1] != 0.0f ? __uint_as_float(o[e + 1]) * factor[e + 1] : 0.0f;
                    const float u = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v0 : v1, 1);
                    const float lo = (lane & 1) ? u : v0, hi = (lane & 1) ? v1 : u;
                    const int r = e + (lane & 1);
                    if (r < j.rows) *reinterpret_cast<uint32_t*>(p + r * 512) = whole ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
                }
            }
            tc_fence_before_sync();
            if (!whole && seg_tile == 0) {
                // the first part of a cut job: its last tile lies (tiles - t_end - 1) behind the end of this run
                const int64_t end = run_begin(run.total, run.runs, static_cast<int64_t>(blockIdx.x) + 1);
                hdr = make_int4(static_cast<int>(row), j.rows, run_of(run, end - (t_end + 1) + j.tiles - 1) - static_cast<int>(blockIdx.x) + 1,
                                2 * static_cast<int>(blockIdx.x) + 1);
            }
            named_bar_sync(bar_all, kSoftThreads);   // the factors and references have been read
            s0 = s1;
        }
        if (threadIdx.x == 0) a.hdr[blockIdx.x] = hdr;
    } else if (warp < kWarpQk) {
        // ============ converters: two groups of eight warps, group g the 128-dim blocks g and g + 2 ============
        const int group = (warp - kSoft) >> 3;
        const int t = (threadIdx.x - 32 * kSoft) & 255;
        // Lane l of a group's warp w: quarter q = l & 3 of key j, so that four lanes load one 64-byte run, and a quarter-warp
        // the runs of keys j and j + 2, which lie in different banks of the load's data stage: 6 of its cycles a load,
        // against 17.6 with the eight keys of a quarter-warp in lanes beside one another. Its eight stores go to
        // eight bank slots as the chunks of each pair are swapped in the second half of a block (q >> 1).
        const int q = t & 3;
        const int j = 8 * (t >> 5) + ((t >> 3) & 1) + 2 * ((t >> 2) & 1) + 4 * ((t >> 4) & 1);
        const bool with_rope = (t >> 7) == group;     // group 0 the RoPE dims of keys 0-31, group 1 of keys 32-63
        // the thread's four chunks of a block are 16-byte slots x, x ^ 1, x ^ 2, x ^ 3 of row j of its half (128B swizzle)
        const uint32_t store0 = sbase + kOffK + (q >> 1) * kSubBlk + 128 * j + (((4 * (q & 1)) ^ (q >> 1) ^ (j & 7)) << 4);
        bool ok = true;
        HalfRecord<R, kBlkOrder> raw;
        auto slot_at = [&](int k) { return static_cast<int>(lds_u32(sbase + kOffSlot + 4 * kTile * (k % kAhead) + 4 * j)); };
        auto tile_bar = [&](int k) { return &ctl->tfull[k % kAhead]; };
        auto taken = [&](int k) {   // behind a __syncwarp()
            if (lane == 0) mbar_arrive(&ctl->tfree[k % kAhead]);
        };
        int cur = -1, nxt = -1;                       // slots of this thread's key in this tile, in the next
#pragma unroll 1
        for (int k = 0; k < min(count, 2); ++k) {
            if (ok) ok = wait_warp(ctl, tile_bar(k), 0, a.status);
            if (ok) (k == 0 ? cur : nxt) = slot_at(k);
            __syncwarp();
            if (ok) taken(k);
        }
        if (cur >= 0) {
            const uint8_t* rec = a.cache + static_cast<int64_t>(cur) * R;
            raw.load_codes(rec, q, group, 0);
            raw.load_codes(rec, q, group, 1);
            raw.load_scales(rec, q, group);
            if (with_rope) raw.load_rope(rec, q);
        }
        int slot = group, round = 0;                  // ring slot of this group's next block, times around the ring
        for (int k = 0; k < count && ok; ++k) {
            // the tile's three barriers are asked ahead of the work that does not need them
            const bool more = k + 2 < count;
            const int slot1 = slot + 2 >= kRing ? slot + 2 - kRing : slot + 2, round1 = round + (slot + 2 >= kRing ? 1 : 0);
            uint32_t ready = test_three(&ctl->kfree[slot], (round - 1) & 1, &ctl->kfree[slot1], (round1 - 1) & 1, tile_bar(k + 2), ((k + 2) / kAhead) & 1);
            if (round == 0) ready |= 1u;
            if (round1 == 0) ready |= 2u;
            ready = __reduce_and_sync(0xffffffffu, ready);
            const uint8_t* next_rec = a.cache + static_cast<int64_t>(max(nxt, 0)) * R;
            uint32_t sp[2] = {raw.scale_pair(q, group, 0), raw.scale_pair(q, group, 1)};
            // dims with a NaN scale become zeros, and the key's scores NaN; a key that is not there is zeros: scales 0
            const uint32_t nan = __ballot_sync(0xffffffffu, cur >= 0 && has_nan_e4m3(sp[0] | (sp[1] << 16)));
            const bool bad = ((nan >> (lane & 28)) & 0xFu) != 0u;
            if (cur < 0 || bad) sp[0] = sp[1] = 0u;
            if (q == 0) sts_u8(sbase + kOffNan + 128 * (k & 3) + 64 * group + j, bad ? 1u : 0u);
            if (nxt >= 0) raw.load_scales(next_rec, q, group);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if ((ready & (1u << i)) == 0u &&
                    !wait_warp(ctl, &ctl->kfree[i == 0 ? slot : slot1], ((i == 0 ? round : round1) - 1) & 1, a.status)) {
                    ok = false;
                    break;
                }
                const uint32_t at = store0 + (i == 0 ? slot : slot1) * kBlk;
                const __half2 sa = scale_half2(sp[i] & 0xFFu), sb = scale_half2(sp[i] >> 8);
                sts_u128(at, dq8(raw.codes[i].x, sa));
                sts_u128(at ^ 16u, dq8(raw.codes[i].y, sa));
                sts_u128(at ^ 32u, dq8(raw.codes[i].z, sb));
                sts_u128(at ^ 48u, dq8(raw.codes[i].w, sb));
                // The RoPE dims go to the buffer of kRopeRing tiles ago: the PV commit that freed this group's first
                // block of the tile (or, before the ring's first round, no tile at all) came behind that QK
                if (i == 0 && with_rope) {
                    const uint32_t rope = sbase + kOffRope + (k % kRopeRing) * kSubBlk;
                    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                    const int c = 4 * (q >> 1) + (q & 1);   // chunks 1 and 2 of four swapped, for eight bank slots here too
                    sts_u128(rope + swz(j, c), cur >= 0 ? raw.rope_values(0) : zero);
                    sts_u128(rope + swz(j, c + 2), cur >= 0 ? raw.rope_values(1) : zero);
                }
                if (nxt >= 0) {
                    raw.load_codes(next_rec, q, group, i);
                    if (i == 0 && with_rope) raw.load_rope(next_rec, q);
                }
            }
            if (!ok) break;
            if (more && (ready & 4u) == 0u) ok = wait_warp(ctl, tile_bar(k + 2), ((k + 2) / kAhead) & 1, a.status);
            cur = nxt;
            nxt = more && ok ? slot_at(k + 2) : -1;
            slot = slot1 + 2 >= kRing ? slot1 + 2 - kRing : slot1 + 2;
            round = round1 + (slot1 + 2 >= kRing ? 1 : 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->kfull[k & 3]);
            if (more && ok) taken(k + 2);
        }
    } else if (warp == kWarpLook) {
        // ============ look-up warp: the slots of the keys of every tile, and their records into L2 ============
        // kLook tiles at a time: their loads from the page table are in flight together (64 sequences x 16 heads: 206 us
        // with one tile at a time, 197 with two, 200 with four)
        Walk w;
        w.start(a.jobs, run.job, run.tile, count);
        bool first = true, ok = true;
        for (int it0 = 0; it0 < count && ok; it0 += kLook) {
            int slot[kLook][2];
            uint4 tile[kLook];
#pragma unroll
            for (int u = 0; u < kLook; ++u) {
#pragma unroll
                for (int e = 0; e < 2; ++e) slot[u][e] = it0 + u < count ? slot_of(a.jobs, w.j.seq, w.j.keys, kTile * w.t + 32 * e + lane) : -1;
                const int left = min(w.left, w.j.tiles - w.t);
                tile[u] = make_uint4(static_cast<uint32_t>(kTile * w.t), static_cast<uint32_t>(w.j.first_pos), (first ? 1u : 0u) | static_cast<uint32_t>(left << 1),
                                     static_cast<uint32_t>(w.job));
                first = left == 1;
                w.next(a.jobs);
            }
#pragma unroll
            for (int u = 0; u < kLook; ++u) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (slot[u][e] == -2 && a.status != nullptr) atomicOr(a.status, 0x2u);
                    // eight keys are one run of a page (of eight records or more)
                    if (a.jobs.page_shift >= 3) {
                        if ((lane & 7) == 0 && slot[u][e] >= 0) prefetch_l2_bulk(a.cache + static_cast<int64_t>(slot[u][e]) * R, 8u * R);
                    } else if (slot[u][e] >= 0) {
                        prefetch_l2_bulk(a.cache + static_cast<int64_t>(slot[u][e]) * R, R);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kLook; ++u) {
                const int it = it0 + u, at = it % kAhead;
                if (it >= count) break;
                if (ok && it >= kAhead) ok = wait_warp(ctl, &ctl->tfree[at], (it / kAhead - 1) & 1, a.status);
                if (!ok) break;
#pragma unroll
                for (int e = 0; e < 2; ++e) sts_u32(sbase + kOffSlot + 4 * (kTile * at + 32 * e + lane), static_cast<uint32_t>(slot[u][e]));
                if (lane == 0) sts_u128(sbase + kOffTile + 16 * at, tile[u]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->tfull[at]);
            }
        }
    } else if (warp == kWarpQk) {
        // ======================= QK issuer: S^T = K Q^T =======================
        const uint32_t idesc_qk = idesc_f16_f32(64, kRows, false, false);
        const uint32_t idesc_rope = R == 432 ? idesc_bf16_f32(64, kRows, false, false) : idesc_qk;
        const uint64_t kdesc0 = sdesc_sw128(sbase + kOffK, 16, 1024);          // K-major: keys x dims
        const uint64_t rdesc0 = sdesc_sw128(sbase + kOffRope, 16, 1024);       // K-major: keys x RoPE dims
        const uint64_t qdesc0 = sdesc_sw128(sbase + kOffQ, 16, 1024);             // K-major: rows x dims
        const bool leader = elect_one_in_warp();
        if (leader) {
            bool ok = true;
            int slot = 0, rslot = 0, seg = 0, s1 = 0;
            for (int it = 0; it < count; ++it) {
                if (it == s1) {   // a segment begins: its length, its rows
                    ok = wait_one(ctl, &ctl->tfull[it % kAhead], (it / kAhead) & 1, a.status);
                    if (!ok) break;
                    s1 = it + static_cast<int>(lds_u32(sbase + kOffTile + 16 * (it % kAhead) + 8) >> 1);
                    ok = wait_one(ctl, &ctl->qready, seg++ & 1, a.status);
                }
                // the score buffer (its scores of two tiles ago have been read) and the keys
                const bool free = it < 2 || mbar_test_wait(&ctl->pfull[it & 1], ((it - 2) >> 1) & 1);
                const bool full = mbar_test_wait(&ctl->kfull[it & 3], (it >> 2) & 1);
                if (ok && !free) ok = wait_one(ctl, &ctl->pfull[it & 1], ((it - 2) >> 1) & 1, a.status);
                if (ok && !full) ok = wait_one(ctl, &ctl->kfull[it & 3], (it >> 2) & 1, a.status);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t d = tmem + kColS + kRows * (it & 1);
                // (short loops: straight-line code of 36 MMAs runs at the pace of the instruction fetch, 50 to 60 clk
                // an MMA against 25)
#pragma unroll 3
                for (int b = 0; b < 9; ++b) {   // 64 dims each, the RoPE dims last
                    const uint64_t kd = b < 8 ? kdesc0 + static_cast<uint64_t>((slot * kBlk + (b & 1) * kSubBlk) >> 4)
                                              : rdesc0 + static_cast<uint64_t>((rslot * kSubBlk) >> 4);
                    const uint64_t qd = qdesc0 + static_cast<uint64_t>((b * kQBlk) >> 4);
                    const uint32_t idesc = b < 8 ? idesc_qk : idesc_rope;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ss(d, kd + static_cast<uint64_t>((kk * 32) >> 4), qd + static_cast<uint64_t>((kk * 32) >> 4), idesc, (b | kk) != 0 ? 1u : 0u);
                    if ((b & 1) && ++slot == kRing) slot = 0;
                }
                if (++rslot == kRopeRing) rslot = 0;
                mma_commit(&ctl->sfull[it & 1]);
            }
        }
        __syncwarp();
        if (leader) mma_commit(&ctl->drain);
        __syncwarp();
        if (!mbar_wait(&ctl->drain, 0)) set_abort(ctl, a.status);
        __syncwarp();
    } else {
        // ======================= PV issuer: O^T += V^T P^T; the tile's ring blocks are free then =======================
        const uint32_t idesc_pv = idesc_f16_f32(128, kRows, true, false);
        const uint64_t vdesc0 = sdesc_sw128(sbase + kOffK, kSubBlk, 1024);     // MN-major: dims x keys
        const uint64_t pdesc0 = sdesc_sw128(sbase + kOffP, 16, 1024);          // K-major: rows x keys
        const bool leader = elect_one_in_warp();
        if (leader) {
            int slot = 0;
            for (int it = 0; it < count; ++it) {
                if (!wait_one(ctl, &ctl->pfull[it & 1], (it >> 1) & 1, a.status)) break;
                tc_fence_after_sync();
                const bool first = *reinterpret_cast<volatile uint32_t*>(&ctl->pfirst[it & 1]) != 0u;
                const uint64_t pd = pdesc0 + static_cast<uint64_t>((kPBytes * (it & 1)) >> 4);
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    const uint64_t vd = vdesc0 + static_cast<uint64_t>((slot * kBlk) >> 4);
#pragma unroll
                    for (int s = 0; s < 4; ++s)    // keys 16s .. 16s + 15
                        mma_ss(tmem + kColO + kRows * b, vd + static_cast<uint64_t>((s * 2048) >> 4),
                               pd + static_cast<uint64_t>((s * 32) >> 4), idesc_pv, (!first || s > 0) ? 1u : 0u);
                    mma_commit(&ctl->kfree[slot]);
                    if (++slot == kRing) slot = 0;
                }
            }
        }
        __syncwarp();
        if (leader) mma_commit(&ctl->drain);
        __syncwarp();
        if (!mbar_wait(&ctl->drain, 0)) set_abort(ctl, a.status);
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kWarpQk) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// q as bf16 [rows, 576], box 64 dims x kRows rows, 128B swizzle.
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
    const cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(kRows)};
    const cuuint32_t elem_strides[2] = {1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(q), dims, strides, box, elem_strides,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int R, bool kBlkOrder>
cudaError_t prepare_kernel() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit != 0 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    err = cudaFuncSetAttribute(paged_decode_kernel<R, kBlkOrder>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
    if (err == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

}  // namespace paged

cudaError_t launch_paged_decode_few(const PagedDecodeArgs& d, cudaStream_t stream) {
    using namespace paged;
    KernelArgs a;
    const int64_t rows = static_cast<int64_t>(d.jobs.batch) * d.jobs.rows_per_seq;
    if (!encode_q_map(&a.qmap, d.q, rows)) return cudaErrorInvalidValue;
    a.cache = d.cache;
    a.jobs = d.jobs;
    a.jobs.row_tiles = (a.jobs.rows_per_seq + kRows - 1) / kRows;
    a.sm_scale = d.sm_scale;
    a.sink = d.attn_sink;
    a.out = static_cast<__nv_bfloat16*>(d.out);
    a.lse = d.lse;
    a.part_out = d.part_out;
    a.part_lse = d.part_lse;
    a.hdr = reinterpret_cast<int4*>(d.hdr);
    a.status = d.dev_status;
    const auto kernel = d.record_bytes == 432 ? paged_decode_kernel<432, false>
                        : d.block_scales      ? paged_decode_kernel<352, true>
                                              : paged_decode_kernel<352, false>;
    cudaError_t err = d.record_bytes == 432 ? prepare_kernel<432, false>()
                      : d.block_scales      ? prepare_kernel<352, true>()
                                            : prepare_kernel<352, false>();
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(d.runs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemAlloc;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddepcontrol.wait
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel, a);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace nvfp4mla

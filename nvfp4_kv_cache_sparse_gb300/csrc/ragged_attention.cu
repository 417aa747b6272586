// ragged_attention.cu -- attention of chunks of new tokens over their sequences' expanded keys and values (head dims 128 + 64
// shared RoPE dims for scores, 128 for values), sequences of any lengths packed one behind the other.
//
//   z[i, n] = sm_scale (q[i, h, 0:128] . kv[n, h, 0:128] + q[i, h, 128:192] . k_pe[n]),   n <= lk - lq + i
//   out[i, h] = sum_n e^z kv[n, h, 128:256] / (sum_n e^z + e^sink[h]),   lse[i, h] = log sum_n e^z
// 640 FLOP per query, key and head against 2176 in the absorbed form, which works on the latents themselves: the tensor cores
// bound it. One pass over the keys with a running reference m of each row: P = 2^(z log2 e - m) in bf16, whose range
// is that of fp32, so that no weight is lost however far it lies below the largest; row sums and outputs in fp32. m, a whole number in log2
// units, moves only when a score passes it by 2^8 (the output in tensor memory is rescaled then).
//
// A tile is 256 query rows of one sequence and head, in two halves of 128. S = Q K^T of a half is one tcgen05.mma chain
// (M = 128 rows, N = 128 keys, K = 192) into tensor memory; a warpgroup per half turns it into P, which overwrites S
// and feeds P V from tensor memory. While one half's softmax runs, the tensor cores work for the other. Keys and
// values come through a ring of eight 16 KB units (a key block is three units of 128 keys x 64 dims, its values two
// units of 64 keys x 128 dims).
//
// Tiles are of very different lengths and often fewer than SMs, so the CTAs, one per SM, take equal runs of (tile, head, block
// of 128 keys) units, heads inside tiles: neighbouring tiles of a head are then read by several CTAs at about the same
// time, from L2. A tile that two runs share leaves fp32 parts in the workspace, which a second kernel joins.
#include "head_tiles.cuh"
#include "launch.h"

namespace nvfp4mla {
namespace {

using namespace tiles;

constexpr int kUnits = 8;              // ring
constexpr int kOffQ = 1024;
constexpr int kOffRing = kOffQ + 6 * kBox;
constexpr int kSmem = kOffRing + kUnits * kBox;
static_assert(kSmem <= 232448, "shared memory");
constexpr int kWarpLoad = 8, kWarpFix = 9, kWarpMma = 10;    // 10 and 11: products of the two halves; 0-3 and 4-7: their softmax
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;              // two halves of 128 columns each
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMoveLog2 = 8.0f;      // a reference moves, a block later, when a score passes it by 2^8,
constexpr float kFarLog2 = 64.0f;      // and at once when one passes it by 2^64
constexpr int kExtra = 1;              // what a tile costs besides its blocks, in blocks
constexpr int kMinRun = 2;
constexpr int kItems = 4;              // items that are known ahead
constexpr int kMaxCtas = kPagedMaxSms;

// A tile's part in a run.
struct Item {
    int q0, k0;                        // first query row of the tile and first key of its sequence, of all rows
    int rows;                          // rows of the tile from its first one to the sequence's end
    int seen;                          // keys that the tile's first row sees (negative: rows before the first key)
    int keys;                          // of the sequence
    int head, from, count0, count1;    // first block; blocks of each half
    int slot;                          // of the part where the tile is cut, else -1
    int valid;                         // 0: no more items
};

struct Ctl {
    // Block g of the CTA's run uses entry g & 1 of each; both issuers hand a block back, the values also the warp that cleans them.
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t q_full[2], q_free[2];     // a half's queries landed; its last scores are done
    uint64_t s_full[2];                // scores in tensor memory
    uint64_t p_full[2];                // 4 warps: P written, O rescaled
    uint64_t turn[2];                  // the other half's chain of products is issued
    uint64_t o_done[2];                // a tile's last P V is done
    uint64_t v_clean[2];               // rows behind a sequence's end were zeroed (in turn: there may be the values of two tiles)
    uint64_t drain;
    uint64_t item_full[kItems], item_empty[kItems];
    uint32_t tmem_base, abort;
    Item items[kItems];                // what the CTA works on, one behind the other
};
static_assert(sizeof(Ctl) <= kOffQ, "control block");

struct KernelArgs {
    CUtensorMap q_map;                 // [rows_q, heads, 192], box 128 x 1 x 64
    CUtensorMap k_map;                 // kv [rows_k, heads, 256], box 128 x 1 x 64
    CUtensorMap v_map;                 // the same, box 64 x 1 x 64
    CUtensorMap pe_map;                // [rows_k, 1, 64], box 128 x 1 x 64
    RaggedArgs p;
    float* part_out;                   // [2 CTAs, 8 warps, 16, 32 lanes, 8]: eight dims of a row, divided by its own sum
    float* part_lse;                   // [2 CTAs, 256], log2
    int4* headers;                     // [CTAs]: first output row, rows, head, parts (0: no tile begins here and ends elsewhere)
};

struct Seq {
    int q0, lq, k0, lk;
};
__device__ __forceinline__ int clamp_start(int v, int64_t rows) { return static_cast<int>(min(max(static_cast<int64_t>(v), int64_t(0)), rows)); }
__device__ __forceinline__ Seq seq_at(const RaggedArgs& p, int b) {
    Seq s;
    s.q0 = clamp_start(__ldg(p.starts_q + b), p.rows_q);
    s.k0 = clamp_start(__ldg(p.starts_k + b), p.rows_k);
    s.lq = max(clamp_start(__ldg(p.starts_q + b + 1), p.rows_q) - s.q0, 0);
    s.lk = max(clamp_start(__ldg(p.starts_k + b + 1), p.rows_k) - s.k0, 0);
    return s;
}
__device__ __forceinline__ int tiles_of(const Seq& s) { return (s.lq + 255) >> 8; }
// Key blocks of rows [0, rows) of a sequence: its last row sees the first lk - lq + rows keys.
__device__ __forceinline__ int blocks_of(const Seq& s, int rows) {
    const int keys = s.lk - s.lq + min(rows, s.lq);
    return keys <= 0 ? 0 : (keys + 127) >> 7;
}
// Units of the first m tiles: a tile before the last one ends on a multiple of 256 rows, tile j has max(0, p + 2 (j + 1)) blocks
// with p = ceil((lk - lq) / 128), and kExtra.
__device__ __forceinline__ int64_t units_of(const Seq& s, int m) {
    const int count = tiles_of(s);
    if (m <= 0) return 0;
    const int whole = m < count ? m : count - 1;            // tiles that are surely full
    const int64_t pre = (s.lk - s.lq + 127) >> 7;           // (rounds up for negative ones too)
    int64_t none = pre < 0 ? (-pre) >> 1 : 0;               // tiles without keys
    if (none > whole) none = whole;
    const int64_t a = none + 1, n = whole - none;           // j + 1 = a .. whole
    int64_t sum = n * pre + n * (a + whole);
    if (m >= count) sum += blocks_of(s, s.lq);
    return sum + static_cast<int64_t>(kExtra) * (m < count ? m : count);
}

// The items of a CTA's run, in order.
struct Walk {
    int64_t left;
    int seq, tile, head, b0;
    Seq s;
    __device__ __forceinline__ Item next(const RaggedArgs& p) {
        Item it = {};
        if (left <= 0) return it;
        while (tile >= tiles_of(s)) {                       // (there is another one, as units are left)
            s = seq_at(p, ++seq);
            tile = 0;
        }
        const int row0 = 256 * tile;
        const int n0 = blocks_of(s, row0 + 128), n = blocks_of(s, row0 + 256), weight = n + kExtra;
        const int take = static_cast<int>(min(left, static_cast<int64_t>(weight - b0))), b1 = b0 + take;
        it.q0 = s.q0 + row0;
        it.k0 = s.k0;
        it.rows = s.lq - row0;
        it.seen = s.lk - s.lq + row0 + 1;
        it.keys = s.lk;
        it.head = head;
        it.from = min(b0, n);
        it.count0 = max(min(b1, n0) - it.from, 0);
        it.count1 = it.rows > 128 ? min(b1, n) - it.from : 0;
        it.slot = b0 > 0 || b1 < weight ? 2 * static_cast<int>(blockIdx.x) + (b0 > 0 ? 0 : 1) : -1;
        it.valid = 1;
        left -= take;
        b0 = 0;
        if (++head == p.heads) head = 0, ++tile;
        return it;
    }
};

// What the warps read of the items: each takes them one behind the other and hands them back.
struct Items {
    Ctl* ctl;
    int at = 0;
    uint32_t phase = 0;
    // nullptr: no more, or given up
    __device__ __forceinline__ const Item* next(uint32_t* status) {
        if (!wait_or_give_up(&ctl->item_full[at], phase, &ctl->abort, status) || ctl->items[at].valid == 0) return nullptr;
        return &ctl->items[at];
    }
    __device__ __forceinline__ void step() {
        if (++at == kItems) at = 0, phase ^= 1u;
    }
    __device__ __forceinline__ void done() {
        mbar_arrive(&ctl->item_empty[at]);
        step();
    }
};

// One warp: where the CTA's run begins. Also its header, where the run's last tile goes on in the next run.
__device__ __forceinline__ Walk find_run(const KernelArgs& a, int lane) {
    const RaggedArgs& p = a.p;
    const unsigned full = 0xffffffffu;
    int64_t total = 0, mine = 0;
    for (int b = 0; b < p.batch; b += 32) {
        int64_t n = 0;
        if (b + lane < p.batch) {
            const Seq s = seq_at(p, b + lane);
            n = units_of(s, tiles_of(s));
        }
        mine = n;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(full, n, o);
        total += n;
    }
    total *= p.heads;
    // (a run has at least kMinRun units: shorter ones would be all parts and joining)
    const int64_t most = (total + kMinRun - 1) / kMinRun, g = most < gridDim.x ? most : gridDim.x, c = blockIdx.x;
    const int64_t u0 = c < g ? total * c / g : 0, u1 = c < g ? total * (c + 1) / g : 0;
    // the sequences that the first and the last unit lie in
    int seq0 = 0, seq1 = 0;
    int64_t at0 = 0, at1 = 0;
    if (u1 > u0) {
        int64_t before = 0;
        bool found0 = false, found1 = false;
        for (int b = 0; b < p.batch && !(found0 && found1); b += 32) {
            int64_t n = mine * p.heads;                     // (of the only 32 sequences, or else read again)
            if (p.batch > 32) {
                n = 0;
                if (b + lane < p.batch) {
                    const Seq s = seq_at(p, b + lane);
                    n = units_of(s, tiles_of(s)) * p.heads;
                }
            }
            int64_t sum = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(full, sum, o);
                if (lane >= o) sum += v;
            }
            const unsigned m0 = __ballot_sync(full, before + sum > u0), m1 = __ballot_sync(full, before + sum > u1 - 1);
            if (!found0 && m0 != 0u) {
                const int lane0 = __ffs(m0) - 1;
                seq0 = b + lane0;
                at0 = before + __shfl_sync(full, sum - n, lane0);
                found0 = true;
            }
            if (!found1 && m1 != 0u) {
                const int lane1 = __ffs(m1) - 1;
                seq1 = b + lane1;
                at1 = before + __shfl_sync(full, sum - n, lane1);
                found1 = true;
            }
            before += __shfl_sync(full, sum, 31);
        }
    }
    Walk first = {};
    int4 header = make_int4(0, 0, 0, 0);
    if (u1 > u0) {
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
            const int seq = e == 0 ? seq0 : seq1;
            const Seq s = seq_at(p, seq);
            const int64_t off = e == 0 ? u0 - at0 : u1 - 1 - at1;
            int lo = 0, hi = tiles_of(s);                   // units_of(lo) * heads <= off < units_of(hi) * heads
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (units_of(s, mid) * p.heads <= off) lo = mid;
                else hi = mid;
            }
            const int64_t in_tile = off - units_of(s, lo) * p.heads;
            const int weight = blocks_of(s, 256 * lo + 256) + kExtra;
            const int head = static_cast<int>(in_tile / weight), b = static_cast<int>(in_tile - static_cast<int64_t>(head) * weight);
            if (e == 0) {
                first.left = u1 - u0;
                first.seq = seq, first.tile = lo, first.head = head, first.b0 = b;
                first.s = s;
            } else {
                const int64_t begin = u1 - 1 - b, end = begin + weight;
                if (begin >= u0 && end > u1) {
                    int parts = 1;
                    for (int64_t n = c + 1; n < g && total * n / g < end; ++n) ++parts;
                    header = make_int4(s.q0 + 256 * lo, min(256, s.lq - 256 * lo), head, parts);
                }
            }
        }
    }
    if (lane == 0) a.headers[c] = header;
    return first;
}

// Among four lanes that hold four 16-byte chunks of a row each: lane j's chunk e becomes lane e's chunk j, so that the lanes then hold
// 64 bytes of one row (a warp's stores of 32 bytes in 32 rows take 130 cycles each; and this code, which runs once a tile, has
// to be short, as it comes from beyond the instruction caches).
__device__ __forceinline__ void transpose4(uint32_t (&x)[4][4], int lane) {
#pragma unroll
    for (int s = 1; s < 4; s <<= 1) {
        const bool up = (lane & s) != 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e & s) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x[e][k] : x[e | s][k], s);
                x[e][k] = up ? got : x[e][k];
                x[e | s][k] = up ? x[e | s][k] : got;
            }
        }
    }
}

// Moves the references m of a warp's rows up to `top` (log2 units; -inf: they stay), to the next whole number, and scales what was weighed
// against the old ones: the row's sum l, its output (where there is one) and the quarters of P that are written. The factors
// are powers of two, so nothing is rounded by it.
__device__ __forceinline__ void move_reference(float top, float& m, float& l, bool outputs, int quarters, uint32_t s_addr, uint32_t o_addr) {
    float alpha = 1.0f;
    if (top > m) {
        const float to = ceilf(top);
        alpha = m - to >= -126.0f ? __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(m - to)) << 23) : 0.0f;
        m = to;
    }
    l *= alpha;
    if (outputs) {
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld16(o_addr + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(o_addr + 16 * c, o);
        }
    }
    const __nv_bfloat162 a2 = __float2bfloat162_rn(alpha);
#pragma unroll 1
    for (int c = 0; c < quarters; ++c) {
        tmem_wait_st();
        uint32_t w[16];
        tmem_ld16(s_addr + 16 * c, w);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]), a2);
            w[e] = *reinterpret_cast<const uint32_t*>(&x);
        }
        tmem_st16(s_addr + 16 * c, w);
    }
}

__global__ void __launch_bounds__(kThreads, 1) ragged_attention_kernel(const __grid_constant__ KernelArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];   // (there is no static shared memory: it begins at a multiple of 1024)
    uint8_t* smem = smem_raw;
    Ctl* ctl = reinterpret_cast<Ctl*>(smem);
    const uint32_t sbase = smem_addr(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const RaggedArgs& p = a.p;
    if (warp == kWarpLoad && lane == 0) {
        prefetch_map(&a.q_map);
        prefetch_map(&a.k_map);
        prefetch_map(&a.v_map);
        prefetch_map(&a.pe_map);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->k_full[i], 1), mbar_init(&ctl->k_empty[i], 2), mbar_init(&ctl->v_full[i], 1), mbar_init(&ctl->v_empty[i], 3);
            mbar_init(&ctl->q_full[i], 1), mbar_init(&ctl->q_free[i], 1);
            mbar_init(&ctl->s_full[i], 1), mbar_init(&ctl->p_full[i], 4), mbar_init(&ctl->o_done[i], 1), mbar_init(&ctl->turn[i], 1), mbar_init(&ctl->v_clean[i], 1);
        }
        for (int i = 0; i < kItems; ++i) mbar_init(&ctl->item_full[i], 1), mbar_init(&ctl->item_empty[i], 11);   // 8 softmax warps, two issuers, loads
        mbar_init(&ctl->drain, 2);
        ctl->abort = 0u;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(&ctl->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;
    uint32_t* abort = &ctl->abort;
    uint32_t* status = p.status;

    if (warp >= kWarpLoad) {
        if (warp == kWarpLoad) {
            if (lane == 0) {
                // Eight units hold three groups in flight: the keys of block g lie where the values of block g - 2 and what came before lay,
                // the values of block g where the keys of block g - 1 lay.
                int unit = 0, g = 0;
                uint32_t q_phase = 3;                        // one bit for each half
                auto step = [&] { unit = unit + 1 == kUnits ? 0 : unit + 1; };
                Items items = {ctl};
                for (const Item* next = items.next(status); next != nullptr; items.done(), next = items.next(status)) {
                    const Item it = *next;
                    const int n = max(it.count0, it.count1);
                    if (n == 0) continue;
                    auto load_q = [&](int h) -> bool {
                        if ((h == 0 ? it.count0 : it.count1) == 0) return true;
                        if (!wait_or_give_up(&ctl->q_free[h], (q_phase >> h) & 1, abort, status)) return false;
                        q_phase ^= 1u << h;
                        mbar_arrive_expect_tx(&ctl->q_full[h], 3 * kBox);
                        for (int c = 0; c < 3; ++c)
                            tma_load_3d(sbase + kOffQ + (3 * h + c) * kBox, &a.q_map, 64 * c, it.head, it.q0 + 128 * h, &ctl->q_full[h]);
                        return true;
                    };
                    auto load_k = [&](int i) -> bool {
                        if (g >= 2 && !wait_or_give_up(&ctl->v_empty[g & 1], ((g >> 1) & 1) ^ 1, abort, status)) return false;
                        const int row = it.k0 + 128 * (it.from + i);
                        uint64_t* bar = &ctl->k_full[g & 1];
                        mbar_arrive_expect_tx(bar, 3 * kBox);
                        for (int c = 0; c < 3; ++c, step()) {
                            if (c < 2) tma_load_3d(sbase + kOffRing + unit * kBox, &a.k_map, 64 * c, it.head, row, bar);
                            else tma_load_3d(sbase + kOffRing + unit * kBox, &a.pe_map, 0, 0, row, bar);
                        }
                        return true;
                    };
                    auto load_v = [&](int i) -> bool {
                        if (g >= 1 && !wait_or_give_up(&ctl->k_empty[(g - 1) & 1], ((g - 1) >> 1) & 1, abort, status)) return false;
                        const int row = it.k0 + 128 * (it.from + i);
                        uint64_t* bar = &ctl->v_full[g & 1];
                        mbar_arrive_expect_tx(bar, 2 * kBox);
                        for (int c = 0; c < 2; ++c, step()) {
                            tma_load_3d(sbase + kOffRing + unit * kBox, &a.v_map, 128, it.head, row + 64 * c, bar);
                            tma_load_3d(sbase + kOffRing + unit * kBox + kBox / 2, &a.v_map, 192, it.head, row + 64 * c, bar);
                        }
                        ++g;
                        return true;
                    };
                    bool ok = load_q(0) && load_k(0) && load_q(1) && load_v(0);
                    for (int i = 1; i < n && ok; ++i) ok = load_k(i) && load_v(i);
                    if (!ok) break;
                }
            }
            __syncwarp();
        } else if (warp >= kWarpMma) {
            // Each half has an issuer of its own: a product's issue blocks until the tensor cores take it, and what lies between two chains (waits,
            // commits, instruction fetches: 150 to 300 cycles each) would leave them idle; now the other half's chain runs meanwhile.
            if (elect_one_in_warp()) {
                const int h = warp - kWarpMma;
                // (a negative scale negates the queries in the product: bit 13)
                const uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false) | (p.sm_scale < 0.0f ? 1u << 13 : 0u);
                constexpr uint32_t idesc_o = idesc_bf16_f32(128, 128, false, true);
                const uint64_t q0 = sdesc_sw128(sbase + kOffQ + 3 * h * kBox, 16, 1024);   // K-major: rows x dims
                const uint64_t k0 = sdesc_sw128(sbase + kOffRing, 16, 1024);               // K-major: keys x dims
                const uint64_t v0 = sdesc_sw128(sbase + kOffRing, kBox / 2, 1024);         // MN-major: dims x keys
                const uint32_t s_addr = tmem + kColS + 128 * h, o_addr = tmem + kColO + 128 * h;
                int unit = 0, g = 0, cleans = 0;                                           // g: blocks whose values were waited for
                uint32_t q_phase = 0, p_phase = 0, turn_phase = h == 0 ? 1u : 0u;
                auto scores = [&](int at) {                 // S from the three units at `at`
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < 3; ++c) {
                        const uint64_t qd = q0 + static_cast<uint32_t>(c * (kBox >> 4)), kd = k0 + static_cast<uint32_t>(((at + c) & (kUnits - 1)) * (kBox >> 4));
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) mma_ss(s_addr, qd + 2 * ks, kd + 2 * ks, idesc_s, c > 0 || ks > 0 ? 1u : 0u);
                    }
                    mma_commit(&ctl->s_full[h]);
                };
                Items items = {ctl};
                bool ok = true;
                for (const Item* next = items.next(status); next != nullptr; items.done(), next = items.next(status)) {
                    const int n = max(next->count0, next->count1), count = h == 0 ? next->count0 : next->count1;
                    const int whole = (next->keys >> 7) - next->from;      // blocks before the one that the sequence ends in
                    if (n == 0) continue;
                    if (count > 0) {                        // the first block's scores
                        ok = wait_or_give_up(&ctl->k_full[g & 1], (g >> 1) & 1, abort, status) && wait_or_give_up(&ctl->q_full[h], q_phase, abort, status);
                        if (!ok) break;
                        q_phase ^= 1u;
                    }
                    ok = wait_or_give_up(&ctl->turn[h], turn_phase, abort, status);
                    if (!ok) break;
                    turn_phase ^= 1u;
                    if (count > 0) {
                        scores(unit);
                        if (count == 1) mma_commit(&ctl->q_free[h]);
                    }
                    mbar_arrive(&ctl->turn[h ^ 1]);
                    mma_commit(&ctl->k_empty[g & 1]);
#pragma unroll 1
                    for (int i = 0; i < n; ++i, ++g) {
                        ok = wait_or_give_up(&ctl->v_full[g & 1], (g >> 1) & 1, abort, status);
                        if (ok && i >= whole) {
                            ok = wait_or_give_up(&ctl->v_clean[cleans & 1], (cleans >> 1) & 1, abort, status);
                            ++cleans;
                        }
                        if (!ok) break;
                        bool keys_here = false;
                        if (i < count) {                    // O (+)= P V
                            // (the next keys are mostly there already: seen to while P is not)
                            keys_here = i + 1 < count && mbar_test_wait(&ctl->k_full[(g + 1) & 1], ((g + 1) >> 1) & 1);
                            ok = wait_or_give_up(&ctl->p_full[h], p_phase, abort, status);
                            if (!ok) break;
                            p_phase ^= 1u;
                        }
                        ok = wait_or_give_up(&ctl->turn[h], turn_phase, abort, status);
                        if (!ok) break;
                        turn_phase ^= 1u;
                        if (i < count) {
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int c = 0; c < 2; ++c) {
                                const uint64_t vd = v0 + static_cast<uint32_t>(((unit + 3 + c) & (kUnits - 1)) * (kBox >> 4));
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks)
                                    mma_ts(o_addr, s_addr + 32 * c + 8 * ks, vd + 128 * ks, idesc_o, i == 0 && c == 0 && ks == 0 ? 0u : 1u);
                            }
                            if (i + 1 == count) mma_commit(&ctl->o_done[h]);
                        }
                        mma_commit(&ctl->v_empty[g & 1]);
                        unit = (unit + 5) & (kUnits - 1);
                        if (i + 1 < count) {
                            ok = keys_here || wait_or_give_up(&ctl->k_full[(g + 1) & 1], ((g + 1) >> 1) & 1, abort, status);
                            if (!ok) break;
                            scores(unit);
                            if (i + 2 == count) mma_commit(&ctl->q_free[h]);
                        }
                        mbar_arrive(&ctl->turn[h ^ 1]);
                        if (i + 1 < n) mma_commit(&ctl->k_empty[(g + 1) & 1]);
                    }
                    if (!ok) break;
                }
                mma_commit(&ctl->drain);
                wait_or_give_up(&ctl->drain, 0, abort, status);
            }
            __syncwarp();
        } else if (warp == kWarpFix) {
            // The CTA's items, one ahead of the one that is worked on.
            Walk walk = find_run(a, lane);
            int slot = 0;
            uint32_t slot_phase = 1;
            auto publish = [&](const Item& it) -> bool {
                if (!wait_warp(&ctl->item_empty[slot], slot_phase, abort, status)) return false;
                if (lane == 0) {
                    ctl->items[slot] = it;
                    mbar_arrive(&ctl->item_full[slot]);
                }
                if (++slot == kItems) slot = 0, slot_phase ^= 1u;
                return true;
            };
            // Values behind a sequence's end belong to other sequences or to nobody and may be anything: zeros, as 0 x NaN is NaN.
            // (The warp takes note of every block and hands it back beside the products, so that it stays within the ring.)
            int unit = 0, g = 0, cleans = 0;
            Item it = walk.next(p);
            bool ok = publish(it);
            while (ok && it.valid) {
                const Item ahead = walk.next(p);
                ok = publish(ahead);
                const int n = max(it.count0, it.count1);
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i, ++g) {
                    const int left = it.keys - 128 * (it.from + i);
                    unit = (unit + 3) & (kUnits - 1);
                    ok = wait_warp(&ctl->v_full[g & 1], (g >> 1) & 1, abort, status);
                    if (!ok) break;
                    if (left < 128) {
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t base = sbase + kOffRing + ((unit + c) & (kUnits - 1)) * kBox;
                            for (int x = max(left - 64 * c, 0) * 8 + lane; x < 64 * 8; x += 32) {
                                sts_u128(base + 16 * x, make_uint4(0u, 0u, 0u, 0u));
                                sts_u128(base + kBox / 2 + 16 * x, make_uint4(0u, 0u, 0u, 0u));
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctl->v_clean[cleans & 1]);
                        ++cleans;
                    }
                    unit = (unit + 2) & (kUnits - 1);
                    if (lane == 0) mbar_arrive(&ctl->v_empty[g & 1]);
                }
                it = ahead;
            }
        }
    } else {
        const int h = warp >> 2, w = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * w) << 16);
        const uint32_t s_addr = lanes + kColS + 128 * h, o_addr = lanes + kColO + 128 * h;
        const float mul = p.sm_scale == 0.0f ? 1e-30f : fabsf(p.sm_scale) * kLog2e;   // (0 x -inf would be NaN where a key is masked)
        int seen = 0;                  // blocks of this half so far
        uint32_t done = 0;             // and tiles
        Items items = {ctl};
        bool ok = true;
        for (;;) {
            const Item* const it = items.next(status);
            if (it == nullptr) break;
            const int n = h == 0 ? it->count0 : it->count1;
            // keys that the row, and the half's first row, see of those from the first block on
            const int limit = min(it->seen + 128 * h + 32 * w + lane, it->keys) - 128 * it->from;
            const int first_limit = it->seen + 128 * h - 128 * it->from;
            float m = -INFINITY, l = 0.0f, top = -INFINITY;   // top: what the reference moves up to, if anything
            for (int i = 0; i < n; ++i, ++seen) {
                ok = wait_warp(&ctl->s_full[h], seen & 1, abort, status);
                if (!ok) break;
                tc_fence_after_sync();
                // The reference follows a block behind: weights up to 2^kMoveLog2 above it are as good as others in bf16 and fp32, so that nobody
                // has to wait for a block's largest score before its weights. (These scores are there, so the last P V is done.)
                float most = -INFINITY;
                if (__any_sync(0xffffffffu, top > m)) move_reference(top, m, l, i > 0, 0, s_addr, o_addr);
                uint64_t la = f32x2_pack(0.0f, 0.0f), lb = la;
                // 32 keys at a time in a short loop (unrolled as a whole, the code would push the issuers' out of the instruction caches); P of a
                // quarter goes over scores that were read already.
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t s[32], pw[16];
                    tmem_ld32_wait(s_addr + 32 * c, s);
                    if (128 * i + 32 * c + 32 > first_limit) {
                        const int keep = limit - 128 * i - 32 * c;
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[e] = e < keep ? s[e] : __float_as_uint(-INFINITY);
                    }
                    float t0 = -INFINITY, t1 = t0;
                    uint64_t pa, pb;
                    for (;;) {
                        const float neg_m = m == -INFINITY ? 0.0f : -m;
                        const uint64_t mul2 = f32x2_pack(mul, mul), neg2 = f32x2_pack(neg_m, neg_m);
                        pa = la, pb = lb;
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float2 z0 = f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), mul2, neg2));
                            const float2 z1 = f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), mul2, neg2));
                            const float e0 = ex2_approx(z0.x), e1 = ex2_approx(z0.y), e2 = ex2_approx(z1.x), e3 = ex2_approx(z1.y);
                            pa = f32x2_add(pa, f32x2_pack(e0, e1));
                            pb = f32x2_add(pb, f32x2_pack(e2, e3));
                            pw[e / 2] = pack_bf16x2(e0, e1);
                            pw[e / 2 + 1] = pack_bf16x2(e2, e3);
                            t0 = fmax3(t0, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                            t1 = fmax3(t1, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
                        }
                        top = fmaxf(t0, t1) * mul;
                        if (!__any_sync(0xffffffffu, top > m + kFarLog2)) break;
                        // too far above (or the first keys that the row sees): the reference moves now, and these weights are worked out again
                        const float2 sa = f32x2_unpack(la), sb = f32x2_unpack(lb);
                        l += (sa.x + sa.y) + (sb.x + sb.y);
                        la = lb = f32x2_pack(0.0f, 0.0f);
                        move_reference(top > m + kFarLog2 ? top : -INFINITY, m, l, i > 0, c, s_addr, o_addr);
                    }
                    la = pa, lb = pb;
                    most = fmaxf(most, top);
                    tmem_st16(s_addr + 16 * c, pw);
                }
                top = most > m + kMoveLog2 ? most : -INFINITY;
                const float2 sa = f32x2_unpack(la), sb = f32x2_unpack(lb);
                l += (sa.x + sa.y) + (sb.x + sb.y);
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->p_full[h]);
            }
            if (n > 0) {
                ok = ok && wait_warp(&ctl->o_done[h], done++ & 1, abort, status);
                if (!ok) break;
                tc_fence_after_sync();
            }
            const int rows = it->rows - 128 * h - 32 * w;      // of this warp (32 and more: all)
            const int head = it->head, slot = it->slot;
            const bool empty = l == 0.0f;
            const float lse2 = empty ? -INFINITY : m + log2f(l);
            float f = empty ? 0.0f : 1.0f / l;
            if (slot < 0 && !empty && p.attn_sink != nullptr) f = 1.0f / (l + exp2f(__ldg(p.attn_sink + head) * kLog2e - m));
            const bool none = n == 0 || empty;
            if (slot >= 0 && rows > 0) {
                a.part_lse[static_cast<int64_t>(slot) * 256 + 128 * h + 32 * w + lane] = lse2;
                float* dst = a.part_out + (static_cast<int64_t>(slot) * 8 + 4 * h + w) * 4096 + 8 * lane;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    tmem_ld32_wait(o_addr + 32 * c, o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = none ? 0u : __float_as_uint(__uint_as_float(o[e]) * f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) st_sector(dst + (4 * c + e) * 256, o + 8 * e);
                }
            } else if (rows > 0) {
                const int64_t at = static_cast<int64_t>(it->q0 + 128 * h + 32 * w) * p.heads + head;   // of lane 0's row
                if (lane < rows) p.lse[at + static_cast<int64_t>(lane) * p.heads] = lse2 * kLn2;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32], x[4][4];
                    tmem_ld32_wait(o_addr + 32 * c, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        x[e >> 2][e & 3] = none ? 0u : pack_bf16x2(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
                    transpose4(x, lane);
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (at + static_cast<int64_t>(lane & 28) * p.heads) * 128 + 32 * c + 8 * (lane & 3);
#pragma unroll
                    for (int e = 0; e < 4; ++e, dst += 128 * p.heads)
                        if ((lane & 28) + e < rows) *reinterpret_cast<uint4*>(dst) = make_uint4(x[e][0], x[e][1], x[e][2], x[e][3]);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->item_empty[items.at]);
            items.step();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (*reinterpret_cast<volatile uint32_t*>(abort) != 0u) let_copies_land();
    if (warp == kWarpMma) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the parts of a tile that was cut: with part s's lse L_s (log2) and output O_s, w_s = 2^(L_s - max L),
// out = sum_s w_s O_s / (sum_s w_s + 2^(sink - max L)). The first part of header c lies in slot 2c + 1, the others in slots
// 2 (c + 1), 2 (c + 2), ... A lane per row and 16 dims, in the parts' order.
__global__ void __launch_bounds__(256) ragged_join_kernel(const float* __restrict__ part_out, const float* __restrict__ part_lse,
                                                          const int4* __restrict__ headers, const float* __restrict__ sink, int heads,
                                                          __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");   // (all CTAs of this grid are resident at once: nothing of it waits for an SM)
    const int c = blockIdx.x, lane = threadIdx.x & 31, dims = threadIdx.x >> 5, r = 32 * blockIdx.y + lane;
    const int4 hd = __ldcg(headers + c);
    if (hd.w == 0 || r >= hd.y) return;
    auto slot = [&](int s) { return static_cast<int64_t>(s == 0 ? 2 * c + 1 : 2 * (c + s)); };
    auto lse_of = [&](int s) { return __ldcg(part_lse + slot(s) * 256 + r); };
    float m = -INFINITY;
    for (int s = 0; s < hd.w; ++s) m = fmaxf(m, lse_of(s));
    if (m == -INFINITY) m = 0.0f;
    float sum = 0.0f, acc[16] = {};
#pragma unroll 2
    for (int s = 0; s < hd.w; ++s) {
        const float w = exp2f(lse_of(s) - m);
        const float4* x = reinterpret_cast<const float4*>(part_out + (slot(s) * 8 + blockIdx.y) * 4096 + 512 * dims + 8 * lane);
        const float4 v[4] = {__ldcg(x), __ldcg(x + 1), __ldcg(x + 64), __ldcg(x + 65)};
        sum += w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc[4 * e] = fmaf(w, v[e].x, acc[4 * e]);
            acc[4 * e + 1] = fmaf(w, v[e].y, acc[4 * e + 1]);
            acc[4 * e + 2] = fmaf(w, v[e].z, acc[4 * e + 2]);
            acc[4 * e + 3] = fmaf(w, v[e].w, acc[4 * e + 3]);
        }
    }
    const float denom = sink != nullptr ? sum + exp2f(__ldg(sink + hd.z) * kLog2e - m) : sum;
    const float f = sum == 0.0f ? 0.0f : 1.0f / denom;
    uint32_t o[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(f != 0.0f ? acc[e] * f : 0.0f);
    const int64_t at = static_cast<int64_t>(hd.x + r) * heads + hd.z;
    st_bf16x16(out + at * 128 + 16 * dims, o, 1.0f);
    if (dims == 0) lse[at] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

constexpr size_t kPartsBytes = static_cast<size_t>(2 * kMaxCtas) * 256 * 128 * sizeof(float);
constexpr size_t kLseBytes = static_cast<size_t>(2 * kMaxCtas) * 256 * sizeof(float);

}  // namespace

size_t ragged_workspace_bytes() { return kPartsBytes + kLseBytes + kMaxCtas * sizeof(int4); }

cudaError_t launch_ragged_attention(const RaggedArgs& p, void* workspace, int sms, cudaStream_t stream) {
    KernelArgs a;
    a.p = p;
    a.part_out = static_cast<float*>(workspace);
    a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kPartsBytes);
    a.headers = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + kPartsBytes + kLseBytes);
    const int64_t rows_k = p.rows_k > 0 ? p.rows_k : 1;      // (no row is read where there is none)
    if (!encode_map(&a.q_map, p.q, 192, p.heads, p.rows_q, p.q_head_stride, p.q_token_stride, 1, 128) ||
        !encode_map(&a.k_map, p.kv, 256, p.heads, rows_k, p.kv_head_stride, p.kv_token_stride, 1, 128) ||
        !encode_map(&a.v_map, p.kv, 256, p.heads, rows_k, p.kv_head_stride, p.kv_token_stride, 1, 64) ||
        !encode_map(&a.pe_map, p.k_pe, 64, 1, rows_k, 64, p.pe_stride, 1, 128))
        return cudaErrorInvalidValue;
    cudaError_t err = allow_smem<ragged_attention_kernel>(kSmem);
    if (err != cudaSuccess) return err;
    const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
    err = launch_dependent(ragged_attention_kernel, dim3(ctas), kThreads, kSmem, 1, stream, a);
    if (err != cudaSuccess) return err;
    return launch_dependent(ragged_join_kernel, dim3(ctas, 8), 256, 0, 1, stream, static_cast<const float*>(a.part_out),
                            static_cast<const float*>(a.part_lse), static_cast<const int4*>(a.headers), p.attn_sink, p.heads,
                            static_cast<__nv_bfloat16*>(p.out), p.lse);
}

}  // namespace nvfp4mla

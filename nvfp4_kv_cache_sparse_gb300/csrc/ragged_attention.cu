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
// and feeds P V from tensor memory. While one half's softmax runs, the tensor cores work for the other: the halves' chains (P V of a
// block, S of the next) take turns. Keys and values come through a ring of eight 16 KB units (a key block is three units of 128 keys x
// 64 dims, its values two units of 64 keys x 128 dims).
// What bounds one CTA is that ring: a block's keys can be sent for only when both halves are done with the values of the block
// before the last, some 1300 cycles before they are needed (waits of 500 to 1000 cycles a block of 3550, of which the products
// take 2560). So long sequences go to CTA pairs (kPair): tiles of 512 rows in halves of 256 (M = 256, tcgen05.mma on the pair), each CTA
// with its own 128 rows of either half and half of the keys and values, three blocks of them in flight, and half the reads from L2.
//
// Tiles are of very different lengths and often fewer than SMs, so the CTAs (or pairs), one per SM, take equal runs of (tile, head, block
// of 128 keys) units, heads inside tiles: neighbouring tiles of a head are then read by several CTAs at about the same
// time, from L2. A tile that two runs share leaves fp32 parts in the workspace, which a second kernel joins.
//
// 2048 rows over 16640 keys, 64 heads: 760 us in a short run, 1.72 PFLOP/s (one CTA each: 868), 870 to 890 in a long one, where power limits the
// clock; 4 chunks of 512 rows over 500 to 16000 keys, 16 heads: 139 to 154 us, 1.31 to 1.45 PFLOP/s (one CTA each: 159); 16 prompts of 30 to 700 tokens,
// 16 heads: 45 to 48 us on one CTA each, where a tile's first loads, its softmax and its way out (4 us) count more than its few blocks.
#include "head_tiles.cuh"
#include "launch.h"

namespace nvfp4mla {
namespace {

using namespace tiles;

constexpr int kUnits = 8;              // ring of one CTA
constexpr int kOffQ = 1024;
constexpr int kOffRing = kOffQ + 6 * kBox;
constexpr int kSmem = kOffRing + kUnits * kBox;
static_assert(kSmem <= 232448, "shared memory");
// One CTA or a pair (kPair): rows of a half and of a tile, blocks of keys, and of values, that the ring holds.
template <bool kPair> constexpr int kHalf = kPair ? 256 : 128;
template <bool kPair> constexpr int kTile = 2 * kHalf<kPair>;
template <bool kPair> constexpr int kDepth = kPair ? 3 : 2;
constexpr int kPairK = 3 * kBox / 2, kOffPairV = kOffRing + 3 * kPairK;   // a pair's CTA: 64 keys x 192 dims, then 128 keys x 64 dims of values
static_assert(kOffPairV + 3 * kBox <= kSmem, "shared memory");
constexpr int kWarpLoad = 8, kWarpFix = 9, kWarpMma = 10;    // 10 and 11: products of the two halves; 0-3 and 4-7: their softmax
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;              // two halves of 128 columns each
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMoveLog2 = 8.0f;      // a reference moves, a block later, when a score passes it by 2^8,
constexpr float kFarLog2 = 64.0f;      // and at once when one passes it by 2^64
constexpr int kExtra = 1;              // what a tile costs besides its blocks, in blocks
constexpr int kMinRun = 2;
constexpr int kWhole = 6;              // tiles of up to so many units are not cut
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
    // Block g of the run uses entry g % kDepth of each. k_full, v_ready, q_full, p_full, turn and drain count in CTA 0 of a pair, where the
    // products are issued; what those hand back is counted in both CTAs.
    uint64_t k_full[3], k_empty[3], v_empty[3];   // (both issuers hand a block back)
    uint64_t v_full[3], v_ready[3];    // this CTA's values landed; they are clean (from each CTA)
    uint64_t q_full[2], q_free[2];     // a half's queries landed; its last scores are done
    uint64_t s_full[2];                // scores in tensor memory
    uint64_t p_full[2];                // 4 warps of each CTA: P written, O rescaled
    uint64_t turn[2];                  // the other half's chain of products is issued
    uint64_t o_done[2];                // a tile's last P V is done
    uint64_t drain;
    uint64_t item_full[kItems], item_empty[kItems];
    uint32_t tmem_base, abort;
    Item items[kItems];                // what the CTA works on, one behind the other
    int bad[16];                       // of item k with blocks (entry k % 16): its first key with a value that is not finite and was taken out
};
static_assert(sizeof(Ctl) <= kOffQ, "control block");

struct KernelArgs {
    CUtensorMap q_map;                 // [rows_q, heads, 192], box 128 x 1 x 64
    CUtensorMap k_map;                 // kv [rows_k, heads, 256], box 128 x 1 x 64; for a pair 64 x 1 x 64
    CUtensorMap v_map;                 // the same, box 64 x 1 x 64; for a pair 128 x 1 x 64
    CUtensorMap pe_map;                // [rows_k, 1, 64], box as k_map's
    RaggedArgs p;
    float* part_out;                   // [2 runs, rows of a tile / 32, 16, 32 lanes, 8]: eight dims of a row, divided by its own sum
    float* part_lse;                   // [2 runs, rows of a tile], log2
    int4* headers;                     // [runs]: first output row, rows, head, parts (0: no tile begins here and ends elsewhere)
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
template <bool kPair>
__device__ __forceinline__ int tiles_of(const Seq& s) { return (s.lq + kTile<kPair> - 1) / kTile<kPair>; }
// Key blocks of rows [0, rows) of a sequence: its last row sees the first lk - lq + rows keys.
__device__ __forceinline__ int blocks_of(const Seq& s, int rows) {
    const int keys = s.lk - s.lq + min(rows, s.lq);
    return keys <= 0 ? 0 : (keys + 127) >> 7;
}
// Units of the first m tiles: a tile before the last one ends on a multiple of kTile rows, tile j has max(0, p + r (j + 1)) blocks
// with p = ceil((lk - lq) / 128) and r = kTile / 128, and kExtra.
template <bool kPair>
__device__ __forceinline__ int64_t units_of(const Seq& s, int m) {
    constexpr int r = kTile<kPair> / 128;
    const int count = tiles_of<kPair>(s);
    if (m <= 0) return 0;
    const int whole = m < count ? m : count - 1;            // tiles that are surely full
    const int64_t pre = (s.lk - s.lq + 127) >> 7;           // (rounds up for negative ones too)
    int64_t none = pre < 0 ? -pre / r : 0;                  // tiles without keys
    if (none > whole) none = whole;
    const int64_t a = none + 1, n = whole - none;           // j + 1 = a .. whole
    int64_t sum = n * pre + (r / 2) * n * (a + whole);
    if (m >= count) sum += blocks_of(s, s.lq);
    return sum + static_cast<int64_t>(kExtra) * (m < count ? m : count);
}

// The items of a run (a CTA's, or a pair's), in order.
template <bool kPair>
struct Walk {
    int64_t left;
    int seq, tile, head, b0;
    Seq s;
    __device__ __forceinline__ Item next(const RaggedArgs& p, int run, int lane) {   // (of the whole warp)
        Item it = {};
        if (left <= 0) return it;
        while (tile >= tiles_of<kPair>(s)) {                       // the next sequence with rows, 32 lengths at a time
            if (seq + 1 >= p.batch) {
                left = 0;
                return it;
            }
            const int b = seq + 1 + lane;
            const unsigned rows = __ballot_sync(0xffffffffu, b < p.batch && seq_at(p, b).lq > 0);
            seq += rows != 0u ? __ffs(rows) : 32;
            if (rows != 0u) s = seq_at(p, seq), tile = 0;
        }
        const int row0 = kTile<kPair> * tile;
        const int n0 = blocks_of(s, row0 + kHalf<kPair>), n = blocks_of(s, row0 + kTile<kPair>), weight = n + kExtra;
        const int take = static_cast<int>(min(left, static_cast<int64_t>(weight - b0))), b1 = b0 + take;
        it.q0 = s.q0 + row0;
        it.k0 = s.k0;
        it.rows = s.lq - row0;
        it.seen = s.lk - s.lq + row0 + 1;
        it.keys = s.lk;
        it.head = head;
        it.from = min(b0, n);
        it.count0 = max(min(b1, n0) - it.from, 0);
        it.count1 = it.rows > kHalf<kPair> ? min(b1, n) - it.from : 0;
        it.slot = b0 > 0 || b1 < weight ? 2 * run + (b0 > 0 ? 0 : 1) : -1;
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
    // nullptr: no more, or given up. For one thread, or for a whole warp with one answer.
    template <bool kWarp = false>
    __device__ __forceinline__ const Item* next(uint32_t* status) {
        const bool there = kWarp ? wait_warp(&ctl->item_full[at], phase, &ctl->abort, status) : wait_or_give_up(&ctl->item_full[at], phase, &ctl->abort, status);
        return there && ctl->items[at].valid != 0 ? &ctl->items[at] : nullptr;
    }
    __device__ __forceinline__ void step() {
        if (++at == kItems) at = 0, phase ^= 1u;
    }
    __device__ __forceinline__ void done() {
        mbar_arrive(&ctl->item_empty[at]);
        step();
    }
};

// One warp: where run c of `runs` begins and ends. Also its header, where the run's last tile goes on in the next run. Runs are equal in units, but
// where a border falls into a tile of at most kWhole units it goes to the nearer end of that tile: writing and joining parts costs more.
template <bool kPair>
__device__ __forceinline__ Walk<kPair> find_run(const KernelArgs& a, int c, int runs, int lane) {
    const RaggedArgs& p = a.p;
    const unsigned full = 0xffffffffu;
    Seq mine = {};
    int64_t total = 0, n = 0;
    for (int b = 0; b < p.batch; b += 32) {
        n = 0;
        if (b + lane < p.batch) {
            mine = seq_at(p, b + lane);
            n = units_of<kPair>(mine, tiles_of<kPair>(mine));
        }
        int64_t sum = n;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(full, sum, o);
        total += sum;
    }
    total *= p.heads;
    // (a run has at least kMinRun units: shorter ones would be all parts and joining)
    const int64_t most = (total + kMinRun - 1) / kMinRun, g = most < runs ? most : runs;
    // Lanes 0 and 1 (the others like them) look for the two borders.
    const int64_t border = c >= g ? total : total * (c + (lane & 1)) / g;
    const int64_t u0 = __shfl_sync(full, border, 0), u1 = __shfl_sync(full, border, 1);
    int seq = 0;                                            // of this lane's border
    int64_t at = 0;                                         // units before it
    {
        int64_t before = 0;
        bool found0 = false, found1 = false;
        for (int b = 0; b < p.batch && !(found0 && found1); b += 32) {
            if (p.batch > 32) {                             // (else known already)
                n = 0;
                if (b + lane < p.batch) {
                    const Seq s = seq_at(p, b + lane);
                    n = units_of<kPair>(s, tiles_of<kPair>(s));
                }
            }
            int64_t sum = n * p.heads;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(full, sum, o);
                if (lane >= o) sum += v;
            }
            const unsigned m0 = __ballot_sync(full, before + sum > u0), m1 = __ballot_sync(full, before + sum > u1);
            const bool here0 = !found0 && m0 != 0u, here1 = !found1 && m1 != 0u;
            const unsigned m = (lane & 1) == 0 ? m0 : m1;
            const int64_t first = before + __shfl_sync(full, sum - n * p.heads, (__ffs(m) - 1) & 31);
            if ((lane & 1) == 0 ? here0 : here1) seq = b + __ffs(m) - 1, at = first;
            found0 |= here0, found1 |= here1;
            before += __shfl_sync(full, sum, 31);
        }
    }
    Seq s;
    if (p.batch > 32) {
        s = seq_at(p, seq);
    } else {
        s.q0 = __shfl_sync(full, mine.q0, seq), s.lq = __shfl_sync(full, mine.lq, seq);
        s.k0 = __shfl_sync(full, mine.k0, seq), s.lk = __shfl_sync(full, mine.lk, seq);
    }
    int tile = 0, head = 0, b = 0, weight = 0;
    int64_t snapped = total;
    if (border < total) {
        const int64_t off = border - at;
        int lo = 0, hi = tiles_of<kPair>(s);                // units_of(lo) * heads <= off < units_of(hi) * heads
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (units_of<kPair>(s, mid) * p.heads <= off) lo = mid;
            else hi = mid;
        }
        tile = lo;
        const int64_t in_tile = off - units_of<kPair>(s, lo) * p.heads;
        weight = blocks_of(s, kTile<kPair> * (lo + 1)) + kExtra;
        if (in_tile <= 0x7FFFFFFF) head = static_cast<int>(in_tile) / weight;
        else head = static_cast<int>(in_tile / weight);
        b = static_cast<int>(in_tile - static_cast<int64_t>(head) * weight);
        snapped = border;
        if (weight <= kWhole && b > 0) {
            if (2 * b >= weight) snapped += weight - b, ++head;
            else snapped -= b;
            b = 0;
        }
    }
    const int64_t s0 = __shfl_sync(full, snapped, 0), s1 = __shfl_sync(full, snapped, 1);
    Walk<kPair> first = {};
    first.left = s1 - s0;
    first.seq = __shfl_sync(full, seq, 0), first.tile = __shfl_sync(full, tile, 0);
    first.head = __shfl_sync(full, head, 0), first.b0 = __shfl_sync(full, b, 0);
    first.s.q0 = __shfl_sync(full, s.q0, 0), first.s.lq = __shfl_sync(full, s.lq, 0);
    first.s.k0 = __shfl_sync(full, s.k0, 0), first.s.lk = __shfl_sync(full, s.lk, 0);
    if (first.head == p.heads) first.head = 0, ++first.tile;
    if (lane == 1 && (!kPair || cluster_ctarank() == 0)) {
        int4 header = make_int4(0, 0, 0, 0);
        const int64_t begin = s1 - b, end = begin + weight;
        if (b > 0 && begin >= s0) {                         // the run's last tile begins here and ends elsewhere
            int parts = 1;
            for (int64_t r = c + 1; r < g && total * r / g < end; ++r) ++parts;
            header = make_int4(s.q0 + kTile<kPair> * tile, min(kTile<kPair>, s.lq - kTile<kPair> * tile), head, parts);
        }
        a.headers[c] = header;
    }
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

__device__ __forceinline__ void red_min_cluster(uint32_t cluster_saddr, int v) {
    asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" ::"r"(cluster_saddr), "r"(v) : "memory");
}

// A warp looks through 16 KB of bf16 values, rows of 128 bytes (row & last_row is the key's): values that are not finite become zeros.
// Returns the first key that had one, or INT32_MAX.
__device__ __forceinline__ int clean_values(uint32_t base, int last_row, int lane) {
    auto odd = [](uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; };   // bit 15 and 31: exponent all ones
    uint32_t any = 0;
#pragma unroll 8
    for (int x = lane; x < 1024; x += 32) {
        const uint4 v = lds_u128(base + 16 * x);
        any |= odd(v.x) | odd(v.y) | odd(v.z) | odd(v.w);
    }
    if (!__any_sync(0xffffffffu, any != 0u)) return INT32_MAX;
    int key = INT32_MAX;
#pragma unroll 1
    for (int x = lane; x < 1024; x += 32) {
        const uint4 v = lds_u128(base + 16 * x);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        bool here = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t o = odd(w[e]);
            here |= o != 0u;
            w[e] &= ((o & 0x8000u) != 0u ? 0u : 0x0000FFFFu) | ((o & 0x80000000u) != 0u ? 0u : 0xFFFF0000u);
        }
        if (here) {
            sts_u128(base + 16 * x, make_uint4(w[0], w[1], w[2], w[3]));
            key = min(key, (x >> 3) & last_row);
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
    return __reduce_min_sync(0xffffffffu, key);
}

template <bool kPair>
__global__ void __launch_bounds__(kThreads, 1) ragged_attention_kernel(const __grid_constant__ KernelArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];   // (there is no static shared memory: it begins at a multiple of 1024)
    uint8_t* smem = smem_raw;
    Ctl* ctl = reinterpret_cast<Ctl*>(smem);
    const uint32_t sbase = smem_addr(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
    const int run = kPair ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x), runs = kPair ? gridDim.x >> 1 : gridDim.x;
    const RaggedArgs& p = a.p;
    if (warp == kWarpLoad && lane == 0) {
        prefetch_map(&a.q_map);
        prefetch_map(&a.k_map);
        prefetch_map(&a.v_map);
        prefetch_map(&a.pe_map);
        for (int i = 0; i < 3; ++i) {
            mbar_init(&ctl->k_full[i], 1), mbar_init(&ctl->k_empty[i], 2), mbar_init(&ctl->v_empty[i], 2);
            mbar_init(&ctl->v_full[i], 1), mbar_init(&ctl->v_ready[i], kPair ? 2 : 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->q_full[i], 1), mbar_init(&ctl->q_free[i], 1), mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->p_full[i], kPair ? 8 : 4), mbar_init(&ctl->o_done[i], 1), mbar_init(&ctl->turn[i], 1);
        }
        // (an item is read by 8 softmax warps, the loads and, in CTA 0, two issuers)
        for (int i = 0; i < kItems; ++i) mbar_init(&ctl->item_full[i], 1), mbar_init(&ctl->item_empty[i], rank == 0 ? 11 : 9);
        for (int i = 0; i < 16; ++i) ctl->bad[i] = INT32_MAX;
        mbar_init(&ctl->drain, 2);
        ctl->abort = 0u;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        if (kPair) tmem_alloc_cg2(&ctl->tmem_base, kTmemCols), tmem_relinquish_cg2();
        else tmem_alloc(&ctl->tmem_base, kTmemCols), tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    tc_fence_before_sync();
    __syncthreads();
    if (kPair) cluster_sync();             // the peer's barriers are ready
    tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;
    // a commit of the products, counted in both CTAs of a pair
    auto commit = [](uint64_t* bar) {
        if (kPair) mma_commit_cg2(bar, 0x3u);
        else mma_commit(bar);
    };
    // An arrival on a barrier of CTA 0. Weights are in tensor memory: what orders their stores ahead of the products is that they were waited for
    // (tcgen05.wait::st), with tcgen05's own fences ahead of the arrival and behind the issuer's wait. Where nothing else is handed over the
    // arrival itself is relaxed: a release at cluster scope would order shared and global memory, and takes about 1000 cycles.
    auto arrive_first = [](uint64_t* bar, bool relaxed) {
        if (!kPair) mbar_arrive(bar);
        else if (relaxed) mbar_arrive_cluster_relaxed(mapa_shared(smem_addr(bar), 0));
        else mbar_arrive_cluster(mapa_shared(smem_addr(bar), 0));
    };
    uint32_t* abort = &ctl->abort;
    uint32_t* status = p.status;

    if (warp >= kWarpLoad) {
        if (warp == kWarpLoad) {
            if (lane == 0) {
                // One CTA: eight units of the ring hold three groups in flight: the keys of block g lie where the values of block g - 2 and what came before
                // lay, the values of block g where the keys of block g - 1 lay. A pair's CTAs hold half of each block, three blocks of both.
                int unit = 0, g = 0, e = 0;                  // e: g % kDepth
                uint32_t q_phase = 3, phase = 0;             // q_phase: one bit for each half; phase: of entry e
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
                        if (rank == 0) mbar_arrive_expect_tx(&ctl->q_full[h], (kPair ? 6 : 3) * kBox);
                        for (int c = 0; c < 3; ++c) {
                            const uint32_t to = sbase + kOffQ + (3 * h + c) * kBox;
                            const int row = it.q0 + kHalf<kPair> * h + 128 * rank;
                            if (kPair) tma_load_3d_cg2(to, &a.q_map, 64 * c, it.head, row, mapa_shared(smem_addr(&ctl->q_full[h]), 0));
                            else tma_load_3d(to, &a.q_map, 64 * c, it.head, row, &ctl->q_full[h]);
                        }
                        return true;
                    };
                    auto load_k = [&](int i) -> bool {
                        // (one CTA: entry e of v_empty had block g - 2, so its phase is the same as for a pair's k_empty)
                        if (g >= kDepth<kPair> && !wait_or_give_up(kPair ? &ctl->k_empty[e] : &ctl->v_empty[e], phase ^ 1, abort, status)) return false;
                        const int row = it.k0 + 128 * (it.from + i) + 64 * rank;
                        uint64_t* bar = &ctl->k_full[e];
                        if (rank == 0) mbar_arrive_expect_tx(bar, 3 * kBox);
                        for (int c = 0; c < 3; ++c) {
                            const void* map = c < 2 ? &a.k_map : &a.pe_map;
                            const int x = c < 2 ? 64 * c : 0, y = c < 2 ? it.head : 0;
                            if (kPair) {
                                tma_load_3d_cg2(sbase + kOffRing + e * kPairK + c * (kBox / 2), map, x, y, row, mapa_shared(smem_addr(bar), 0));
                            } else {
                                tma_load_3d(sbase + kOffRing + unit * kBox, map, x, y, row, bar);
                                step();
                            }
                        }
                        return true;
                    };
                    auto load_v = [&](int i) -> bool {
                        const int row = it.k0 + 128 * (it.from + i);
                        uint64_t* bar = &ctl->v_full[e];
                        if (kPair) {
                            if (g >= kDepth<kPair> && !wait_or_give_up(&ctl->v_empty[e], phase ^ 1, abort, status)) return false;
                            mbar_arrive_expect_tx(bar, kBox);
                            tma_load_3d(sbase + kOffPairV + e * kBox, &a.v_map, 128 + 64 * rank, it.head, row, bar);
                        } else {
                            // the keys of block g - 1: the other entry, in this phase for e = 1, in the one before for e = 0
                            if (g >= 1 && !wait_or_give_up(&ctl->k_empty[e ^ 1], e == 1 ? phase : phase ^ 1, abort, status)) return false;
                            mbar_arrive_expect_tx(bar, 2 * kBox);
                            for (int c = 0; c < 2; ++c, step()) {
                                tma_load_3d(sbase + kOffRing + unit * kBox, &a.v_map, 128, it.head, row + 64 * c, bar);
                                tma_load_3d(sbase + kOffRing + unit * kBox + kBox / 2, &a.v_map, 192, it.head, row + 64 * c, bar);
                            }
                        }
                        ++g;
                        if (++e == kDepth<kPair>) e = 0, phase ^= 1;
                        return true;
                    };
                    bool ok = load_q(0) && load_k(0) && load_q(1) && load_v(0);
                    for (int i = 1; i < n && ok; ++i) ok = load_k(i) && load_v(i);
                    if (!ok) break;
                }
                // The last arrivals: no barrier of the cluster orders what a commit sends to the other CTA, and it must not reach this CTA's shared
                // memory after the CTA has left. (They come with products that the softmax warps wait for anyway.)
                bool landed = *reinterpret_cast<volatile uint32_t*>(abort) == 0u;
                for (int i = 0; i < kDepth<kPair> && landed; ++i) {
                    landed = wait_or_give_up(&ctl->k_empty[e], phase ^ 1, abort, status) && wait_or_give_up(&ctl->v_empty[e], phase ^ 1, abort, status);
                    if (++e == kDepth<kPair>) e = 0, phase ^= 1;
                }
                for (int h = 0; h < 2 && landed; ++h) landed = wait_or_give_up(&ctl->q_free[h], (q_phase >> h) & 1, abort, status);
            }
            __syncwarp();
        } else if (warp >= kWarpMma) {
            // Each half has an issuer of its own: a product's issue blocks until the tensor cores take it, and what lies between two chains (waits,
            // commits, instruction fetches: 150 to 300 cycles each) would leave them idle; now the other half's chain runs meanwhile.
            if (rank == 0 && elect_one_in_warp()) {
                const int h = warp - kWarpMma;
                // (a negative scale negates the queries in the product: bit 13)
                const uint32_t idesc_s = idesc_bf16_f32(kHalf<kPair>, 128, false, false) | (p.sm_scale < 0.0f ? 1u << 13 : 0u);
                constexpr uint32_t idesc_o = idesc_bf16_f32(kHalf<kPair>, 128, false, true);
                const uint64_t q0 = sdesc_sw128(sbase + kOffQ + 3 * h * kBox, 16, 1024);                     // K-major: rows x dims
                const uint64_t k0 = sdesc_sw128(sbase + kOffRing, 16, 1024);                                 // K-major: keys x dims
                const uint64_t v0 = sdesc_sw128(sbase + (kPair ? kOffPairV : kOffRing), kBox / 2, 1024);     // MN-major: dims x keys
                const uint32_t s_addr = tmem + kColS + 128 * h, o_addr = tmem + kColO + 128 * h;
                int unit = 0, e = 0;                        // of the block at hand: first unit (one CTA), entry
                uint32_t phase = 0, q_phase = 0, p_phase = 0, turn_phase = h == 0 ? 1u : 0u;
                auto next_e = [](int x) { return x + 1 == kDepth<kPair> ? 0 : x + 1; };
                auto scores = [&](int at, int entry) {      // S from the keys of that block
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < 3; ++c) {
                        const uint64_t qd = q0 + static_cast<uint32_t>(c * (kBox >> 4));
                        const uint64_t kd = k0 + static_cast<uint32_t>(kPair ? entry * (kPairK >> 4) + c * (kBox >> 5) : ((at + c) & (kUnits - 1)) * (kBox >> 4));
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            if (kPair) mma_ss_cg2(s_addr, qd + 2 * ks, kd + 2 * ks, idesc_s, c > 0 || ks > 0 ? 1u : 0u);
                            else mma_ss(s_addr, qd + 2 * ks, kd + 2 * ks, idesc_s, c > 0 || ks > 0 ? 1u : 0u);
                        }
                    }
                    commit(&ctl->s_full[h]);
                };
                // The halves take turns: chains that run at the same time would both be late, and their softmax would run at the same time too.
                auto my_turn = [&]() -> bool {
                    const bool mine = wait_or_give_up(&ctl->turn[h], turn_phase, abort, status);
                    turn_phase ^= 1u;
                    return mine;
                };
                Items items = {ctl};
                bool ok = true;
                for (const Item* next = items.next(status); next != nullptr; items.done(), next = items.next(status)) {
                    const int n = max(next->count0, next->count1), count = h == 0 ? next->count0 : next->count1;
                    if (n == 0) continue;
                    if (count > 0) {                        // the first block's scores
                        ok = wait_or_give_up<kPair>(&ctl->k_full[e], phase, abort, status) && wait_or_give_up<kPair>(&ctl->q_full[h], q_phase, abort, status);
                        if (!ok) break;
                        q_phase ^= 1u;
                    }
                    ok = my_turn();
                    if (!ok) break;
                    if (count > 0) {
                        scores(unit, e);
                        if (count == 1) commit(&ctl->q_free[h]);
                    }
                    mbar_arrive(&ctl->turn[h ^ 1]);
                    commit(&ctl->k_empty[e]);
#pragma unroll 1
                    for (int i = 0; i < n; ++i) {
                        const int e1 = next_e(e);           // the next block's entry and its phase
                        const uint32_t phase1 = e1 == 0 ? phase ^ 1u : phase;
                        ok = wait_or_give_up<kPair>(&ctl->v_ready[e], phase, abort, status);
                        if (!ok) break;
                        bool keys_here = false;
                        if (i < count) {
                            // (the next keys are mostly there already: seen to while P is not)
                            keys_here = !kPair && i + 1 < count && mbar_test_wait(&ctl->k_full[e1], phase1);
                            ok = wait_or_give_up<kPair>(&ctl->p_full[h], p_phase, abort, status);
                            if (!ok) break;
                            p_phase ^= 1u;
                        }
                        ok = my_turn();
                        if (!ok) break;
                        if (i < count) {                    // O (+)= P V
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int c = 0; c < 2; ++c) {
                                const uint64_t vd = v0 + static_cast<uint32_t>(kPair ? e * (kBox >> 4) + 512 * c : ((unit + 3 + c) & (kUnits - 1)) * (kBox >> 4));
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks) {
                                    const uint32_t add = i == 0 && c == 0 && ks == 0 ? 0u : 1u;
                                    if (kPair) mma_ts_cg2(o_addr, s_addr + 32 * c + 8 * ks, vd + 128 * ks, idesc_o, add);
                                    else mma_ts(o_addr, s_addr + 32 * c + 8 * ks, vd + 128 * ks, idesc_o, add);
                                }
                            }
                            if (i + 1 == count) commit(&ctl->o_done[h]);
                        }
                        commit(&ctl->v_empty[e]);
                        unit = (unit + 5) & (kUnits - 1);
                        if (i + 1 < count) {
                            ok = keys_here || wait_or_give_up<kPair>(&ctl->k_full[e1], phase1, abort, status);
                            if (!ok) break;
                            scores(unit, e1);
                            if (i + 2 == count) commit(&ctl->q_free[h]);
                        }
                        mbar_arrive(&ctl->turn[h ^ 1]);
                        if (i + 1 < n) commit(&ctl->k_empty[e1]);
                        e = e1;
                        phase = phase1;
                    }
                    if (!ok) break;
                }
                if (kPair) mma_commit_cg2(&ctl->drain, 0x1u);
                else mma_commit(&ctl->drain);
                wait_or_give_up(&ctl->drain, 0, abort, status);
            }
            __syncwarp();
        } else if (warp == kWarpFix) {
            // The run's items, one ahead of the one that is worked on (in both CTAs of a pair alike).
            Walk<kPair> walk = find_run<kPair>(a, run, runs, lane);
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
            // Values behind a sequence's end belong to other sequences or to nobody and may be anything: zeros, as 0 x NaN is NaN. Where some
            // rows of the tile do not see all keys of a block, values that are not finite would reach them in the same way: they
            // become zeros too, and the rows that see such a key are made NaN on their way out. (The values are there long before the
            // weights, so the look at them costs little: 16 short prompts, where it is all blocks, 45.8 -> 47.6 us, long chunks 0.5%.)
            int unit = 0, e = 0, number = 0;               // number: of items with blocks
            uint32_t phase = 0;
            Item it = walk.next(p, run, lane);
            bool ok = publish(it);
            while (ok && it.valid) {
                const Item ahead = walk.next(p, run, lane);
                ok = publish(ahead);
                const int n = max(it.count0, it.count1);
                int* const bad = &ctl->bad[number & 15];
                if (n > 0) {
                    // (items that lie 8 apart are never at work together: values are at most three blocks ahead of the products)
                    if (lane == 0) ctl->bad[(number + 8) & 15] = INT32_MAX;
                    ++number;
                }
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i) {
                    const int left = it.keys - 128 * (it.from + i);
                    unit = (unit + 3) & (kUnits - 1);
                    ok = wait_warp(&ctl->v_full[e], phase, abort, status);
                    if (!ok) break;
                    if (left < 128) {
                        if (kPair) {
                            for (int x = max(left, 0) * 8 + lane; x < 128 * 8; x += 32) sts_u128(sbase + kOffPairV + e * kBox + 16 * x, make_uint4(0u, 0u, 0u, 0u));
                        } else {
                            for (int c = 0; c < 2; ++c) {
                                const uint32_t base = sbase + kOffRing + ((unit + c) & (kUnits - 1)) * kBox;
                                for (int x = max(left - 64 * c, 0) * 8 + lane; x < 64 * 8; x += 32) {
                                    sts_u128(base + 16 * x, make_uint4(0u, 0u, 0u, 0u));
                                    sts_u128(base + kBox / 2 + 16 * x, make_uint4(0u, 0u, 0u, 0u));
                                }
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (128 * (it.from + i + 1) > it.seen) {
                        int key = INT32_MAX;
                        if (kPair) {
                            key = clean_values(sbase + kOffPairV + e * kBox, 127, lane);
                        } else {
                            for (int c = 0; c < 2; ++c) {
                                const int k = clean_values(sbase + kOffRing + ((unit + c) & (kUnits - 1)) * kBox, 63, lane);
                                if (k != INT32_MAX) key = min(key, 64 * c + k);
                            }
                        }
                        if (key != INT32_MAX && lane == 0) {
                            key += 128 * (it.from + i);
                            atomicMin(bad, key);
                            if (kPair) red_min_cluster(mapa_shared(smem_addr(bad), rank ^ 1), key);
                        }
                    }
                    unit = (unit + 2) & (kUnits - 1);
                    if (lane == 0) arrive_first(&ctl->v_ready[e], false);
                    if (++e == kDepth<kPair>) e = 0, phase ^= 1;
                }
                it = ahead;
            }
        }
    } else {
        const int h = warp >> 2, w = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * w) << 16);
        const uint32_t s_addr = lanes + kColS + 128 * h, o_addr = lanes + kColO + 128 * h;
        // (0 x -inf would be NaN where a key is masked: 2^-149, which takes the largest score there is to 2^-21)
        const float mul = p.sm_scale == 0.0f ? __uint_as_float(1u) : fabsf(p.sm_scale) * kLog2e;
        int seen = 0, number = 0;      // blocks of this half, items with blocks so far
        uint32_t done = 0;             // and tiles
        Items items = {ctl};
        bool ok = true;
        for (;;) {
            const Item* const it = items.next<true>(status);
            if (it == nullptr) break;
            const int n = h == 0 ? it->count0 : it->count1;
            // keys that the row, and the half's first row, see of those from the first block on
            const int first = kHalf<kPair> * h + 128 * rank;          // row of the tile that this CTA's half begins with
            const int limit = min(it->seen + first + 32 * w + lane, it->keys) - 128 * it->from;
            const int first_limit = it->seen + first - 128 * it->from;
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
                if (lane == 0) arrive_first(&ctl->p_full[h], true);
            }
            if (n > 0) {
                ok = ok && wait_warp(&ctl->o_done[h], done++ & 1, abort, status);
                if (!ok) break;
                tc_fence_after_sync();
            }
            const int rows = it->rows - first - 32 * w;      // of this warp (32 and more: all)
            const int head = it->head, slot = it->slot;
            const bool empty = l == 0.0f;
            const float lse2 = empty ? -INFINITY : m + log2f(l);
            float f = empty ? 0.0f : 1.0f / l;
            if (slot < 0 && !empty && p.attn_sink != nullptr) f = 1.0f / (l + exp2f(__ldg(p.attn_sink + head) * kLog2e - m));
            const bool none = n == 0 || empty;
            // a value that was taken out, of a key that the row sees
            const bool spoilt = max(it->count0, it->count1) > 0 && min(it->seen + first + 32 * w + lane, it->keys) > ctl->bad[number++ & 15];
            if (spoilt) f = __uint_as_float(0x7FC00000u);
            if (slot >= 0 && rows > 0) {                   // (where a part has no keys the join does not look at its outputs)
                a.part_lse[static_cast<int64_t>(slot) * kTile<kPair> + first + 32 * w + lane] = lse2;
                float* dst = a.part_out + (static_cast<int64_t>(slot) * (kTile<kPair> / 32) + first / 32 + w) * 4096 + 8 * lane;
#pragma unroll 1
                for (int c = n > 0 ? 0 : 4; c < 4; ++c) {
                    uint32_t o[32];
                    tmem_ld32_wait(o_addr + 32 * c, o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = none ? 0u : __float_as_uint(__uint_as_float(o[e]) * f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) st_sector(dst + (4 * c + e) * 256, o + 8 * e);
                }
            } else if (rows > 0) {
                const int64_t at = static_cast<int64_t>(it->q0 + first + 32 * w) * p.heads + head;   // of lane 0's row
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
    if (kPair) cluster_sync();             // no CTA leaves while the other's products may read its shared or tensor memory
    if (warp == kWarpMma) {
        tc_fence_after_sync();
        if (kPair) tmem_dealloc_cg2(tmem, kTmemCols);
        else tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the parts of a tile that was cut: with part s's lse L_s (log2) and output O_s, w_s = 2^(L_s - max L),
// out = sum_s w_s O_s / (sum_s w_s + 2^(sink - max L)). The first part of header c lies in slot 2c + 1, the others in slots
// 2 (c + 1), 2 (c + 2), ... A lane per row and 16 dims, in the parts' order.
template <bool kPair>
__global__ void __launch_bounds__(256) ragged_join_kernel(const float* __restrict__ part_out, const float* __restrict__ part_lse,
                                                          const int4* __restrict__ headers, const float* __restrict__ sink, int heads,
                                                          __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");   // (all CTAs of this grid are resident at once: nothing of it waits for an SM)
    const int c = blockIdx.x, lane = threadIdx.x & 31, dims = threadIdx.x >> 5, r = 32 * blockIdx.y + lane;
    const int4 hd = __ldcg(headers + c);
    if (hd.w == 0 || r >= hd.y) return;
    auto slot = [&](int s) { return static_cast<int64_t>(s == 0 ? 2 * c + 1 : 2 * (c + s)); };
    auto lse_of = [&](int s) { return __ldcg(part_lse + slot(s) * kTile<kPair> + r); };
    float m = -INFINITY;
    for (int s = 0; s < hd.w; ++s) m = fmaxf(m, lse_of(s));
    if (m == -INFINITY) m = 0.0f;
    float sum = 0.0f, acc[16] = {};
#pragma unroll 2
    for (int s = 0; s < hd.w; ++s) {
        const float part = lse_of(s), w = exp2f(part - m);
        if (part == -INFINITY) continue;
        const float4* x = reinterpret_cast<const float4*>(part_out + (slot(s) * (kTile<kPair> / 32) + blockIdx.y) * 4096 + 512 * dims + 8 * lane);
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

namespace {

template <bool kPair>
cudaError_t launch_runs(KernelArgs& a, int sms, cudaStream_t stream) {
    const RaggedArgs& p = a.p;
    const int64_t rows_k = p.rows_k > 0 ? p.rows_k : 1;      // (no row is read where there is none)
    constexpr int kKeyBox = kPair ? 64 : 128;
    if (!encode_map(&a.q_map, p.q, 192, p.heads, p.rows_q, p.q_head_stride, p.q_token_stride, 1, 128) ||
        !encode_map(&a.k_map, p.kv, 256, p.heads, rows_k, p.kv_head_stride, p.kv_token_stride, 1, kKeyBox) ||
        !encode_map(&a.v_map, p.kv, 256, p.heads, rows_k, p.kv_head_stride, p.kv_token_stride, 1, 192 - kKeyBox) ||
        !encode_map(&a.pe_map, p.k_pe, 64, 1, rows_k, 64, p.pe_stride, 1, kKeyBox))
        return cudaErrorInvalidValue;
    cudaError_t err = allow_smem<ragged_attention_kernel<kPair>>(kSmem);
    if (err != cudaSuccess) return err;
    const int runs = (sms < kMaxCtas ? sms : kMaxCtas) / (kPair ? 2 : 1);
    err = launch_dependent(ragged_attention_kernel<kPair>, dim3(kPair ? 2 * runs : runs), kThreads, kSmem, kPair ? 2 : 1, stream, a);
    if (err != cudaSuccess) return err;
    return launch_dependent(ragged_join_kernel<kPair>, dim3(runs, kTile<kPair> / 32), 256, 0, 1, stream, static_cast<const float*>(a.part_out),
                            static_cast<const float*>(a.part_lse), static_cast<const int4*>(a.headers), p.attn_sink, p.heads,
                            static_cast<__nv_bfloat16*>(p.out), p.lse);
}

// A block of keys takes a tile of 256 rows on one CTA about as long as (7 to 6) a tile of 512 rows on two; a tile costs what one and three
// blocks cost besides. So pairs are for long sequences whose rows fill their tiles, by the average rows and keys of a sequence (one CTA / pairs, us):
// 4 chunks of 512 rows over 4512 keys, 64 heads 276 / 246, of 384 rows 259 / 236, of 256 rows 148 / 210; one of 700 rows over 16700 keys
// 355 / 390; 16 prompts of 512, 16 heads 51 / 55; 2 prompts of 4096, 64 heads 509 / 498; 2048 rows over 16640 keys, 64 heads 868 / 760.
// The averages are all that the host knows, as lengths lie on the device. Where sequences are of very different lengths, or the tensors larger than
// what they hold, the choice can be the slower one: that last chunk beside one token over 4000 keys, or in a batch padded with 63 empty
// sequences, goes to one CTA each (920 and 910 us in a run where it alone takes 818).
bool pairs_are_faster(const RaggedArgs& p) {
    const int64_t rows = (p.rows_q + p.batch - 1) / p.batch, keys = p.rows_k / p.batch;
    const int64_t blocks = keys > rows / 2 ? (keys - rows / 2) / 128 : 0;
    return 12 * ((rows + 511) / 512) * (blocks + 3) < 7 * ((rows + 255) / 256) * (blocks + 1);
}

}  // namespace

cudaError_t launch_ragged_attention(const RaggedArgs& p, void* workspace, int sms, cudaStream_t stream) {
    KernelArgs a;
    a.p = p;
    a.part_out = static_cast<float*>(workspace);
    a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kPartsBytes);
    a.headers = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + kPartsBytes + kLseBytes);
    return pairs_are_faster(p) ? launch_runs<true>(a, sms, stream) : launch_runs<false>(a, sms, stream);
}

}  // namespace nvfp4mla

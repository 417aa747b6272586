// head_products.cu -- the two products per head around the absorbed form of the latent attention.
//
// With c the latent of a key token, head h's key is W_uk[h] c and its value W_uv[h] c (128 x 512 each, rows 0-127 and
// 128-255 of kv_b[h]). The attention over the cache works on c itself, so a query is taken into the latent
// space first and its output back out of it:
//   absorb   q'[t, h, 0:512]   = W_uk[h]^T q[t, h, 0:128],   q'[t, h, 512:576] = R(position[t]) q[t, h, 128:192]
//   project  out[t, h, 0:128]  = W_uv[h] o[t, h, 0:512]
// R turns pairs of the RoPE dims by the caller's tables, in fp32. Sums run in fp32 in tensor memory and are rounded to bf16 once.
//
// Either is one product [tokens, K] x [K, N] per head, (K, N) = (128, 512) and (512, 128): 131 kFLOP against 1.5 and 1.3 KB
// a token and head, far below the 290 FLOP per byte at which the tensor cores would be the bound, so what counts
// is that every byte moves once. A job is a tile of 128 tokens of one head (and one piece of N, below). CTAs, one per SM, take
// equal runs of jobs, all tiles of a head one behind the other, and keep the head's weights (128 KB) in
// shared memory while the tokens' boxes of 64 dims stream through a ring; accumulators alternate between two
// halves of the tensor memory, so that loads, products and stores of neighbouring tiles overlap. Results leave through shared
// memory as boxes (32-byte stores of 32 rows at once take 130 cycles a warp).
// 4001 tokens x 128 heads: absorb 160 to 162 us, 5.0 TB/s (73% of a copy's rate; 154 us without rotation), project 112 to 116 us,
// 5.9 TB/s (87%). One token x 16 heads: 3.5 and 3.9 us on the device.
#include "head_tiles.cuh"
#include "launch.h"

namespace nvfp4mla {
namespace {

using namespace tiles;

constexpr int kStages = 4;            // ring of boxes of 128 tokens x 64 dims
constexpr int kStage = 4096;          // a warp's 32 tokens x 64 columns on the way out, two of them a warp
constexpr int kOffW = 1024;
constexpr int kWarpLoad = 4, kWarpMma = 5, kWarpRope = 6;   // warps 0-3 read the accumulators out
constexpr int kRopeWarps = 8;
constexpr int kTmemCols = 512;

template <bool kAbsorb> constexpr int kK = kAbsorb ? 128 : 512;
template <bool kAbsorb> constexpr int kN = kAbsorb ? 512 : 128;
template <bool kAbsorb> constexpr int kThreads = kAbsorb ? 32 * (kWarpRope + kRopeWarps) : 32 * kWarpRope;
template <bool kAbsorb, int kPiece> constexpr int kWBytes = kK<kAbsorb> * kPiece * 2;
template <bool kAbsorb, int kPiece> constexpr int kSmem = kOffW + kWBytes<kAbsorb, kPiece> + kStages * kBox + 8 * kStage + 1024;
static_assert(kSmem<true, 512> <= 232448 && kSmem<false, 128> <= 232448, "shared memory");

struct Ctl {
    uint64_t full[kStages], empty[kStages];
    uint64_t w_full, w_empty;          // the weights of a head (piece) landed; no product reads them any more
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base, abort;
};

struct KernelArgs {
    CUtensorMap a_map;                 // [tokens, heads, 192 or 512], box 128 x 1 x 64
    CUtensorMap w_map;                 // kv_b [heads, 256, 512], box 1 x rows x 64
    CUtensorMap out_map;               // [tokens, heads, 576 or 128], box 32 x 1 x 64
    HeadProductArgs p;
    int64_t jobs;
    int tiles, pieces;
};

// Four pairs of a token's RoPE dims. half: values 4j .. 4j + 3 and 32 + 4j .. in x; else values 8j .. 8j + 7.
__device__ __forceinline__ void rotate4(uint32_t (&x)[4], bool half, float4 c, float4 s) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&x[e]);
        v[2 * e] = __low2float(b);
        v[2 * e + 1] = __high2float(b);
    }
    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int f = 0; f < 4; ++f) {
        const float a = half ? v[f] : v[2 * f], b = half ? v[4 + f] : v[2 * f + 1];
        const float u = a * cs[f] - b * sn[f], w = b * cs[f] + a * sn[f];
        if (half) {
            v[f] = u;
            v[4 + f] = w;
        } else {
            v[2 * f] = u;
            v[2 * f + 1] = w;
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
}

// Positions of a lane's tokens of a tile (16 tokens a warp, four at a time, eight lanes a token); -1: none to rotate by.
__device__ __forceinline__ void rope_positions(const HeadProductArgs& p, int64_t t0, int lane, int64_t (&pos)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t t = t0 + 4 * e + (lane >> 3);
        pos[e] = p.positions != nullptr && t < p.tokens ? __ldg(p.positions + t) : -1;
    }
}

// The RoPE dims of a tile's tokens: all of a lane's loads are in flight at once (in four rounds of loads a tile,
// positions ahead of tables, these warps bound the kernel: 262 against 161 us at 4001 tokens x 128 heads, 154 without rotation). Fourteen
// warps leave 128 registers a thread, of which these loads want a few more: 60 bytes are spilled.
template <bool kHalf>
__device__ __forceinline__ void rope_tile(const HeadProductArgs& p, int64_t t0, int head, int lane, const int64_t (&pos)[4]) {
    const int j = lane & 7;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.in) + head * p.in_head_stride + 128;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + 512;
    uint32_t x[4][4];
    float4 c[4], s[4];
    bool use[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t t = t0 + 4 * e + (lane >> 3);
        use[e] = t < p.tokens;
        if (!use[e]) continue;
        const __nv_bfloat16* src = q + t * p.in_token_stride;
        if (kHalf) {
            const uint2 lo = __ldg(reinterpret_cast<const uint2*>(src + 4 * j)), hi = __ldg(reinterpret_cast<const uint2*>(src + 32 + 4 * j));
            x[e][0] = lo.x, x[e][1] = lo.y, x[e][2] = hi.x, x[e][3] = hi.y;
        } else {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(src + 8 * j));
            x[e][0] = w.x, x[e][1] = w.y, x[e][2] = w.z, x[e][3] = w.w;
        }
        if (p.positions != nullptr) {
            if (pos[e] < 0 || pos[e] >= p.num_positions) {
                use[e] = false;
                if (p.status != nullptr && j == 0) atomicOr(p.status, 0x10u);
                continue;
            }
            c[e] = __ldg(reinterpret_cast<const float4*>(p.cos_table + pos[e] * 32 + 4 * j));
            s[e] = __ldg(reinterpret_cast<const float4*>(p.sin_table + pos[e] * 32 + 4 * j));
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (!use[e]) continue;
        const int64_t t = t0 + 4 * e + (lane >> 3);
        if (p.positions != nullptr) rotate4(x[e], kHalf, c[e], s[e]);
        __nv_bfloat16* dst = out + (t * p.heads + head) * 576;
        if (kHalf) {
            *reinterpret_cast<uint2*>(dst + 4 * j) = make_uint2(x[e][0], x[e][1]);
            *reinterpret_cast<uint2*>(dst + 32 + 4 * j) = make_uint2(x[e][2], x[e][3]);
        } else {
            *reinterpret_cast<uint4*>(dst + 8 * j) = make_uint4(x[e][0], x[e][1], x[e][2], x[e][3]);
        }
    }
}

template <bool kAbsorb, int kPiece>
__global__ void __launch_bounds__(kThreads<kAbsorb>, 1) head_product_kernel(const __grid_constant__ KernelArgs a) {
    constexpr int kChunks = kK<kAbsorb> / 64;
    constexpr int kSub = kPiece < 256 ? kPiece : 256;       // columns of an accumulator
    constexpr int kSubs = kPiece / kSub;
    constexpr int kWBox = kAbsorb ? kBox : kPiece * 128;     // bytes of a weight box: 128 k x 64 n, or kPiece n x 64 k
    constexpr int kWBoxes = kWBytes<kAbsorb, kPiece> / kWBox;
    constexpr int kOffRing = kOffW + kWBytes<kAbsorb, kPiece>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    Ctl* ctl = reinterpret_cast<Ctl*>(smem);
    const uint32_t sbase = smem_addr(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kWarpLoad && lane == 0) {
        prefetch_map(&a.a_map);
        prefetch_map(&a.w_map);
        prefetch_map(&a.out_map);
        for (int i = 0; i < kStages; ++i) mbar_init(&ctl->full[i], 1), mbar_init(&ctl->empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&ctl->acc_full[i], 1), mbar_init(&ctl->acc_empty[i], 4);
        mbar_init(&ctl->w_full, 1), mbar_init(&ctl->w_empty, 1), mbar_init(&ctl->drain, 1);
        ctl->abort = 0u;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(&ctl->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int64_t u0 = a.jobs * blockIdx.x / gridDim.x, u1 = a.jobs * (blockIdx.x + 1) / gridDim.x;
    int hp = static_cast<int>(u0 / a.tiles), tile = static_cast<int>(u0 - static_cast<int64_t>(hp) * a.tiles);
    const int n_jobs = static_cast<int>(u1 - u0);
    uint32_t* abort = &ctl->abort;
    uint32_t* status = a.p.status;

    if (warp == kWarpLoad) {
        if (lane == 0) {
            int cur = -1, stage = 0, loads = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int i = 0; i < n_jobs && ok; ++i) {
                const int head = hp / a.pieces, n0 = (hp - head * a.pieces) * kPiece;
                if (hp != cur) {
                    if (cur >= 0) ok = wait_or_give_up(&ctl->w_empty, (loads - 1) & 1, abort, status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&ctl->w_full, kWBytes<kAbsorb, kPiece>);
                    for (int b = 0; b < kWBoxes; ++b)
                        tma_load_3d(sbase + kOffW + b * kWBox, &a.w_map, kAbsorb ? n0 + 64 * b : 64 * b, kAbsorb ? 0 : 128 + n0, head, &ctl->w_full);
                    cur = hp;
                    ++loads;
                }
                for (int c = 0; c < kChunks && ok; ++c) {
                    ok = wait_or_give_up(&ctl->empty[stage], phase, abort, status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&ctl->full[stage], kBox);
                    tma_load_3d(sbase + kOffRing + stage * kBox, &a.a_map, 64 * c, head, tile * 128, &ctl->full[stage]);
                    if (++stage == kStages) stage = 0, phase ^= 1;
                }
                if (++tile == a.tiles) tile = 0, ++hp;
            }
        }
    } else if (warp == kWarpMma) {
        if (elect_one_in_warp()) {
            constexpr uint32_t idesc = idesc_bf16_f32(128, kSub, false, kAbsorb);
            const uint64_t a0 = sdesc_sw128(sbase + kOffRing, 16, 1024);                                        // K-major: tokens x dims
            const uint64_t w0 = sdesc_sw128(sbase + kOffW, kAbsorb ? kBox : 16, 1024);   // absorb MN-major: n x k, else K-major
            int cur = -1, stage = 0, loads = 0, acc = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int i = 0; i < n_jobs && ok; ++i) {
                if (hp != cur) {
                    ok = wait_or_give_up(&ctl->w_full, loads & 1, abort, status);
                    cur = hp;
                    ++loads;
                }
#pragma unroll 1
                for (int sub = 0; sub < kSubs && ok; ++sub, ++acc) {
                    const int buf = acc & 1;
                    ok = wait_or_give_up(&ctl->acc_empty[buf], ((acc >> 1) & 1) ^ 1, abort, status);
                    int st = stage;
                    uint32_t ph = phase;
#pragma unroll 1
                    for (int c = 0; c < kChunks && ok; ++c) {
                        if (sub == 0) ok = wait_or_give_up(&ctl->full[st], ph, abort, status);
                        if (!ok) break;
                        tc_fence_after_sync();
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            const uint64_t ad = a0 + static_cast<uint64_t>((st * kBox + ks * 32) >> 4);
                            const int woff = kAbsorb ? sub * (kSub / 64) * kBox + (4 * c + ks) * 2048 : c * kWBox + ks * 32;
                            mma_ss(tmem + 256 * buf, ad, w0 + static_cast<uint64_t>(woff >> 4), idesc, c > 0 || ks > 0 ? 1u : 0u);
                        }
                        if (sub == kSubs - 1) mma_commit(&ctl->empty[st]);
                        if (++st == kStages) st = 0, ph ^= 1;
                    }
                    if (sub == kSubs - 1) stage = st, phase = ph;
                    if (ok) mma_commit(&ctl->acc_full[buf]);
                }
                if (++tile == a.tiles) {
                    tile = 0, ++hp;
                    if (ok && i + 1 < n_jobs) mma_commit(&ctl->w_empty);
                }
            }
            mma_commit(&ctl->drain);
            wait_or_give_up(&ctl->drain, 0, abort, status);
        }
        __syncwarp();
    } else if (warp < 4) {
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * warp) << 16);
        const uint32_t stage = sbase + kOffRing + kStages * kBox + 2 * warp * kStage;
        int acc = 0, boxes = 0;
        bool ok = true;
        for (int i = 0; i < n_jobs && ok; ++i) {
            const int head = hp / a.pieces, n0 = (hp - head * a.pieces) * kPiece;
            const int t0 = tile * 128 + 32 * warp;
#pragma unroll 1
            for (int sub = 0; sub < kSubs && ok; ++sub, ++acc) {
                const int buf = acc & 1;
                ok = wait_warp(&ctl->acc_full[buf], (acc >> 1) & 1, abort, status);
                if (!ok) break;
                tc_fence_after_sync();
                if (t0 < a.p.tokens) {   // (the same for the whole warp)
#pragma unroll 1
                    for (int c = 0; c < kSub / 64; ++c, ++boxes) {
                        const uint32_t box = stage + (boxes & 1) * kStage;
                        if (lane == 0) tma_store_wait_read<1>();     // the box before the last one has left
                        __syncwarp();
                        stage_box(lanes + 256 * buf + 64 * c, box, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) tma_store_3d(&a.out_map, n0 + kSub * sub + 64 * c, head, t0, box);
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->acc_empty[buf]);
            }
            if (++tile == a.tiles) tile = 0, ++hp;
        }
        if (lane == 0) tma_store_wait();
        __syncwarp();
    } else if constexpr (kAbsorb) {
        const int mine = 16 * (warp - kWarpRope);
        int64_t pos[4], next[4];
        rope_positions(a.p, static_cast<int64_t>(tile) * 128 + mine, lane, pos);
        for (int i = 0; i < n_jobs; ++i) {
            const int head = hp / a.pieces;
            const int64_t t0 = static_cast<int64_t>(tile) * 128 + mine;
            const bool takes = hp == head * a.pieces;   // one of the head's pieces takes the RoPE dims along
            if (++tile == a.tiles) tile = 0, ++hp;
            rope_positions(a.p, static_cast<int64_t>(tile) * 128 + mine, lane, next);   // (a job ahead)
            if (takes) {
                if (a.p.rotate_half)
                    rope_tile<true>(a.p, t0, head, lane, pos);
                else
                    rope_tile<false>(a.p, t0, head, lane, pos);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) pos[e] = next[e];
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

template <bool kAbsorb, int kPiece>
cudaError_t launch_piece(KernelArgs& a, int sms, cudaStream_t stream) {
    const HeadProductArgs& p = a.p;
    if (!encode_map(&a.a_map, p.in, kAbsorb ? 192 : 512, p.heads, p.tokens, p.in_head_stride, p.in_token_stride, 1, 128) ||
        !encode_map(&a.w_map, p.kv_b, 512, 256, p.heads, p.w_row_stride, p.w_head_stride, kAbsorb ? 128 : kPiece, 1) ||
        !encode_map(&a.out_map, p.out, kAbsorb ? 576 : 128, p.heads, p.tokens, kAbsorb ? 576 : 128, static_cast<int64_t>(p.heads) * (kAbsorb ? 576 : 128), 1, 32))
        return cudaErrorInvalidValue;
    constexpr int kBytes = kSmem<kAbsorb, kPiece>;
    const cudaError_t err = allow_smem<head_product_kernel<kAbsorb, kPiece>>(kBytes);
    if (err != cudaSuccess) return err;
    a.tiles = static_cast<int>((p.tokens + 127) / 128);
    a.pieces = kN<kAbsorb> / kPiece;
    a.jobs = static_cast<int64_t>(a.tiles) * p.heads * a.pieces;
    const unsigned grid = static_cast<unsigned>(a.jobs < sms ? a.jobs : sms);
    return launch_dependent(head_product_kernel<kAbsorb, kPiece>, dim3(grid), kThreads<kAbsorb>, kBytes, 1, stream, a);
}

}  // namespace

cudaError_t launch_head_product(const HeadProductArgs& p, bool absorb, int sms, cudaStream_t stream) {
    KernelArgs a;
    a.p = p;
    // With few jobs the weights are cut into pieces of N, so that more SMs load them (cut / whole, device time of one token: absorb 16 heads 3.5 / 5.5 us,
    // 64 heads in two 4.7 / 5.9, 128 heads in two 7.3 / 6.9; project 16 heads in two 3.9 / 4.6, in four 3.9 to 4.3, 64 heads in two 4.5 / 4.8,
    // 128 heads in two 7.8 / 6.2).
    const int64_t jobs = ((p.tokens + 127) / 128) * p.heads;
    const int cut = 4 * jobs <= sms ? 4 : 2 * jobs <= sms ? 2 : 1;
    if (absorb) return cut == 4 ? launch_piece<true, 128>(a, sms, stream) : cut == 2 ? launch_piece<true, 256>(a, sms, stream) : launch_piece<true, 512>(a, sms, stream);
    return cut > 1 ? launch_piece<false, 64>(a, sms, stream) : launch_piece<false, 128>(a, sms, stream);
}

}  // namespace nvfp4mla

// dequant.cuh -- record-field conversions and shared-memory addressing used by the decode kernels
// that dequantize NVFP4 records into 16-bit MMA operand tiles.
//
// An NVFP4 value is an e2m1 code times the e4m3 scale of its 16-value block; the product has at
// most five significant bits and lies in [2^-10, 2688] (or is zero), so it is exact in f16 and in
// bf16 and every conversion below is exact.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace nvfp4mla {

// Byte offset of 16-byte chunk `chunk` (0..7) of row `row` in a 128B-swizzled tile of 128-byte
// rows (the canonical SWIZZLE_128B operand layout: 8-row atoms of 1024 bytes).
__device__ __forceinline__ uint32_t swz(int row, int chunk) {
    return static_cast<uint32_t>((row >> 3) * 1024 + (row & 7) * 128 + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ void named_bar_sync(uint32_t id, uint32_t threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// e4m3 scale byte -> (s, s) as f16x2 (exact).
__device__ __forceinline__ __half2 scale_half2(uint32_t sbyte) {
    uint32_t h;
    const uint16_t in = static_cast<uint16_t>(sbyte | (sbyte << 8));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(in));
    return *reinterpret_cast<__half2*>(&h);
}

// Eight e2m1 codes (one word, low nibble first) times a scale -> four f16x2 words (exact).
__device__ __forceinline__ uint4 dq8(uint32_t w, __half2 s2) {
    uint32_t h[4];
    asm("{\n"
        "  .reg .b8 a, b, c, d;\n"
        "  mov.b32 {a, b, c, d}, %4;\n"
        "  cvt.rn.f16x2.e2m1x2 %0, a;\n"
        "  cvt.rn.f16x2.e2m1x2 %1, b;\n"
        "  cvt.rn.f16x2.e2m1x2 %2, c;\n"
        "  cvt.rn.f16x2.e2m1x2 %3, d;\n"
        "}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h[k]), s2);
        h[k] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// Four e4m3 codes -> two f16x2 words (exact).
__device__ __forceinline__ uint2 e4m3x4_to_f16(uint32_t w) {
    uint32_t a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"(static_cast<uint16_t>(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(static_cast<uint16_t>(w >> 16)));
    return make_uint2(a, b);
}

// Byte q of each word of w, low word first.
__device__ __forceinline__ uint32_t gather_byte4(const uint4& w, int q) {
    const uint32_t sel = static_cast<uint32_t>(q) | (static_cast<uint32_t>(q + 4) << 4);
    return __byte_perm(__byte_perm(w.x, w.y, sel), __byte_perm(w.z, w.w, sel), 0x5410);
}

// Read-only global loads that do not allocate in L1 (every record byte is used once per CTA).
__device__ __forceinline__ uint4 ldg_stream16(const void* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// One key's share of a converter thread q (0..3): record bytes 64c + 16q .. + 15 (c = 0..3), the codes
// of 16-dim blocks 8c + 2q and 8c + 2q + 1, and the scale bytes of those blocks.
template <int R, bool kBlkOrder>
struct KeyRaw {
    // 352-byte records with the permuted placement (block s at 320 + 8 (s & 3) + (s >> 2)): the eight
    // scale bytes of the thread's blocks lie in one 16-byte half of the field; otherwise all 32 bytes
    static constexpr bool kPermuted = R == 352 && !kBlkOrder;
    uint4 codes[4];
    uint4 sc[kPermuted ? 1 : 2];

    __device__ __forceinline__ void load_codes(const uint8_t* rec, int q, int c) { codes[c] = ldg_stream16(rec + 64 * c + 16 * q); }
    __device__ __forceinline__ void load_scales(const uint8_t* rec, int q) {
        if constexpr (kPermuted) {
            sc[0] = ldg_stream16(rec + 320 + 16 * (q & 1));
        } else {
            constexpr int sb = R == 352 ? 320 : 256;
            sc[0] = ldg_stream16(rec + sb);
            sc[1] = ldg_stream16(rec + sb + 16);
        }
    }
    __device__ __forceinline__ void load(const uint8_t* rec, int q) {
#pragma unroll
        for (int c = 0; c < 4; ++c) load_codes(rec, q, c);
        load_scales(rec, q);
    }
    // the scale pairs of blocks c = 0..3, two per word (c even: low half)
    __device__ __forceinline__ void scale_pairs(int q, uint32_t (&sp)[2]) const {
        sp[0] = (scale_pair(0, q) & 0xFFFFu) | (scale_pair(1, q) << 16);
        sp[1] = (scale_pair(2, q) & 0xFFFFu) | (scale_pair(3, q) << 16);
    }
    // byte 0: the scale of block 8c + 2q, byte 1: of block 8c + 2q + 1
    __device__ __forceinline__ uint32_t scale_pair(int c, int q) const {
        if constexpr (kPermuted) {
            // block 8c + 2q at byte 16 (q & 1) + 2c + (q >> 1), the next block eight bytes further
            const uint32_t wa = c < 2 ? sc[0].x : sc[0].y, wb = c < 2 ? sc[0].z : sc[0].w;
            const uint32_t bi = static_cast<uint32_t>(2 * c + (q >> 1)) & 3u;
            return __byte_perm(wa, wb, bi | ((bi + 4u) << 4));
        } else {
            // block s at byte s: bytes 2q, 2q + 1 of word 2c + (q >> 1)
            const uint32_t w[8] = {sc[0].x, sc[0].y, sc[0].z, sc[0].w, sc[1].x, sc[1].y, sc[1].z, sc[1].w};
            const uint32_t wv = (q >> 1) != 0 ? w[2 * c + 1] : w[2 * c];
            const uint32_t lo = 2u * static_cast<uint32_t>(q & 1);
            return __byte_perm(wv, 0u, lo | ((lo + 1u) << 4));
        }
    }
};

}  // namespace nvfp4mla

// paged_decode.cu -- host side of the paged attention (paged_decode_few.cu, paged_decode_pair.cu) and the kernel that joins the
// parts of jobs whose tiles lie in the runs of several CTAs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"

namespace nvfp4mla {
namespace {

constexpr int kJoinRows = 4;      // rows of a join CTA, four warps each
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Entry c of hdr names a job that was cut: first output row, rows (0: there is none), parts n, slot f of the
// first part; the others lie in slots next(c), next(c) + step, ... With part lse L_s (log2) and f16 output
// O_s (divided by its own sum, times kPartScale): w_s = 2^(L_s - m), out = sum_s w_s O_s / (kPartScale (sum_s w_s + 2^(sink - m))),
// lse = (m + log2 sum_s w_s) ln 2, in fp32. A warp per row and 128 dims: its lanes weigh the parts (one each, in
// turns of 32), then the warp adds the parts up in their order, eight loads in flight. A NaN L_s makes the
// row NaN; a row without any key gets out = 0, lse = -inf.
__global__ void __launch_bounds__(128 * kJoinRows)
paged_join_kernel(const uint16_t* __restrict__ part_out, const float* __restrict__ part_lse, const int4* __restrict__ hdr,
                  const float* __restrict__ sink, int h_q, int row_tile, int step, __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 h = __ldcg(hdr + blockIdx.x);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * kJoinRows + (warp >> 2), sub = warp & 3;
    if (r >= h.y) return;
    const int parts = h.z;
    const int64_t row = static_cast<int64_t>(h.x) + r;
    const float sk = sink != nullptr ? __ldg(sink + row % h_q) * kLog2e : -INFINITY;
    auto slot = [&](int s) { return static_cast<int64_t>(s == 0 ? h.w : h.w + 1 + (s - 1) * step) * row_tile + r; };
    auto lse_of = [&](int s) { return s < parts ? __ldcg(part_lse + slot(s)) : -INFINITY; };
    const float first = lse_of(lane);
    float m = first, tot;
    for (int s = 32 + lane; s < parts; s += 32) m = fmaxf(m, lse_of(s));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) m = 0.0f;
    tot = exp2f(first - m);
    for (int s = 32 + lane; s < parts; s += 32) tot += exp2f(lse_of(s) - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    const int d = 128 * sub + 4 * lane;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int base = 0; base < parts; base += 32) {
        const float weight = exp2f((base == 0 ? first : lse_of(base + lane)) - m);
        const int n = min(32, parts - base);
        for (int i = 0; i < n; i += 8) {
            uint2 x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = i + e < n ? __ldcg(reinterpret_cast<const uint2*>(part_out + slot(base + i + e) * 512 + d)) : make_uint2(0u, 0u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float w = __shfl_sync(0xffffffffu, weight, (i + e) & 31);
                if (i + e >= n) continue;
                const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&x[e].x)), f1 = __half22float2(*reinterpret_cast<const __half2*>(&x[e].y));
                acc[0] = fmaf(w, f0.x, acc[0]);
                acc[1] = fmaf(w, f0.y, acc[1]);
                acc[2] = fmaf(w, f1.x, acc[2]);
                acc[3] = fmaf(w, f1.y, acc[3]);
            }
        }
    }
    const float f = tot == 0.0f ? 0.0f : 1.0f / (paged::kPartScale * (tot + exp2f(sk - m)));
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = f != 0.0f ? acc[e] * f : 0.0f;
    __nv_bfloat162 o[2] = {__floats2bfloat162_rn(acc[0], acc[1]), __floats2bfloat162_rn(acc[2], acc[3])};
    *reinterpret_cast<uint2*>(out + row * 512 + d) = *reinterpret_cast<const uint2*>(o);
    if (sub == 0 && lane == 0) lse[row] = tot == 0.0f ? -INFINITY : (m + log2f(tot)) * kLn2;
}

}  // namespace

// Up to 16 rows one CTA per SM (paged_decode_few.cu), above that CTA pairs (paged_decode_pair.cu).
// One CTA / pairs at 16 rows: 64 sequences of 1024 to 32768 tokens 166 / 276 us, 8 of up to 8192 tokens 30 / 32 us. The one-CTA
// kernel holds 16 rows; 17 and 32 rows on pairs take 276 and 277 us, 33 us (a pair's 128 rows are filled up).
int paged_row_tile(int64_t rows_per_seq) { return rows_per_seq <= 16 ? 16 : 128; }

namespace {

// f16 parts [parts, row tile, 512], their fp32 log-sum-exps, one int4 per job that may be cut, and for CTA pairs the
// segments. One CTA each: two slots per run. CTA pairs: the segments are at most (jobs + 2 pairs), so there are
// at most 2 pairs cuts, 2 pairs jobs that are cut and 4 pairs parts.
struct PagedWorkspace {
    size_t parts, headers, segments;
    size_t at_lse, at_hdr, at_segments, bytes;
    PagedWorkspace(int64_t batch, int64_t rows_per_seq) {
        const int n = paged_row_tile(rows_per_seq);
        parts = 2 * kPagedMaxSms;
        headers = kPagedMaxSms;
        segments = n < 128 ? 0 : static_cast<size_t>(batch * ((rows_per_seq + 127) / 128) + kPagedMaxSms);
        at_lse = parts * n * 512 * sizeof(uint16_t);
        at_hdr = at_lse + parts * n * sizeof(float);
        at_segments = at_hdr + headers * 4 * sizeof(int32_t);
        bytes = at_segments + segments * 12 * sizeof(int32_t);
    }
};

}  // namespace

size_t paged_workspace_bytes(int64_t batch, int64_t rows_per_seq) { return PagedWorkspace(batch, rows_per_seq).bytes; }

cudaError_t launch_paged_decode(PagedDecodeArgs d, void* workspace, int sms, cudaStream_t stream) {
    const int n = paged_row_tile(d.jobs.rows_per_seq);
    const PagedWorkspace w(d.jobs.batch, d.jobs.rows_per_seq);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (sms > kPagedMaxSms) sms = kPagedMaxSms;
    d.runs = sms;
    d.part_out = reinterpret_cast<uint16_t*>(ws);
    d.part_lse = reinterpret_cast<float*>(ws + w.at_lse);
    d.hdr = reinterpret_cast<int32_t*>(ws + w.at_hdr);
    int headers = sms;
    cudaError_t err;
    if (n == 128) {
        d.pairs = paged_pairs(sms);
        d.segments = ws + w.at_segments;
        const int64_t jobs = static_cast<int64_t>(d.jobs.batch) * ((d.jobs.rows_per_seq + 127) / 128);
        const int64_t most = paged_max_segments(jobs, d.pairs);
        headers = static_cast<int>(jobs < 2 * d.pairs ? jobs : 2 * d.pairs);
        err = launch_paged_decode_pair(d, static_cast<int>(most), headers, stream);
    } else {
        err = launch_paged_decode_few(d, stream);
    }
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(headers), static_cast<unsigned>(n / kJoinRows));
    cfg.blockDim = dim3(128 * kJoinRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, paged_join_kernel, static_cast<const uint16_t*>(d.part_out), static_cast<const float*>(d.part_lse),
                             reinterpret_cast<const int4*>(d.hdr), d.attn_sink, d.jobs.h_q, n, n == 128 ? 1 : 2,
                             static_cast<__nv_bfloat16*>(d.out), d.lse);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace nvfp4mla

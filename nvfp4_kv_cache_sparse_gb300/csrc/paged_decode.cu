// paged_decode.cu -- host side of the paged attention (paged_decode.cuh) and the kernel that joins the
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
// O_s (divided by its own sum): w_s = 2^(L_s - m), out = sum_s w_s O_s / (sum_s w_s + 2^(sink - m)),
// lse = (m + log2 sum_s w_s) ln 2. Four warps take the parts of a row in turn and add up their fp32 sums
// through shared memory, in warp order. A NaN L_s makes the row NaN; a row without any key gets out = 0,
// lse = -inf.
__global__ void __launch_bounds__(128 * kJoinRows)
paged_join_kernel(const uint16_t* __restrict__ part_out, const float* __restrict__ part_lse, const int4* __restrict__ hdr,
                  const float* __restrict__ sink, int h_q, int row_tile, int step, __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
    __shared__ float acc_s[kJoinRows][4][512];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 h = hdr[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r0 = blockIdx.y * kJoinRows;
    if (r0 >= h.y) return;
    const int r = r0 + (warp >> 2), sub = warp & 3;
    const int parts = h.z;
    auto slot = [&](int s) { return static_cast<int64_t>(s == 0 ? h.w : h.w + 1 + (s - 1) * step) * row_tile + r; };
    float m = -INFINITY, tot = 0.0f;
    if (r < h.y) {
        for (int s = lane; s < parts; s += 32) m = fmaxf(m, part_lse[slot(s)]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (m == -INFINITY) m = 0.0f;
        for (int s = lane; s < parts; s += 32) tot += exp2f(part_lse[slot(s)] - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
        float acc[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
#pragma unroll 2
        for (int s = sub; s < parts; s += 4) {
            const float w = exp2f(part_lse[slot(s)] - m);
            const uint4* p = reinterpret_cast<const uint4*>(part_out + slot(s) * 512);
            const uint4 x[2] = {p[lane], p[32 + lane]};   // dims 8 lane.. and 256 + 8 lane..
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[e]));
                    acc[8 * k + 2 * e] = fmaf(w, f.x, acc[8 * k + 2 * e]);
                    acc[8 * k + 2 * e + 1] = fmaf(w, f.y, acc[8 * k + 2 * e + 1]);
                }
            }
        }
        float* dst = acc_s[warp >> 2][sub];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                *reinterpret_cast<float4*>(dst + 256 * k + 8 * lane + e) =
                    make_float4(acc[8 * k + e], acc[8 * k + e + 1], acc[8 * k + e + 2], acc[8 * k + e + 3]);
    }
    __syncthreads();
    if (r >= h.y) return;
    const float den = tot + (sink != nullptr ? exp2f(sink[(h.x + r) % h_q] * kLog2e - m) : 0.0f);
    const float f = tot == 0.0f ? 0.0f : 1.0f / den;
    const int d = 128 * sub + 4 * lane;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float x = (acc_s[warp >> 2][0][d + e] + acc_s[warp >> 2][1][d + e]) + (acc_s[warp >> 2][2][d + e] + acc_s[warp >> 2][3][d + e]);
        v[e] = f != 0.0f ? x * f : 0.0f;
    }
    const int64_t row = static_cast<int64_t>(h.x) + r;
    __nv_bfloat162 o[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
    *reinterpret_cast<uint2*>(out + row * 512 + d) = *reinterpret_cast<const uint2*>(o);
    if (sub == 0 && lane == 0) lse[row] = tot == 0.0f ? -INFINITY : (m + log2f(tot)) * kLn2;
}

}  // namespace

int paged_row_tile(int64_t rows_per_seq) { return rows_per_seq <= 16 ? 16 : rows_per_seq <= 32 ? 32 : 128; }

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
        err = n == 16 ? launch_paged_decode_n16(d, stream) : launch_paged_decode_n32(d, stream);
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

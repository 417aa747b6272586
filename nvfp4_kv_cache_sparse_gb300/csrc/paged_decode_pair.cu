// paged_decode_pair.cu -- host side of attention over whole sequences for jobs of up to 128 query rows on a
// CTA pair (decode_pair.cuh with kPaged).
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "decode_pair.cuh"
#include "launch.h"

namespace nvfp4mla {
namespace {

using pairdec::Segment;
constexpr int kPlanThreads = 256, kPlanWarps = kPlanThreads / 32;
constexpr int kPlanClasses = 8;
constexpr int kPlanEmpty = 31;   // CTAs of the plan that write the rows without a key

// Segments for n jobs that have a key: one per pair if that leaves each job four or more, else a whole wave of
// pairs more than the jobs fill. (For 32 sequences x 2 tokens x 128 heads, lengths 1000 to 8192, on 76 pairs: a
// model of the waves gives 1.17 of the even share, against 1.68 with one wave, 1.25 and 1.33 with 3 and 4.) Both sides
// measured, 128 rows a job, this rule / as few waves as the jobs fill: lengths that differ, that case 116 / 142 us, 2 chunks of
// 256 tokens x 64 heads 919 / 958 us; equal lengths, where the wave more only adds its segments' start and end, 32 jobs
// of 1000 tokens 43 / 33 us, 48 of 1000 51 / 36, 64 of 2000 75 / 53, 32 of 4000 67 / 57, 64 of 8000 171 / 151. Batches of equal
// lengths would be better off with a rule that counts a segment's own 11 us.
__host__ __device__ __forceinline__ int64_t waves(int64_t jobs, int64_t pairs) {
    return 4 * jobs <= pairs ? 1 : (jobs + pairs - 1) / pairs + 1;
}

// Cuts the jobs into segments for the pairs. With m = waves(jobs), T is the smallest number of tiles such that
// jobs cut evenly into ceil(tiles / T) segments make at most m * pairs; the segments are then put in the order
// of eight classes of length, the longest first, so that short ones fill the gaps at the end. (In the jobs'
// order the model gives 1.3 instead of 1.17.) One CTA: sums over the jobs, each thread a contiguous piece of
// them. The other CTAs write the rows of jobs without a key.
__global__ void __launch_bounds__(kPlanThreads, 1)
paged_plan_kernel(const paged::Jobs a, int pairs, int max_segments, int headers, Segment* __restrict__ segments,
                  int4* __restrict__ hdr, void* out, float* lse, uint32_t* status) {
    constexpr int kRows = 128, kKeys = pairdec::kTile;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");   // (the pairs wait for the whole grid all the same)
    if (blockIdx.x > 0) {
        paged::write_empty_jobs<kRows, kKeys, kPlanThreads>(a, static_cast<int>(blockIdx.x) - 1, kPlanEmpty, out, lse);
        return;
    }
    paged::check_lengths(a, static_cast<int>(threadIdx.x), kPlanThreads, status);
    __shared__ int64_t totals[kPlanWarps], cut_totals[kPlanWarps];
    __shared__ int32_t jobs_with_keys[kPlanWarps], counts[2][kPlanWarps], classes[kPlanClasses][kPlanWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int jobs = a.batch * a.row_tiles;
    const int per = (jobs + kPlanThreads - 1) / kPlanThreads;
    const int ja = min(jobs, static_cast<int>(threadIdx.x) * per), jb = min(jobs, ja + per);
    auto warp_scan = [&](auto v) {   // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const auto u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        return v;
    };
    // tiles of the thread's first job stay in a register (most calls have no more jobs than threads)
    const int first_tiles = ja < jb ? paged::job_info<kRows, kKeys>(a, ja).tiles : 0;
    auto tiles_of = [&](int j) { return j == ja ? first_tiles : paged::job_info<kRows, kKeys>(a, j).tiles; };
    int64_t mine = 0, total = 0;
    int mine_n = 0, n = 0;
    for (int j = ja; j < jb; ++j) {
        const int nt = tiles_of(j);
        mine += nt;
        mine_n += nt > 0 ? 1 : 0;
    }
    mine = warp_scan(mine);
    mine_n = __reduce_add_sync(0xffffffffu, mine_n);
    if (lane == 31) {
        totals[warp] = mine;
        jobs_with_keys[warp] = mine_n;
    }
    __syncthreads();
    for (int w = 0; w < kPlanWarps; ++w) {
        total += totals[w];
        n += jobs_with_keys[w];
    }
    const int64_t limit = n > 0 ? waves(n, pairs) * pairs : 0;
    // total / limit <= T; and sum ceil(t / T) < total / T + n, so T = ceil(total / (limit - n)) is enough if that is
    // positive (limit >= n always; with equality one segment per job, T the longest, is). The sums below are under
    // limit + n, which 31 bits hold.
    int64_t lo = 1, hi = 1;
    if (n > 0) {
        lo = max(int64_t(1), (total + limit - 1) / limit);
        hi = limit > n ? (total + limit - n - 1) / (limit - n) : total;
        hi = max(lo, hi);
    }
    for (int turn = 0; lo < hi; turn ^= 1) {
        const int64_t mid = (lo + hi) >> 1;
        const int m32 = static_cast<int>(min(mid, static_cast<int64_t>(INT32_MAX)));
        int c = 0, all = 0;
        for (int j = ja; j < jb; ++j) {
            const int nt = tiles_of(j);
            c += nt / m32 + (nt % m32 != 0 ? 1 : 0);
        }
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) counts[turn][warp] = c;
        __syncthreads();
        for (int w = 0; w < kPlanWarps; ++w) all += counts[turn][w];
        if (all <= limit)
            hi = mid;
        else
            lo = mid + 1;
    }
    const int T = static_cast<int>(min(lo, static_cast<int64_t>(INT32_MAX)));
    auto pieces_of = [&](int nt) { return nt / T + (nt % T != 0 ? 1 : 0); };
    auto class_of = [&](int nt, int np) { return static_cast<int>((static_cast<int64_t>((nt + np - 1) / np - 1) * kPlanClasses) / T); };
    // segments in each class, slots of the parts and numbers of the jobs that are cut: prefix sums over the threads
    int64_t cut = 0, all_cuts = 0;
    int own[kPlanClasses] = {};
    for (int j = ja; j < jb; ++j) {
        const int nt = tiles_of(j);
        if (nt == 0) continue;
        const int np = pieces_of(nt), cl = class_of(nt, np);
        if (np > 1) cut += (static_cast<int64_t>(np) << 32) + 1;
#pragma unroll
        for (int c = 0; c < kPlanClasses; ++c) own[c] += c == cl ? np : 0;
    }
    const int64_t cut_upto = warp_scan(cut);
    if (lane == 31) cut_totals[warp] = cut_upto;
    cut = cut_upto - cut;
#pragma unroll
    for (int c = 0; c < kPlanClasses; ++c) {
        const int upto = warp_scan(own[c]);
        if (lane == 31) classes[c][warp] = upto;
        own[c] = upto - own[c];
    }
    __syncthreads();
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w < warp) cut += cut_totals[w];
        all_cuts += cut_totals[w];
    }
    const int cut_jobs = static_cast<int>(all_cuts & 0xffffffff);
    int begin = 0;   // segments of the longer classes, of this one in the warps before
#pragma unroll
    for (int c = kPlanClasses - 1; c >= 0; --c) {
        own[c] += begin;
        for (int w = 0; w < kPlanWarps; ++w) {
            const int v = classes[c][w];
            if (w < warp) own[c] += v;
            begin += v;
        }
    }
    for (int j = ja; j < jb; ++j) {
        const int nt = tiles_of(j);
        if (nt == 0) continue;
        const int np = pieces_of(nt), cl = class_of(nt, np);
        int at = 0;
#pragma unroll
        for (int c = 0; c < kPlanClasses; ++c)
            if (c == cl) {
                at = own[c];
                own[c] += np;
            }
        const paged::Job job = paged::job_info<kRows, kKeys>(a, j);
        if (np > 1 && static_cast<int>(cut & 0xffffffff) < headers)
            hdr[cut & 0xffffffff] = make_int4(job.seq * a.rows_per_seq + job.row0, job.rows, np, static_cast<int>(cut >> 32));
        for (int p = 0; p < np && at < max_segments; ++p, ++at) {
            const int t0 = static_cast<int>(static_cast<int64_t>(nt) * p / np), t1 = static_cast<int>(static_cast<int64_t>(nt) * (p + 1) / np);
            int4* s = reinterpret_cast<int4*>(segments + at);
            s[0] = make_int4(job.seq, job.row0, job.rows, job.keys);
            s[1] = make_int4(t0 * kKeys, t1 - t0, job.first_pos, job.first_tok);
            s[2] = make_int4(np > 1 ? static_cast<int>(cut >> 32) + p : -1, 0, 0, 0);
        }
        if (np > 1) cut += (static_cast<int64_t>(np) << 32) + 1;
    }
    for (int k = begin + static_cast<int>(threadIdx.x); k < max_segments; k += kPlanThreads)
        reinterpret_cast<int4*>(segments + k)[1] = make_int4(0, 0, 0, 0);
    for (int k = cut_jobs + static_cast<int>(threadIdx.x); k < headers; k += kPlanThreads) hdr[k] = make_int4(0, 0, 0, 0);
}

}  // namespace

// Segments at most, whatever the lengths are.
int64_t paged_max_segments(int64_t jobs, int pairs) { return waves(jobs, pairs) * pairs; }

// How many pairs of this kernel run at once on the current device, asked once per device (every record format
// leaves one CTA per SM).
int paged_pairs(int sms) {
    using namespace pairdec;
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return sms / 2;
    }
    int pairs = known[dev].load(std::memory_order_relaxed);
    if (pairs > 0) return pairs;
    if (prepare_kernel<432, false, true>() == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemAlloc<432>;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&pairs, decode_pair_kernel<432, false, true>, &cfg) != cudaSuccess) pairs = 0;
    }
    (void)cudaGetLastError();
    if (pairs < 1 || pairs > sms / 2) pairs = sms / 2;
    known[dev].store(pairs, std::memory_order_relaxed);
    return pairs;
}

cudaError_t launch_paged_decode_pair(const PagedDecodeArgs& d, int max_segments, int headers, cudaStream_t stream) {
    using namespace pairdec;
    KernelArgs a = {};
    if (!encode_q_map(&a.qmap, d.q, static_cast<int64_t>(d.jobs.batch) * d.jobs.rows_per_seq)) return cudaErrorInvalidValue;
    a.cache = d.cache;
    a.splits = 1;
    a.sm_scale = d.sm_scale;
    a.sink = d.attn_sink;
    a.out = static_cast<__nv_bfloat16*>(d.out);
    a.lse = d.lse;
    a.part_out = d.part_out;
    a.part_lse = d.part_lse;
    a.status = d.dev_status;
    a.jobs = d.jobs;
    a.jobs.row_tiles = (a.jobs.rows_per_seq + 127) / 128;
    a.segments = static_cast<const Segment*>(d.segments);
    const auto kernel = d.record_bytes == 432 ? decode_pair_kernel<432, false, true>
                        : d.block_scales      ? decode_pair_kernel<352, true, true>
                                              : decode_pair_kernel<352, false, true>;
    cudaError_t err = d.record_bytes == 432 ? prepare_kernel<432, false, true>()
                      : d.block_scales      ? prepare_kernel<352, true, true>()
                                            : prepare_kernel<352, false, true>();
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddepcontrol.wait
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(1 + kPlanEmpty);
    cfg.blockDim = dim3(kPlanThreads);
    err = cudaLaunchKernelEx(&cfg, paged_plan_kernel, a.jobs, d.pairs, max_segments, headers, static_cast<Segment*>(d.segments),
                             reinterpret_cast<int4*>(d.hdr), d.out, d.lse, d.dev_status);
    if (err != cudaSuccess) return err;
    // a pair per segment (those behind the last one leave at once)
    cfg.gridDim = dim3(2u * static_cast<unsigned>(max_segments));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = d.record_bytes == 432 ? kSmemAlloc<432> : kSmemAlloc<352>;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, kernel, a);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace nvfp4mla

// paged_jobs.cuh -- how attention through a page table is cut into work: jobs (a sequence and a tile of its
// query rows), their tiles of keys, and the runs of tiles that the CTAs of the one-CTA kernel take.
//
// The s_q * h_q query rows of a sequence lie one behind the other in q; rows row0 .. row0 + rows - 1 of a
// job share every key that is dequantized. For one CTA each (paged_decode_few.cu) the tiles of all jobs, one job behind
// the other, are cut into equal runs; CTA pairs take the segments that a plan kernel cuts the jobs into
// (paged_decode_pair.cu). Lengths are read on the device, so a captured call follows them.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace nvfp4mla {
namespace paged {

struct Jobs {
    const int32_t* page_table;
    int64_t table_stride;
    const int32_t* seq_lens;
    int num_pages;            // pages of the pool
    int page_shift;
    int capacity;             // tokens that a page table row can name
    int batch, s_q, h_q;
    int rows_per_seq;         // s_q * h_q
    int row_tiles;            // ceil(rows_per_seq / rows of a job)
};

struct Job {
    int seq, row0, rows;      // rows row0 .. row0 + rows - 1 of sequence seq
    int keys;                 // keys that some of them sees
    int tiles;
    int first_pos, first_tok; // position and token of row row0
};

// Job `job` of row tiles of kRows rows and key tiles of kKeys keys. Row tiles of 128 cut the rows of a sequence; with
// smaller ones a sequence's rows are one job. (Not inlined: its divisions are long, and it runs once per
// job, beside loops that should stay in the instruction cache.)
template <int kRows, int kKeys>
__device__ __noinline__ Job job_info(const Jobs& a, int job) {
    Job j;
    j.seq = kRows < 128 ? job : job / a.row_tiles;
    j.row0 = kRows < 128 ? 0 : (job - j.seq * a.row_tiles) * kRows;
    j.rows = kRows < 128 ? a.rows_per_seq : min(kRows, a.rows_per_seq - j.row0);
    const int len = min(max(__ldg(a.seq_lens + j.seq), 0), a.capacity);
    const int last_tok = kRows < 128 ? a.s_q - 1 : (j.row0 + j.rows - 1) / a.h_q;
    j.first_tok = kRows < 128 ? 0 : j.row0 / a.h_q;
    j.keys = max(0, len - a.s_q + last_tok + 1);
    j.tiles = j.keys / kKeys + (j.keys % kKeys != 0 ? 1 : 0);   // (keys may lie near 2^31)
    j.first_pos = len - a.s_q + j.first_tok;
    return j;
}

// The reference m of a row whose tile has the largest score zt (log2 units), zmin being the smallest of the largest scores
// of its four quarters. Weights 2^(z - m) are held in f16: off by 2^-11 of themselves down to 2^-14, by 2^-25 below,
// so a key that lies far below the largest is held the better the further m lies below it; a score may exceed m
// by kMaxWeightLog2 until the row's output has to be rescaled. m = zt - 3 costs no time against m = zt (64 sequences x 16
// heads 166 / 166 us, 2 chunks of 256 tokens x 64 heads 904 / 911 us: 15 bits of range above m then, 12.9 now), m = zt - 7
// does (172.5 and 943 us), as ordinary rows meet larger scores later. Where one key outweighs whole quarters of its tile
// (an attention sink, whose own value is often near 0: the others are what the output consists of), larger scores are
// rare, and m lies up to 12 below, so that the others stay above 2^-14 up to 2^26 below the largest.
constexpr float kMaxWeightLog2 = 15.9f;   // 2^15.9 < 65504
__device__ __forceinline__ float new_reference(float zt, float zmin) { return zt - fminf(fmaxf(zt - zmin - 14.0f, 3.0f), 12.0f); }

// Parts of cut rows are f16 outputs times this: |V| is at most 6 x 448 (and 16 times that below 65504), and what is
// rounded to steps of f16 below 2^-14 should be small against the smallest V other than 0, 2^-10.
constexpr float kPartScale = 16.0f;

// Slot of the token at position pos of a sequence; -1: none of the `keys` first, -2: its page is outside the pool.
__device__ __forceinline__ int slot_of(const Jobs& a, int seq, int keys, int pos) {
    if (pos >= keys) return -1;
    const int page = __ldg(a.page_table + seq * a.table_stride + (pos >> a.page_shift));
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.num_pages)) return -2;
    return (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// Where run c of (at most) `runs` begins, its tiles, and the tiles of all jobs (one-CTA kernel). The prefix sum over the jobs'
// tiles takes a contiguous piece of the jobs per thread; scratch: int64 [33 + 2], shared. Block-collective.
struct Run {
    int64_t total, runs;      // tiles of all jobs; runs that are not empty
    int job, tile, count;
};
// The run that holds tile t of all.
__device__ __forceinline__ int run_of(const Run& r, int64_t t) { return static_cast<int>(((t + 1) * r.runs - 1) / r.total); }

// Where run c of runs (at most 160) begins.
__device__ __forceinline__ int64_t run_begin(int64_t total, int64_t runs, int64_t c) {
    if (total < (int64_t(1) << 23)) return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(runs);   // short division
    return total * c / runs;
}

template <int kRows, int kKeys, int kThreads>
__device__ __noinline__ Run find_run(const Jobs& a, int64_t* scratch, int runs, int c) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int jobs = a.batch * a.row_tiles;
    const int per = (jobs + kThreads - 1) / kThreads;
    const int ja = min(jobs, static_cast<int>(threadIdx.x) * per), jb = min(jobs, ja + per);
    int64_t mine = 0;
    for (int j = ja; j < jb; ++j) mine += job_info<kRows, kKeys>(a, j).tiles;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    Run r;
    r.total = 0;
    int64_t before = incl - mine;
    for (int w = 0; w < kThreads / 32; ++w) {
        const int64_t v = scratch[w];
        if (w < warp) before += v;
        r.total += v;
    }
    r.runs = min(static_cast<int64_t>(runs), r.total);
    r.count = 0;
    int* found = reinterpret_cast<int*>(scratch + 33);
    if (c < r.runs) {
        const int64_t g0 = run_begin(r.total, r.runs, c);
        r.count = static_cast<int>(run_begin(r.total, r.runs, c + 1) - g0);
        if (before <= g0 && g0 < before + mine) {
            int64_t at = before;
            int j = ja;
            for (;; ++j) {
                const int nt = job_info<kRows, kKeys>(a, j).tiles;
                if (g0 < at + nt) break;
                at += nt;
            }
            found[0] = j;
            found[1] = static_cast<int>(g0 - at);
        }
    }
    __syncthreads();
    r.job = found[0];
    r.tile = found[1];
    return r;
}

// Jobs without a visible key (block b of `blocks` takes every blocks-th job): out = 0, lse = -inf.
template <int kRows, int kKeys, int kThreads>
__device__ __noinline__ void write_empty_jobs(const Jobs& a, int b, int blocks, void* out, float* lse) {
    const int jobs = a.batch * a.row_tiles;
    for (int job = b; job < jobs; job += blocks) {
        const Job j = job_info<kRows, kKeys>(a, job);
        if (j.tiles > 0) continue;
        const int64_t row = static_cast<int64_t>(j.seq) * a.rows_per_seq + j.row0;
        uint4* o = static_cast<uint4*>(out) + row * 64;
        for (int e = threadIdx.x; e < j.rows * 64; e += kThreads) o[e] = make_uint4(0u, 0u, 0u, 0u);
        for (int e = threadIdx.x; e < j.rows; e += kThreads) lse[row + e] = -INFINITY;
    }
}

// Lengths beyond the page table are reported (and read as its capacity).
__device__ __forceinline__ void check_lengths(const Jobs& a, int thread, int threads, uint32_t* status) {
    if (status == nullptr) return;
    for (int b = thread; b < a.batch; b += threads)
        if (__ldg(a.seq_lens + b) > a.capacity) atomicOr(status, 0x2u);
}

}  // namespace paged
}  // namespace nvfp4mla

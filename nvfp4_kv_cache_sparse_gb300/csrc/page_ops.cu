// page_ops.cu -- operations on the pages of record caches: copying pages, forking sequences (pages shared
// and counted), resizing them (pages taken and given back, a shared page copied before it is written),
// and compacting a pool.
//
// State, all on the device. page_table [batch, max_pages]: the pages of each sequence in order, -1 behind
// its last one. seq_lens [batch]. page_refs [num_pages]: how many table entries name a page; a page
// is free exactly when its count is 0. There is no other free list, so nothing can disagree with it.
// Every page is taken in one fixed order (the lowest free pages, handed out in the order of the
// sequences), so a call's result depends on its inputs alone; counts change by integer atomics,
// whose order does not matter.
//
// Each bookkeeping step is one launch of one cluster of eight CTAs, whose barriers separate its
// phases; the pages' order comes from a prefix sum over the counts (a slice per CTA, the slices'
// totals exchanged through distributed shared memory). Records are copied by a second grid over all
// SMs, launched as a programmatic dependent: how many pages it copies is known on the device only.
//
// What bounds it. Copies the memory: 512 pages in 16 caches (453 MB read and written) 75 us, 6.1 TB/s; a compaction
// that moves 512 of 1024 pages in 16 caches 67 us, 5.5 TB/s. The bookkeeping the latency of its phases, each a few dependent
// loads and a cluster barrier (4 to 8 us on the device: 64 sequences growing by 4 tokens in a pool of 32768
// pages 8 us), and for a call made from Python the host (about 8 us, and 4 to 5 us per launch), hence few launches.
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "sm103_ptx.cuh"

namespace nvfp4mla {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;            // 16-byte vectors of a copy thread in flight
constexpr int kCopyBlocksPerSm = 6;
// A resize copies shared last pages itself where they cannot be many bytes, else in a launch of their own. One launch /
// two, device time, 64-record pages of 352 bytes: 64 sequences, nothing shared (the usual call) 6.0 / 6.7 us, every
// page shared (1.4 MB) 10.0 / 8.8 us; 128 sequences 6.1 / 7.2 and 12.6 / 9.1 us; and 4 us less of the host's time.
constexpr int64_t kResizeCopyBytes = 2 << 20;   // shared pages of a resize that its own cluster copies, at most
constexpr int kResizeCows = 1024;       // of them of one CTA
static_assert(kResizeCopyBytes / 352 / kCluster + 1 <= kResizeCows, "a page has a record or more");
constexpr uint32_t kDevIndex = 0x2u, kDevExhausted = 0x20u, kDevLength = 0x40u;

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void flag(uint32_t* status, uint32_t bit) {
    if (status != nullptr) atomicOr(status, bit);
}

// ---- copies ----------------------------------------------------------------------------------------

struct Caches {
    uint8_t* p[kMaxCaches];
};

struct CopyList {
    const int32_t* src;       // entry k: page src[k] to page dst[k] (a negative one: nothing to copy)
    const int32_t* dst;
    const int32_t* records;   // nullable: records of entry k (else the whole page)
    const int32_t* count;     // nullable: entries (device), else n
    int n;
};

struct CopyShape {
    int num_caches, num_pages;
    int page_vecs, rec_vecs;  // 16-byte vectors of a page, of a record
    int parts;                // pieces a page is cut into
};

// A unit is one piece (at most kCopyThreads x kCopyVecs vectors) of the first `vecs` vectors of one page of one
// cache, for thread t of kCopyThreads: every thread has its loads in flight before it stores any.
__device__ __forceinline__ void copy_unit(uint8_t* cache, const CopyShape& sh, int s, int d, int vecs, int part, int t) {
    const int per = (vecs + sh.parts - 1) / sh.parts;
    const int end = min(vecs, (part + 1) * per);
    const uint4* from = reinterpret_cast<const uint4*>(cache) + static_cast<int64_t>(s) * sh.page_vecs;
    uint4* to = reinterpret_cast<uint4*>(cache) + static_cast<int64_t>(d) * sh.page_vecs;
    const int v0 = part * per + t;
    uint4 x[kCopyVecs];
#pragma unroll
    for (int e = 0; e < kCopyVecs; ++e)
        if (v0 + e * kCopyThreads < end) x[e] = __ldcs(from + v0 + e * kCopyThreads);
#pragma unroll
    for (int e = 0; e < kCopyVecs; ++e)
        if (v0 + e * kCopyThreads < end) __stcs(to + v0 + e * kCopyThreads, x[e]);
}

__device__ __forceinline__ void copy_units(const Caches& caches, const CopyShape& sh, const CopyList& list, uint32_t* status) {
    const int n = list.count != nullptr ? *list.count : list.n;
    const int64_t per_cache = static_cast<int64_t>(n) * sh.parts, units = per_cache * sh.num_caches;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int l = static_cast<int>(u / per_cache);
        const int64_t v = u - l * per_cache;
        const int k = static_cast<int>(v / sh.parts), part = static_cast<int>(v - static_cast<int64_t>(k) * sh.parts);
        const int s = __ldg(list.src + k), d = __ldg(list.dst + k);
        if (s < 0 || d < 0 || s == d) continue;
        if (s >= sh.num_pages || d >= sh.num_pages) {
            if (l == 0 && part == 0 && threadIdx.x == 0) flag(status, kDevIndex);
            continue;
        }
        copy_unit(caches.p[l], sh, s, d, list.records != nullptr ? __ldg(list.records + k) * sh.rec_vecs : sh.page_vecs, part, threadIdx.x);
    }
}

__global__ void __launch_bounds__(kCopyThreads, kCopyBlocksPerSm)
copy_pages_kernel(const __grid_constant__ Caches caches, const CopyShape sh, const CopyList list, uint32_t* status) {
    pdl_wait();
    copy_units(caches, sh, list, status);
}

// ---- cluster helpers -------------------------------------------------------------------------------

// The inclusive sum over the block's threads up to this one, and the sum over all of them.
__device__ __forceinline__ int block_scan(int a, int* scratch, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = a;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    __syncthreads();   // the scratch of the scan before has been read
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    const int t = scratch[lane];
    int s = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    return __shfl_sync(0xffffffffu, s - t, warp) + incl;
}

// Gives every CTA of the cluster this CTA's value at slot[rank]; to be read after cluster_sync(). A CTA's shared memory
// may be written to once it runs, which a barrier of the cluster has to have shown before a kernel's first use.
__device__ __forceinline__ void publish(int* slot, uint32_t rank, int value) {
    if (threadIdx.x < kCluster) {
        const uint32_t remote = mapa_shared(smem_addr(slot + rank), threadIdx.x);
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(value) : "memory");
    }
}

__device__ __forceinline__ int pages_of(int len, int shift) { return static_cast<int>((static_cast<int64_t>(len) + (1 << shift) - 1) >> shift); }

// This CTA's slice of the pages: a multiple of four, so that the counts are read as 16-byte vectors.
__device__ __forceinline__ void slice(int num_pages, uint32_t rank, int* lo, int* hi) {
    const int64_t per = ((static_cast<int64_t>(num_pages) + kCluster - 1) / kCluster + 3) & ~int64_t(3);
    *lo = static_cast<int>(min(static_cast<int64_t>(num_pages), per * rank));
    *hi = static_cast<int>(min(static_cast<int64_t>(num_pages), per * rank + per));
}
// Four counts from page p on (a multiple of four); `fill` behind the end.
__device__ __forceinline__ int4 counts4(const int32_t* refs, int p, int end, int fill) {
    if (end - p >= 4) return __ldcg(reinterpret_cast<const int4*>(refs + p));
    int4 v = make_int4(fill, fill, fill, fill);
    if (end - p > 0) v.x = __ldcg(refs + p);
    if (end - p > 1) v.y = __ldcg(refs + p + 1);
    if (end - p > 2) v.z = __ldcg(refs + p + 2);
    return v;
}

// ---- resize ----------------------------------------------------------------------------------------

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
resize_kernel(const __grid_constant__ Caches caches, const CopyShape sh, const ResizeArgs a) {
    __shared__ int scratch[32];
    __shared__ int need_of[kCluster], free_of[kCluster];
    __shared__ int4 cow_list[kResizeCows];   // {source page, target page, records} that this CTA copies itself
    __shared__ int cows;
    if (threadIdx.x == 0) cows = 0;          // (many barriers ahead of its use)
    pdl_trigger();
    pdl_wait();
    const uint32_t rank = cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b0 = static_cast<int>(static_cast<int64_t>(a.batch) * rank / kCluster);
    const int b1 = static_cast<int>(static_cast<int64_t>(a.batch) * (rank + 1) / kCluster);
    const int cap = a.width << a.shift;
    const int mask = (1 << a.shift) - 1;
    auto old_len = [&](int b) { return min(max(__ldcg(a.seq_lens + b), 0), cap); };
    auto new_len = [&](int b, int old) {
        const int n = __ldg(a.new_lens + b);
        return n < 0 || n > cap ? old : n;
    };
    auto page_ok = [&](int p) { return static_cast<unsigned>(p) < static_cast<unsigned>(a.num_pages); };

    // ---- shrinking: pages behind the new last one are given back
    for (int b = b0 + warp; b < b1; b += kThreads / 32) {
        const int old = old_len(b), now = new_len(b, old);
        if (lane == 0) {
            const int n = __ldg(a.new_lens + b);
            if (n < 0 || n > cap) flag(a.status, kDevLength);
        }
        if (now >= old) continue;
        int32_t* row = a.page_table + b * a.table_stride;
        for (int j = pages_of(now, a.shift) + lane; j < pages_of(old, a.shift); j += 32) {
            const int p = row[j];
            if (page_ok(p))
                atomicSub(a.page_refs + p, 1);
            else
                flag(a.status, kDevIndex);
            row[j] = -1;
        }
        __syncwarp();
        if (lane == 0) a.seq_lens[b] = now;
    }
    cluster_sync();

    // ---- how many pages each sequence takes (one more where its partly filled last page is shared), how
    // many are free
    int need = 0;
    for (int r = b0; r < b1; r += kThreads) {
        const int b = r + threadIdx.x;
        int mine = 0, tail = -1;
        if (b < b1) {
            const int old = old_len(b), now = new_len(b, old);
            if (now > old) {
                mine = pages_of(now, a.shift) - pages_of(old, a.shift);
                if ((old & mask) != 0) {
                    const int p = __ldcg(a.page_table + b * a.table_stride + (old >> a.shift));
                    if (!page_ok(p))
                        flag(a.status, kDevIndex);
                    else if (__ldcg(a.page_refs + p) > 1) {
                        tail = p;
                        ++mine;
                    }
                }
            }
        }
        int total;
        const int incl = block_scan(mine, scratch, &total);
        if (b < b1) {
            a.offset[b] = need + incl - mine;
            a.cow_src[b] = tail;
            a.cow_dst[b] = -1;
        }
        need += total;
    }
    int lo, hi;
    slice(a.num_pages, rank, &lo, &hi);
    int nfree = 0;
    for (int64_t p = lo + 4 * threadIdx.x; p < hi; p += 4 * kThreads) {
        const int4 v = counts4(a.page_refs, static_cast<int>(p), hi, 1);
        nfree += (v.x == 0) + (v.y == 0) + (v.z == 0) + (v.w == 0);
    }
    (void)block_scan(nfree, scratch, &nfree);
    publish(need_of, rank, need);
    publish(free_of, rank, nfree);
    cluster_sync();
    int need_before = 0, free_before = 0;
    int64_t need_all = 0, free_all = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
        if (c < static_cast<int>(rank)) {
            need_before += need_of[c];
            free_before += free_of[c];
        }
        need_all += need_of[c];
        free_all += free_of[c];
    }
    const bool enough = need_all <= free_all;   // the same in every CTA
    if (!enough && rank == 0 && threadIdx.x == 0) flag(a.status, kDevExhausted);

    // ---- the lowest need_all free pages, in order
    if (enough) {
        int at = free_before;
        for (int64_t r = lo; r < hi && at < need_all; r += 4 * kThreads) {
            const int64_t p64 = r + 4 * threadIdx.x;
            const int p = static_cast<int>(p64);
            const int4 v = p64 < hi ? counts4(a.page_refs, p, hi, 1) : make_int4(1, 1, 1, 1);
            const int mine = (v.x == 0) + (v.y == 0) + (v.z == 0) + (v.w == 0);
            int total;
            int w = at + block_scan(mine, scratch, &total) - mine;
            if (v.x == 0 && w++ < need_all) a.free_list[w - 1] = p;
            if (v.y == 0 && w++ < need_all) a.free_list[w - 1] = p + 1;
            if (v.z == 0 && w++ < need_all) a.free_list[w - 1] = p + 2;
            if (v.w == 0 && w++ < need_all) a.free_list[w - 1] = p + 3;
            at += total;
        }
    }
    cluster_sync();

    // ---- growing: table entries, counts, lengths, the new tokens' slots
    for (int b = b0 + warp; b < b1; b += kThreads / 32) {
        const int old = old_len(b), now = enough ? new_len(b, old) : old;
        int32_t* row = a.page_table + b * a.table_stride;
        const int n0 = pages_of(old, a.shift);
        const int32_t* mine = a.free_list + need_before + __ldcg(a.offset + b);
        const int tail = now > old ? __ldcg(a.cow_src + b) : -1;
        const int cow = tail >= 0 ? 1 : 0;
        if (now > old) {
            for (int j = n0 + lane; j < pages_of(now, a.shift); j += 32) {
                const int p = __ldcg(mine + cow + j - n0);
                row[j] = p;
                a.page_refs[p] = 1;
            }
        }
        const int own = cow != 0 ? __ldcg(mine) : -1;
        for (int j = lane; j < a.max_new; j += 32) {
            int64_t slot = -1;
            const int64_t pos = static_cast<int64_t>(old) + j;
            if (pos < now) {
                const int i = static_cast<int>(pos >> a.shift);
                const int p = i >= n0 ? __ldcg(mine + cow + i - n0) : cow != 0 ? own : __ldcg(row + i);
                if (page_ok(p)) slot = (static_cast<int64_t>(p) << a.shift) + (pos & mask);
            }
            a.slots[static_cast<int64_t>(b) * a.max_new + j] = slot;
        }
        __syncwarp();
        if (lane == 0 && now > old) {
            if (cow != 0) {
                atomicSub(a.page_refs + tail, 1);
                a.page_refs[own] = 1;
                row[n0 - 1] = own;
                a.cow_dst[b] = own;
                if (sh.num_caches > 0) cow_list[atomicAdd(&cows, 1)] = make_int4(tail, own, old & mask, 0);
            }
            a.cow_records[b] = old & mask;
            a.seq_lens[b] = now;
        }
    }
    if (sh.num_caches == 0) return;   // nothing to copy, or the copies are a launch of their own
    __syncthreads();
    constexpr int kGroups = kThreads / kCopyThreads;
    for (int u = threadIdx.x / kCopyThreads; u < cows * sh.parts * sh.num_caches; u += kGroups) {
        const int4 c = cow_list[u / sh.parts % cows];
        copy_unit(caches.p[u / sh.parts / cows], sh, c.x, c.y, c.z * sh.rec_vecs, u % sh.parts, threadIdx.x % kCopyThreads);
    }
}

// ---- fork ------------------------------------------------------------------------------------------

// Pair k counts if no later pair names the same target; every pass decides it alike. `t` of `n` threads, all
// of which call it; each has to combine the answers (false anywhere: the pair does not count).
__device__ __forceinline__ bool fork_counts(const ForkArgs& a, int k, int t, int n, int* src, int* dst) {
    const int s = __ldg(a.src + k), d = __ldg(a.dst + k);
    *src = s;
    *dst = d;
    if (s < 0 || d < 0) return false;
    if (s >= a.batch || d >= a.batch) {
        if (t == 0) flag(a.status, kDevIndex);
        return false;
    }
    bool last = true;
    for (int i = k + 1 + t; i < a.pairs; i += n)
        last = last && !(__ldg(a.dst + i) == d && static_cast<unsigned>(__ldg(a.src + i)) < static_cast<unsigned>(a.batch));
    return last;
}

// The first pass reads the table only: the source's row goes to the workspace, its pages are counted once more,
// the target's old pages once less. The second writes the target's row. A permutation of sequences therefore
// sees every row as it was. Thread t of n.
__device__ __forceinline__ void fork_read(const ForkArgs& a, int k, int s, int d, int t, int n) {
    const int cap = a.width << a.shift;
    const int ns = pages_of(min(max(a.seq_lens[s], 0), cap), a.shift), nd = pages_of(min(max(a.seq_lens[d], 0), cap), a.shift);
    const int32_t* from = a.page_table + s * a.table_stride;
    const int32_t* to = a.page_table + d * a.table_stride;
    int32_t* stage = a.stage + static_cast<int64_t>(k) * (a.width + 1);
#pragma unroll 4
    for (int j = t; j < a.width; j += n) {
        int p = -1;
        if (j < ns) {
            p = from[j];
            if (static_cast<unsigned>(p) < static_cast<unsigned>(a.num_pages))
                atomicAdd(a.page_refs + p, 1);
            else
                flag(a.status, kDevIndex);
        }
        stage[1 + j] = p;
        if (j < nd) {
            const int g = to[j];
            if (static_cast<unsigned>(g) < static_cast<unsigned>(a.num_pages))
                atomicSub(a.page_refs + g, 1);
            else
                flag(a.status, kDevIndex);
        }
    }
    if (t == 0) stage[0] = a.seq_lens[s];
}
__device__ __forceinline__ void fork_write(const ForkArgs& a, int k, int d, int t, int n) {
    const int32_t* stage = a.stage + static_cast<int64_t>(k) * (a.width + 1);
    int32_t* to = a.page_table + d * a.table_stride;
#pragma unroll 4
    for (int j = t; j < a.width; j += n) to[j] = __ldcg(stage + 1 + j);
    if (t == 0) a.seq_lens[d] = __ldcg(stage);
}

// Few pairs and short rows: one launch of one cluster, its barrier between the passes; `group` threads per
// pair (a power of two, whole warps: each warp decides for itself whether the pair counts).
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1) fork_cluster_kernel(const ForkArgs a, int group) {
    pdl_trigger();
    pdl_wait();
    const int t = static_cast<int>(threadIdx.x) & (group - 1);
    const int k = static_cast<int>(cluster_ctarank()) + kCluster * (static_cast<int>(threadIdx.x) / group);
    int s = 0, d = 0;
    const bool counts = k < a.pairs && __all_sync(0xffffffffu, fork_counts(a, k, t & 31, 32, &s, &d)) != 0 && s != d;
    if (counts) fork_read(a, k, s, d, t, group);
    cluster_sync();
    if (counts) fork_write(a, k, d, t, group);
}

__global__ void __launch_bounds__(kCopyThreads) fork_read_kernel(const ForkArgs a) {
    pdl_trigger();
    pdl_wait();
    int s, d;
    if (__syncthreads_and(fork_counts(a, blockIdx.x, threadIdx.x, kCopyThreads, &s, &d)) != 0 && s != d)
        fork_read(a, blockIdx.x, s, d, blockIdx.y * kCopyThreads + threadIdx.x, gridDim.y * kCopyThreads);
}

__global__ void __launch_bounds__(kCopyThreads) fork_write_kernel(const ForkArgs a) {
    pdl_wait();
    int s, d;
    if (__syncthreads_and(fork_counts(a, blockIdx.x, threadIdx.x, kCopyThreads, &s, &d)) != 0 && s != d)
        fork_write(a, blockIdx.x, d, blockIdx.y * kCopyThreads + threadIdx.x, gridDim.y * kCopyThreads);
}

// ---- compact ---------------------------------------------------------------------------------------

// With n live pages, the live pages behind page n move into the free pages before it, in order: the i-th
// such page into the i-th such hole. No page is both, so all copies may run at once. With r(p) live
// pages before page p and L = r(n): page p >= n is the mover number r(p) - L, page p < n the hole
// number p - r(p).
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1) compact_plan_kernel(const CompactArgs a) {
    __shared__ int scratch[32];
    __shared__ int live_of[kCluster], below_of[kCluster];
    cluster_arrive();   // (its wait, ahead of the first publish, is hidden by the counting)
    pdl_trigger();
    pdl_wait();
    const uint32_t rank = cluster_ctarank();
    int lo, hi;
    slice(a.num_pages, rank, &lo, &hi);
    auto count_live = [&](int end) {
        int n = 0, total;
        for (int64_t p = lo + 4 * threadIdx.x; p < end; p += 4 * kThreads) {
            const int4 v = counts4(a.page_refs, static_cast<int>(p), end, 0);
            n += (v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0);
        }
        (void)block_scan(n, scratch, &total);
        return total;
    };
    const int mine = count_live(hi);
    cluster_wait();     // every CTA of the cluster runs
    publish(live_of, rank, mine);
    cluster_sync();
    int n = 0, before = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
        if (c < static_cast<int>(rank)) before += live_of[c];
        n += live_of[c];
    }
    publish(below_of, rank, hi <= n ? mine : lo >= n ? 0 : count_live(n));
    cluster_sync();
    int below = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) below += below_of[c];
    const int moves = n - below;

    int at = before;
    for (int64_t r = lo; r < hi; r += 4 * kThreads) {
        const int64_t p64 = r + 4 * threadIdx.x;
        const int p0 = static_cast<int>(min(p64, static_cast<int64_t>(hi)));
        const int4 v4 = counts4(a.page_refs, p0, hi, 0);
        const int v[4] = {v4.x, v4.y, v4.z, v4.w};
        int total;
        int w = (v[0] > 0) + (v[1] > 0) + (v[2] > 0) + (v[3] > 0);
        w = at + block_scan(w, scratch, &total) - w;   // live pages before p0
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (hi - p0 <= e) break;
            const int p = p0 + e;
            if (v[e] > 0) {
                if (p < n) {
                    a.page_map[p] = p;
                    a.refs_out[p] = v[e];
                } else {
                    a.mover[w - below] = p;
                    a.mover_refs[w - below] = v[e];
                    a.refs_out[p] = 0;
                }
                ++w;
            } else {
                a.page_map[p] = -1;
                if (p < n)
                    a.hole[p - w] = p;
                else
                    a.refs_out[p] = 0;
            }
        }
        at += total;
    }
    cluster_sync();
    for (int i = rank * kThreads + threadIdx.x; i < moves; i += kCluster * kThreads) {
        const int p = __ldcg(a.mover + i), h = __ldcg(a.hole + i);
        a.page_map[p] = h;
        a.refs_out[h] = __ldcg(a.mover_refs + i);
    }
    if (rank == 0 && threadIdx.x == 0) {
        *a.live = n;
        *a.moves = moves;
    }
}

__global__ void __launch_bounds__(kCopyThreads, kCopyBlocksPerSm)
compact_apply_kernel(const __grid_constant__ Caches caches, const CopyShape sh, const CompactArgs a) {
    pdl_wait();
    const int cap = a.width << a.shift;
    const int64_t entries = static_cast<int64_t>(a.batch) * a.width;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; i < entries; i += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
        const int b = static_cast<int>(i / a.width), j = static_cast<int>(i - static_cast<int64_t>(b) * a.width);
        int to = -1;
        if (j < pages_of(min(max(__ldg(a.seq_lens + b), 0), cap), a.shift)) {
            const int p = a.page_table[b * a.table_stride + j];
            if (static_cast<unsigned>(p) < static_cast<unsigned>(a.num_pages)) to = __ldg(a.page_map + p);
            if (to < 0) flag(a.status, kDevIndex);
        }
        a.table_out[b * a.table_out_stride + j] = to;
    }
    const CopyList list = {a.mover, a.hole, nullptr, a.moves, 0};
    copy_units(caches, sh, list, a.status);
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddepcontrol.wait
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args...);
    return err != cudaSuccess ? err : cudaGetLastError();
}

Caches caches_of(const PoolArgs& pool) {
    Caches c = {};
    for (int i = 0; i < pool.num_caches; ++i) c.p[i] = pool.caches[i];
    return c;
}
CopyShape shape_of(const PoolArgs& pool) {
    CopyShape s;
    s.num_caches = pool.num_caches;
    s.num_pages = pool.num_pages;
    s.rec_vecs = pool.record_bytes / 16;
    s.page_vecs = s.rec_vecs << pool.shift;
    s.parts = (s.page_vecs + kCopyThreads * kCopyVecs - 1) / (kCopyThreads * kCopyVecs);
    return s;
}
// Blocks for at most `entries` pages in every cache: one wave, or fewer where that is enough.
unsigned copy_blocks(const CopyShape& s, int64_t entries, int sms) {
    const int64_t units = entries * s.num_caches * s.parts, wave = static_cast<int64_t>(sms) * kCopyBlocksPerSm;
    return static_cast<unsigned>(units < wave ? (units > 0 ? units : 1) : wave);
}

}  // namespace

cudaError_t launch_copy_pages(const PoolArgs& pool, const int32_t* src, const int32_t* dst, int n, uint32_t* status, int sms,
                              cudaStream_t stream) {
    const CopyShape s = shape_of(pool);
    const CopyList list = {src, dst, nullptr, nullptr, n};
    return launch(copy_pages_kernel, dim3(copy_blocks(s, n, sms)), kCopyThreads, stream, caches_of(pool), s, list, status);
}

cudaError_t launch_resize(const ResizeArgs& a, const PoolArgs& pool, int sms, cudaStream_t stream) {
    const CopyShape s = shape_of(pool);
    CopyShape here = s;
    const int64_t most = static_cast<int64_t>(a.batch) * s.num_caches * s.page_vecs * 16;
    const bool apart = most > kResizeCopyBytes;
    if (apart) here.num_caches = 0;
    const cudaError_t err = launch(resize_kernel, dim3(kCluster), kThreads, stream, caches_of(pool), here, a);
    if (err != cudaSuccess || !apart) return err;
    const CopyList list = {a.cow_src, a.cow_dst, a.cow_records, nullptr, a.batch};
    return launch(copy_pages_kernel, dim3(copy_blocks(s, a.batch, sms)), kCopyThreads, stream, caches_of(pool), s, list, a.status);
}

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t stream) {
    // One launch where a row is at most four passes of the threads of its pair. Back to back on the device (one
    // launch / two): 4 pairs x 1024 pages 3.6 / 5.6 us, 32 x 512 4.7 / 5.0,
    // 256 x 128 6.9 / 4.7; a launch less also saves 4 us of the host's time.
    int group = kThreads;
    while (group > 32 && a.pairs > kCluster * (kThreads / group)) group /= 2;
    if (a.pairs <= kCluster * (kThreads / group) && a.width <= 4 * group) return launch(fork_cluster_kernel, dim3(kCluster), kThreads, stream, a, group);
    const int cols = (a.width + kCopyThreads * 4 - 1) / (kCopyThreads * 4);
    const dim3 grid(static_cast<unsigned>(a.pairs), static_cast<unsigned>(cols < 64 ? (cols > 0 ? cols : 1) : 64));
    const cudaError_t err = launch(fork_read_kernel, grid, kCopyThreads, stream, a);
    return err != cudaSuccess ? err : launch(fork_write_kernel, grid, kCopyThreads, stream, a);
}

cudaError_t launch_compact(const CompactArgs& a, const PoolArgs& pool, int sms, cudaStream_t stream) {
    const cudaError_t err = launch(compact_plan_kernel, dim3(kCluster), kThreads, stream, a);
    if (err != cudaSuccess) return err;
    const CopyShape s = shape_of(pool);
    const int64_t tables = (static_cast<int64_t>(a.batch) * a.width + kCopyThreads - 1) / kCopyThreads;
    const int64_t wave = static_cast<int64_t>(sms) * kCopyBlocksPerSm;
    int64_t blocks = copy_blocks(s, (static_cast<int64_t>(pool.num_pages) + 1) / 2, sms);
    if (blocks < tables) blocks = tables < wave ? tables : wave;
    return launch(compact_apply_kernel, dim3(static_cast<unsigned>(blocks)), kCopyThreads, stream, caches_of(pool), s, a);
}

}  // namespace nvfp4mla

// launch.h -- host-side launchers shared between the kernel translation units and the C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "paged_jobs.cuh"

namespace nvfp4mla {

// The fused producer stage ahead of the quantizer (nvfp4_mla_norm_rope_quantize_append).
struct ProducerArgs {
    const uint16_t* norm_weight;   // bf16 [512]
    float eps;
    const int64_t* positions;      // [num_tokens]
    const float* cos_table;        // fp32 [num_positions, 32]
    const float* sin_table;
    int64_t num_positions;
    int rotate_half;               // 1: pairs (f, f + 32); 0: pairs (2f, 2f + 1)
};

cudaError_t launch_quantize_append(const void* kv_latent, int64_t latent_row_stride, const void* k_rope,
                                   int64_t rope_row_stride, const int64_t* slot_mapping, int64_t num_tokens,
                                   uint8_t* cache, int64_t num_slots, int record_bytes, bool block_scales,
                                   uint32_t* dev_status, int sm_count, cudaStream_t stream,
                                   const ProducerArgs* producer = nullptr);

struct DecodeArgs {
    const void* q;             // bf16 [rows, h_q, 576]
    const uint8_t* cache;      // [num_slots, record_bytes]
    int64_t num_slots;
    int record_bytes;          // 352 or 432
    bool block_scales;         // 352 only: scales in block order instead of the permuted placement
    const int32_t* indices;    // [rows, topk]
    int rows;                  // batch * s_q
    int h_q;
    int topk;
    float sm_scale;
    const float* attn_sink;    // nullable [h_q]
    void* out;                 // bf16 [rows, h_q, 512]
    float* lse;                // [rows, h_q]
    int splits;
    uint16_t* part_out;        // f16 [rows, splits, h_q, 512] when splits > 1 (O / l of each split)
    float* part_lse;           // fp32 [rows, splits, h_q], log2 domain
    uint32_t* dev_status;
};

// The host-side checks of a decode call, in the order the entry points apply them: shape and
// record width, pointers and alignment (skipped when there are no rows), then a usable sm_103
// device. Sets rows (batch x s_q) and sms (0 unless every check passed).
int check_decode_call(const void* q, const uint8_t* cache, int64_t num_slots, int32_t record_bytes,
                      const int32_t* indices, int32_t batch, int32_t s_q, int32_t h_q, int32_t topk,
                      const float* attn_sink, const void* out, const float* lse, int32_t num_splits, int64_t* rows,
                      int* sms);

// Keys of one split, rounded to whole tiles.
int decode_keys_per_split(int topk, int splits);
cudaError_t launch_sparse_decode(const DecodeArgs& a, cudaStream_t stream);

// The CTA-pair decode with shared MMAs (sparse_decode_pair.cu): 128 heads, 352- or 432-byte records.
bool decode_pair_supported(const DecodeArgs& a);
int decode_pair_keys_per_split(int topk, int splits);
// Whether a decode of these arguments merges its splits inside the decode grid (2-4 splits per
// row in one cluster, the whole grid resident at once).
bool decode_pair_merges(const DecodeArgs& a);
// merged: set when the grid merges the splits itself (2-4 splits per row in one cluster).
cudaError_t launch_decode_pair(const DecodeArgs& a, cudaStream_t stream, bool* merged);
// The transposed-score decode for 64 heads on one SM (sparse_decode_h64.cu): 352- or 432-byte
// records.
bool decode_h64_supported(const DecodeArgs& a);
int decode_h64_keys_per_split(int topk, int splits);
cudaError_t launch_decode_h64(const DecodeArgs& a, cudaStream_t stream);
// The split merge (out, lse from the f16 partials), launched as a programmatic dependent.
cudaError_t launch_split_merge(const DecodeArgs& a, cudaStream_t stream);
// One time-bounded mbarrier wait that runs out (see nvfp4_mla_selftest_wait_timeout).
cudaError_t launch_wait_timeout_probe(uint32_t* status, uint64_t* elapsed_ns, cudaStream_t stream);

// ---- attention over whole sequences through a page table (paged_decode.cu)
struct PagedDecodeArgs {
    const void* q;               // bf16 [batch, s_q, h_q, 576]
    const uint8_t* cache;        // [num_pages << page_shift, record_bytes]
    int record_bytes;            // 352 or 432
    bool block_scales;
    paged::Jobs jobs;            // page table, lengths, shapes (row_tiles set by the launchers)
    float sm_scale;
    const float* attn_sink;      // nullable [h_q]
    void* out;                   // bf16 [batch, s_q, h_q, 512]
    float* lse;
    int runs;                    // one CTA each: equal runs that all tiles are cut into
    int pairs;                   // CTA pairs that run at once
    void* segments;              // workspace, see PagedWorkspace
    uint16_t* part_out;
    float* part_lse;
    int32_t* hdr;
    uint32_t* dev_status;
};
constexpr int kPagedMaxSms = 160;                // no sm_103 device has more SMs
int paged_row_tile(int64_t rows_per_seq);        // query rows that share dequantized keys: 16 (one CTA) or 128 (a pair)
size_t paged_workspace_bytes(int64_t batch, int64_t rows_per_seq);
int64_t paged_max_segments(int64_t jobs, int pairs);
cudaError_t launch_paged_decode(PagedDecodeArgs d, void* workspace, int sms, cudaStream_t stream);
int paged_pairs(int sms);
cudaError_t launch_paged_decode_few(const PagedDecodeArgs& d, cudaStream_t stream);
cudaError_t launch_paged_decode_pair(const PagedDecodeArgs& d, int max_segments, int headers, cudaStream_t stream);

// ---- operations on pages (page_ops.cu)
constexpr int kMaxCaches = 256;
struct PoolArgs {
    uint8_t* const* caches;      // host array of num_caches device pointers
    int num_caches, num_pages, shift;
    int record_bytes;
};
struct ResizeArgs {
    int32_t* page_table;
    int64_t table_stride;
    int width, shift;
    int32_t* seq_lens;
    const int32_t* new_lens;
    int batch;
    int32_t* page_refs;
    int num_pages;
    int64_t* slots;              // [batch, max_new]
    int max_new;
    int32_t *free_list, *offset, *cow_src, *cow_dst, *cow_records;   // workspace
    uint32_t* status;
};
struct ForkArgs {
    int32_t* page_table;
    int64_t table_stride;
    int width, shift;
    int32_t* seq_lens;
    int batch;
    int32_t* page_refs;
    int num_pages;
    const int32_t *src, *dst;
    int pairs;
    int32_t* stage;              // workspace [pairs, width + 1]
    uint32_t* status;
};
struct CompactArgs {
    const int32_t* page_table;
    int64_t table_stride;
    int32_t* table_out;
    int64_t table_out_stride;
    int width, shift;
    const int32_t* seq_lens;
    int batch;
    const int32_t* page_refs;
    int32_t* refs_out;
    int num_pages;
    int32_t *page_map, *live;
    int32_t *mover, *mover_refs, *hole, *moves;   // workspace
    uint32_t* status;
};
cudaError_t launch_copy_pages(const PoolArgs& pool, const int32_t* src, const int32_t* dst, int n, uint32_t* status, int sms,
                              cudaStream_t stream);
cudaError_t launch_resize(const ResizeArgs& a, const PoolArgs& pool, int sms, cudaStream_t stream);
cudaError_t launch_fork(const ForkArgs& a, cudaStream_t stream);
cudaError_t launch_compact(const CompactArgs& a, const PoolArgs& pool, int sms, cudaStream_t stream);

}  // namespace nvfp4mla

// api.cu -- the C ABI (include/nvfp4_mla.h): host-side argument checks, the platform gate,
// the split choice, and the kernel launches. Nothing here allocates device memory.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include "../../include/nvfp4_mla.h"
#include "launch.h"

namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxSplits = 64;
constexpr int kDecodeTile = 64;

// Per-device cache of (arch ok, SM count); 0 = unknown.
std::atomic<int> g_dev_state[kMaxDevices];   // -1 unsupported, >0 SM count

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Platform gate: the kernels are built for sm_103a only. Returns the SM count (> 0) or a
// negative status.
int device_sm_count(int* status) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        *status = NVFP4_MLA_ERR_CUDA;
        return -1;
    }
    if (dev >= 0 && dev < kMaxDevices) {
        const int cached = g_dev_state[dev].load(std::memory_order_relaxed);
        if (cached > 0) return cached;
        if (cached < 0) {
            *status = NVFP4_MLA_ERR_UNSUPPORTED;
            return -1;
        }
    }
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        *status = NVFP4_MLA_ERR_CUDA;
        return -1;
    }
    const bool ok = (major == 10 && minor == 3);
    if (dev >= 0 && dev < kMaxDevices) g_dev_state[dev].store(ok ? sms : -1, std::memory_order_relaxed);
    if (!ok) {
        *status = NVFP4_MLA_ERR_UNSUPPORTED;
        return -1;
    }
    return sms;
}

// 352, 432, 656 (fp8), or 352 with its scales in block order (NVFP4_MLA_SCALES_BLOCK_ORDER)
bool record_ok(int32_t r) {
    return r == 352 || r == 432 || r == 656 || r == (352 | NVFP4_MLA_SCALES_BLOCK_ORDER);
}
int record_width(int32_t r) { return r & 0xFFFF; }
bool block_scales(int32_t r) { return (r & NVFP4_MLA_SCALES_BLOCK_ORDER) != 0; }

// One CTA per SM: aim for one full wave. The 64-head decode of NVFP4 records runs one CTA per
// (row, split), the other decodes two; the NVFP4 decodes take keys in tiles of 128, the fp8 one 64.
int auto_splits(int64_t rows, int32_t topk, int sm_count, int32_t h_q, int32_t record_bytes) {
    const int r = record_width(record_bytes);
    const bool nvfp4 = r == 352 || r == 432;
    const int64_t ctas_per_split = rows * (nvfp4 && h_q == 64 ? 1 : 2);
    const int tile = nvfp4 ? 2 * kDecodeTile : kDecodeTile;
    int64_t s = ctas_per_split >= sm_count ? 1 : sm_count / ctas_per_split;
    const int64_t max_by_keys = (topk + tile - 1) / tile;
    if (s > max_by_keys) s = max_by_keys;
    if (s > kMaxSplits) s = kMaxSplits;
    if (s < 1) s = 1;
    return static_cast<int>(s);
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace (splits > 1): f16 partial outputs [rows, splits, h_q, 512], then the fp32 partial
// log2-sum-exps [rows, splits, h_q].
size_t workspace_for(int64_t rows, int32_t h_q, int splits) {
    if (splits <= 1) return 0;
    const size_t n = static_cast<size_t>(rows) * splits * h_q;
    return n * 512 * sizeof(uint16_t) + round256(n * sizeof(float));
}

int check_decode_shape(int32_t batch, int32_t s_q, int32_t h_q, int32_t topk, int32_t record_bytes,
                       int32_t num_splits) {
    if (batch < 0 || s_q < 0 || topk < 1 || num_splits < 0 || num_splits > kMaxSplits) return NVFP4_MLA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(batch) * s_q > (int64_t(1) << 31) / (2 * kMaxSplits)) return NVFP4_MLA_ERR_INVALID_ARG;
    if (!record_ok(record_bytes) || (h_q != 64 && h_q != 128)) return NVFP4_MLA_ERR_UNSUPPORTED;
    return NVFP4_MLA_OK;
}

// log2 of a page size, -1 for one that is not allowed
int page_shift_of(int32_t page_size) {
    if (page_size < 1 || page_size > 4096 || (page_size & (page_size - 1)) != 0) return -1;
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

// The sizes shared by the calls on sequences in pages.
int check_pages(int32_t batch, int32_t max_pages, int64_t num_pages, int32_t page_size, int64_t table_stride) {
    if (page_shift_of(page_size) < 0 || batch < 0 || max_pages < 0 || num_pages < 0 || num_pages > 0x7FFFFFFF) return NVFP4_MLA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(batch) * max_pages > 0x7FFFFFFF || static_cast<int64_t>(max_pages) * page_size > 0x7FFFFFFF ||
        num_pages * page_size > 0x7FFFFFFF)
        return NVFP4_MLA_ERR_INVALID_ARG;
    return table_stride < max_pages ? NVFP4_MLA_ERR_INVALID_ARG : NVFP4_MLA_OK;
}

int check_caches(uint8_t* const* caches, int32_t num_caches, int32_t record_bytes) {
    if (!record_ok(record_bytes)) return NVFP4_MLA_ERR_UNSUPPORTED;
    if (num_caches < 0 || num_caches > nvfp4mla::kMaxCaches || (num_caches > 0 && !caches)) return NVFP4_MLA_ERR_INVALID_ARG;
    for (int i = 0; i < num_caches; ++i)
        if (!caches[i] || !aligned(caches[i], 16)) return NVFP4_MLA_ERR_INVALID_ARG;
    return NVFP4_MLA_OK;
}

// Sizes of the calls around the latent attention: rows and heads.
int check_heads(int64_t rows, int32_t h_q) {
    if (rows < 0 || rows > 0x7FFFF000) return NVFP4_MLA_ERR_INVALID_ARG;
    return h_q < 1 || h_q > 128 ? NVFP4_MLA_ERR_UNSUPPORTED : NVFP4_MLA_OK;
}

// Whether TMA can read bf16 [outer, mid, inner] with these strides (elements): a 16-byte aligned base, strides that are multiples
// of 16 bytes. The stride of a dimension of one entry is never used and may be anything.
bool strides_ok(const void* base, int64_t outer, int64_t mid, int64_t inner, int64_t* outer_stride, int64_t* mid_stride) {
    if (outer == 1) *outer_stride = inner;
    if (mid == 1) *mid_stride = inner;
    for (const int64_t s : {*outer_stride, *mid_stride})
        if (s < 8 || s % 8 != 0 || s >= (int64_t(1) << 38)) return false;
    return base != nullptr && aligned(base, 16);
}

// Workspaces of the page calls, in 32-bit words. Resize: the free pages it hands out, four words per
// sequence. Fork: a staged row and a length per pair. Compact: movers, their counts and holes.
size_t resize_words(int32_t batch, int64_t num_pages) { return static_cast<size_t>(num_pages) + 4 * static_cast<size_t>(batch); }
size_t fork_words(int32_t max_pages, int32_t num_pairs) { return static_cast<size_t>(num_pairs) * (static_cast<size_t>(max_pages) + 1); }
size_t compact_words(int64_t num_pages) { return 3 * static_cast<size_t>(num_pages / 2) + 1; }

int check_workspace(const void* workspace, size_t bytes, size_t need) {
    return workspace && bytes >= need && aligned(workspace, 256) ? NVFP4_MLA_OK : NVFP4_MLA_ERR_WORKSPACE;
}

int check_paged_shape(int32_t batch, int32_t s_q, int32_t h_q) {
    if (batch < 0 || s_q < 0) return NVFP4_MLA_ERR_INVALID_ARG;
    if (h_q < 1 || h_q > 128) return NVFP4_MLA_ERR_UNSUPPORTED;
    // query rows are counted in 31 bits
    return static_cast<int64_t>(batch) * s_q > 0x7FFFFFFF / 128 ? NVFP4_MLA_ERR_INVALID_ARG : NVFP4_MLA_OK;
}

}  // namespace

namespace nvfp4mla {

int check_decode_call(const void* q, const uint8_t* cache, int64_t num_slots, int32_t record_bytes,
                      const int32_t* indices, int32_t batch, int32_t s_q, int32_t h_q, int32_t topk,
                      const float* attn_sink, const void* out, const float* lse, int32_t num_splits, int64_t* rows,
                      int* sms) {
    *rows = 0;
    *sms = 0;
    const int st = check_decode_shape(batch, s_q, h_q, topk, record_bytes, num_splits);
    if (st != NVFP4_MLA_OK) return st;
    if (num_slots < 0) return NVFP4_MLA_ERR_INVALID_ARG;
    *rows = static_cast<int64_t>(batch) * s_q;
    if (*rows == 0) return NVFP4_MLA_OK;
    if (!q || !cache || !indices || !out || !lse) return NVFP4_MLA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(indices, 4) || !aligned(lse, 4))
        return NVFP4_MLA_ERR_INVALID_ARG;
    if (attn_sink && !aligned(attn_sink, 4)) return NVFP4_MLA_ERR_INVALID_ARG;
    int status = NVFP4_MLA_OK;
    *sms = device_sm_count(&status);
    return *sms > 0 ? NVFP4_MLA_OK : status;
}

}  // namespace nvfp4mla

extern "C" {

NVFP4_MLA_API int nvfp4_mla_quantize_append(const void* kv_latent, int64_t latent_row_stride, const void* k_rope,
                                            int64_t rope_row_stride, const int64_t* slot_mapping,
                                            int64_t num_tokens, uint8_t* cache, int64_t num_slots,
                                            int32_t record_bytes, uint32_t* dev_status, void* stream) {
    if (!record_ok(record_bytes)) return NVFP4_MLA_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_slots < 0) return NVFP4_MLA_ERR_INVALID_ARG;
    if (num_tokens == 0) return NVFP4_MLA_OK;
    if (!kv_latent || !k_rope || !slot_mapping || !cache) return NVFP4_MLA_ERR_INVALID_ARG;
    if (!aligned(kv_latent, 16) || !aligned(k_rope, 16) || !aligned(cache, 16) || !aligned(slot_mapping, 8))
        return NVFP4_MLA_ERR_INVALID_ARG;
    if (latent_row_stride < 512 || latent_row_stride % 8 != 0) return NVFP4_MLA_ERR_INVALID_ARG;
    if (rope_row_stride < 64 || rope_row_stride % 8 != 0) return NVFP4_MLA_ERR_INVALID_ARG;
    int status = NVFP4_MLA_OK;
    const int sms = device_sm_count(&status);
    if (sms <= 0) return status;
    const cudaError_t e = nvfp4mla::launch_quantize_append(kv_latent, latent_row_stride, k_rope, rope_row_stride,
                                                           slot_mapping, num_tokens, cache, num_slots,
                                                           record_width(record_bytes), block_scales(record_bytes),
                                                           dev_status, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_mla_norm_rope_quantize_append(const void* kv_latent, int64_t latent_row_stride,
                                                      const void* norm_weight, float eps, const void* k_pe,
                                                      int64_t rope_row_stride, const int64_t* positions,
                                                      const float* cos_table, const float* sin_table,
                                                      int64_t num_positions, int32_t rotate_half,
                                                      const int64_t* slot_mapping, int64_t num_tokens,
                                                      uint8_t* cache, int64_t num_slots, int32_t record_bytes,
                                                      uint32_t* dev_status, void* stream) {
    if (!record_ok(record_bytes)) return NVFP4_MLA_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_slots < 0 || num_positions < 0 || !(eps >= 0.0f) || (rotate_half != 0 && rotate_half != 1))
        return NVFP4_MLA_ERR_INVALID_ARG;
    if (num_tokens == 0) return NVFP4_MLA_OK;
    if (!kv_latent || !k_pe || !slot_mapping || !cache || !norm_weight || !positions || !cos_table || !sin_table)
        return NVFP4_MLA_ERR_INVALID_ARG;
    if (!aligned(kv_latent, 16) || !aligned(k_pe, 16) || !aligned(cache, 16) || !aligned(slot_mapping, 8) ||
        !aligned(norm_weight, 16) || !aligned(positions, 8) || !aligned(cos_table, 8) || !aligned(sin_table, 8))
        return NVFP4_MLA_ERR_INVALID_ARG;
    if (latent_row_stride < 512 || latent_row_stride % 8 != 0) return NVFP4_MLA_ERR_INVALID_ARG;
    if (rope_row_stride < 64 || rope_row_stride % 8 != 0) return NVFP4_MLA_ERR_INVALID_ARG;
    int status = NVFP4_MLA_OK;
    const int sms = device_sm_count(&status);
    if (sms <= 0) return status;
    nvfp4mla::ProducerArgs pr;
    pr.norm_weight = static_cast<const uint16_t*>(norm_weight);
    pr.eps = eps;
    pr.positions = positions;
    pr.cos_table = cos_table;
    pr.sin_table = sin_table;
    pr.num_positions = num_positions;
    pr.rotate_half = rotate_half;
    const cudaError_t e = nvfp4mla::launch_quantize_append(kv_latent, latent_row_stride, k_pe, rope_row_stride,
                                                           slot_mapping, num_tokens, cache, num_slots,
                                                           record_width(record_bytes), block_scales(record_bytes),
                                                           dev_status, sms, static_cast<cudaStream_t>(stream), &pr);
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_sparse_mla_decode_workspace_size(int32_t batch, int32_t s_q, int32_t h_q, int32_t topk,
                                                         int32_t record_bytes, int32_t num_splits, size_t* bytes) {
    if (!bytes) return NVFP4_MLA_ERR_INVALID_ARG;
    const int st = check_decode_shape(batch, s_q, h_q, topk, record_bytes, num_splits);
    if (st != NVFP4_MLA_OK) return st;
    const int64_t rows = static_cast<int64_t>(batch) * s_q;
    int splits = num_splits;
    if (splits == 0) {
        int status = NVFP4_MLA_OK;
        const int sms = device_sm_count(&status);
        if (sms <= 0) return status;
        splits = auto_splits(rows, topk, sms, h_q, record_bytes);
    }
    *bytes = workspace_for(rows, h_q, splits);
    return NVFP4_MLA_OK;
}

NVFP4_MLA_API int nvfp4_sparse_mla_decode_plan(int32_t batch, int32_t s_q, int32_t h_q, int32_t topk,
                                               int32_t record_bytes, int32_t num_splits, int32_t* splits,
                                               int32_t* kernels) {
    if (!splits || !kernels) return NVFP4_MLA_ERR_INVALID_ARG;
    const int st = check_decode_shape(batch, s_q, h_q, topk, record_bytes, num_splits);
    if (st != NVFP4_MLA_OK) return st;
    const int64_t rows = static_cast<int64_t>(batch) * s_q;
    int status = NVFP4_MLA_OK;
    const int sms = device_sm_count(&status);
    if (sms <= 0) return status;
    const int sp = num_splits > 0 ? num_splits : auto_splits(rows, topk, sms, h_q, record_bytes);
    nvfp4mla::DecodeArgs d;
    d.record_bytes = record_width(record_bytes);
    d.block_scales = block_scales(record_bytes);
    d.rows = static_cast<int>(rows);
    d.h_q = h_q;
    d.topk = topk;
    d.splits = sp;
    *splits = sp;
    *kernels = rows == 0 ? 0 : (sp == 1 || nvfp4mla::decode_pair_merges(d)) ? 1 : 2;
    return NVFP4_MLA_OK;
}

NVFP4_MLA_API int nvfp4_sparse_mla_decode(const void* q, const uint8_t* cache, int64_t num_slots, int32_t record_bytes,
                                          const int32_t* indices, int32_t batch, int32_t s_q, int32_t h_q,
                                          int32_t topk, float sm_scale, const float* attn_sink, void* out, float* lse,
                                          int32_t num_splits, void* workspace, size_t workspace_bytes,
                                          uint32_t* dev_status, void* stream) {
    int64_t rows = 0;
    int sms = 0;
    const int st = nvfp4mla::check_decode_call(q, cache, num_slots, record_bytes, indices, batch, s_q, h_q, topk,
                                               attn_sink, out, lse, num_splits, &rows, &sms);
    if (st != NVFP4_MLA_OK || rows == 0) return st;
    const int splits = num_splits > 0 ? num_splits : auto_splits(rows, topk, sms, h_q, record_bytes);
    const size_t need = workspace_for(rows, h_q, splits);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return NVFP4_MLA_ERR_WORKSPACE;

    nvfp4mla::DecodeArgs d;
    d.q = q;
    d.cache = cache;
    d.num_slots = num_slots;
    d.record_bytes = record_width(record_bytes);
    d.block_scales = block_scales(record_bytes);
    d.indices = indices;
    d.rows = static_cast<int>(rows);
    d.h_q = h_q;
    d.topk = topk;
    d.sm_scale = sm_scale;
    d.attn_sink = attn_sink;
    d.out = out;
    d.lse = lse;
    d.splits = splits;
    const size_t n_part = static_cast<size_t>(rows) * splits * h_q;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    d.part_out = need ? reinterpret_cast<uint16_t*>(ws) : nullptr;
    d.part_lse = need ? reinterpret_cast<float*>(ws + n_part * 512 * sizeof(uint16_t)) : nullptr;
    d.dev_status = dev_status;
    const cudaError_t e = nvfp4mla::launch_sparse_decode(d, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_paged_mla_decode_workspace_size(int32_t batch, int32_t s_q, int32_t h_q, size_t* bytes) {
    if (!bytes) return NVFP4_MLA_ERR_INVALID_ARG;
    const int st = check_paged_shape(batch, s_q, h_q);
    if (st != NVFP4_MLA_OK) return st;
    *bytes = batch == 0 || s_q == 0 ? 0 : nvfp4mla::paged_workspace_bytes(batch, static_cast<int64_t>(s_q) * h_q);
    return NVFP4_MLA_OK;
}

NVFP4_MLA_API int nvfp4_paged_mla_decode(const void* q, const uint8_t* cache, int64_t num_pages, int32_t page_size,
                                         int32_t record_bytes, const int32_t* page_table, int64_t table_stride,
                                         int32_t max_pages, const int32_t* seq_lens, int32_t batch, int32_t s_q,
                                         int32_t h_q, float sm_scale, const float* attn_sink, void* out, float* lse,
                                         void* workspace, size_t workspace_bytes, uint32_t* dev_status, void* stream) {
    int st = check_paged_shape(batch, s_q, h_q);
    if (st != NVFP4_MLA_OK) return st;
    if (!record_ok(record_bytes) || record_width(record_bytes) == 656) return NVFP4_MLA_ERR_UNSUPPORTED;
    st = check_pages(batch, max_pages, num_pages, page_size, table_stride);
    if (st != NVFP4_MLA_OK) return st;
    if (batch == 0 || s_q == 0) return NVFP4_MLA_OK;
    // a table without columns (or a pool without pages) has nothing to read: its pointer may be null
    if (!q || !seq_lens || !out || !lse || (max_pages > 0 && !page_table) || (num_pages > 0 && !cache)) return NVFP4_MLA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(lse, 4) || !aligned(attn_sink, 4))
        return NVFP4_MLA_ERR_INVALID_ARG;
    const int64_t rows_per_seq = static_cast<int64_t>(s_q) * h_q;
    st = check_workspace(workspace, workspace_bytes, nvfp4mla::paged_workspace_bytes(batch, rows_per_seq));
    if (st != NVFP4_MLA_OK) return st;
    const int sms = device_sm_count(&st);
    if (sms <= 0) return st;
    nvfp4mla::PagedDecodeArgs d;
    d.q = q;
    d.cache = cache;
    d.record_bytes = record_width(record_bytes);
    d.block_scales = block_scales(record_bytes);
    d.jobs.page_table = page_table;
    d.jobs.table_stride = table_stride;
    d.jobs.seq_lens = seq_lens;
    d.jobs.num_pages = static_cast<int>(num_pages);
    d.jobs.page_shift = page_shift_of(page_size);
    d.jobs.capacity = max_pages << d.jobs.page_shift;
    d.jobs.batch = batch;
    d.jobs.s_q = s_q;
    d.jobs.h_q = h_q;
    d.jobs.rows_per_seq = static_cast<int>(rows_per_seq);
    d.jobs.row_tiles = 0;
    d.sm_scale = sm_scale;
    d.attn_sink = attn_sink;
    d.out = out;
    d.lse = lse;
    d.dev_status = dev_status;
    const cudaError_t e = nvfp4mla::launch_paged_decode(d, workspace, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_mla_pages_workspace_size(int32_t batch, int32_t max_pages, int64_t num_pages,
                                                 int32_t num_pairs, size_t* bytes) {
    if (!bytes || num_pairs < 0) return NVFP4_MLA_ERR_INVALID_ARG;
    const int st = check_pages(batch, max_pages, num_pages, 1, max_pages);
    if (st != NVFP4_MLA_OK) return st;
    size_t words = resize_words(batch, num_pages);
    if (fork_words(max_pages, num_pairs) > words) words = fork_words(max_pages, num_pairs);
    if (compact_words(num_pages) > words) words = compact_words(num_pages);
    *bytes = round256(4 * words);
    return NVFP4_MLA_OK;
}

NVFP4_MLA_API int nvfp4_mla_copy_pages(uint8_t* const* caches, int32_t num_caches, int64_t num_pages,
                                       int32_t page_size, int32_t record_bytes, const int32_t* src,
                                       const int32_t* dst, int32_t n, uint32_t* dev_status, void* stream) {
    int st = check_pages(0, 0, num_pages, page_size, 0);
    if (st == NVFP4_MLA_OK) st = check_caches(caches, num_caches, record_bytes);
    if (st != NVFP4_MLA_OK) return st;
    if (n < 0 || num_caches < 1) return NVFP4_MLA_ERR_INVALID_ARG;
    if (n == 0) return NVFP4_MLA_OK;
    if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return NVFP4_MLA_ERR_INVALID_ARG;
    const int sms = device_sm_count(&st);
    if (sms <= 0) return st;
    const nvfp4mla::PoolArgs pool = {caches, num_caches, static_cast<int>(num_pages), page_shift_of(page_size), record_width(record_bytes)};
    const cudaError_t e = nvfp4mla::launch_copy_pages(pool, src, dst, n, dev_status, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_mla_fork_sequences(int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                           int32_t* seq_lens, int32_t batch, int32_t* page_refs, int64_t num_pages,
                                           int32_t page_size, const int32_t* src, const int32_t* dst,
                                           int32_t num_pairs, void* workspace, size_t workspace_bytes,
                                           uint32_t* dev_status, void* stream) {
    int st = check_pages(batch, max_pages, num_pages, page_size, table_stride);
    if (st != NVFP4_MLA_OK) return st;
    if (num_pairs < 0) return NVFP4_MLA_ERR_INVALID_ARG;
    if (num_pairs == 0) return NVFP4_MLA_OK;
    if (!seq_lens || !src || !dst || (max_pages > 0 && !page_table) || (num_pages > 0 && !page_refs)) return NVFP4_MLA_ERR_INVALID_ARG;
    if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(page_refs, 16))
        return NVFP4_MLA_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, round256(4 * fork_words(max_pages, num_pairs)));
    if (st != NVFP4_MLA_OK) return st;
    if (device_sm_count(&st) <= 0) return st;
    nvfp4mla::ForkArgs a;
    a.page_table = page_table;
    a.table_stride = table_stride;
    a.width = max_pages;
    a.shift = page_shift_of(page_size);
    a.seq_lens = seq_lens;
    a.batch = batch;
    a.page_refs = page_refs;
    a.num_pages = static_cast<int>(num_pages);
    a.src = src;
    a.dst = dst;
    a.pairs = num_pairs;
    a.stage = static_cast<int32_t*>(workspace);
    a.status = dev_status;
    const cudaError_t e = nvfp4mla::launch_fork(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_mla_resize_sequences(int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                             int32_t* seq_lens, const int32_t* new_lens, int32_t batch,
                                             int32_t* page_refs, int64_t num_pages, int32_t page_size,
                                             uint8_t* const* caches, int32_t num_caches, int32_t record_bytes,
                                             int64_t* slots, int32_t max_new, void* workspace,
                                             size_t workspace_bytes, uint32_t* dev_status, void* stream) {
    int st = check_pages(batch, max_pages, num_pages, page_size, table_stride);
    if (st == NVFP4_MLA_OK) st = check_caches(caches, num_caches, record_bytes);
    if (st != NVFP4_MLA_OK) return st;
    if (max_new < 0) return NVFP4_MLA_ERR_INVALID_ARG;
    if (batch == 0) return NVFP4_MLA_OK;
    if (!seq_lens || !new_lens || (max_pages > 0 && !page_table) || (num_pages > 0 && !page_refs) || (max_new > 0 && !slots))
        return NVFP4_MLA_ERR_INVALID_ARG;
    if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(page_refs, 16) || !aligned(slots, 8))
        return NVFP4_MLA_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, round256(4 * resize_words(batch, num_pages)));
    if (st != NVFP4_MLA_OK) return st;
    const int sms = device_sm_count(&st);
    if (sms <= 0) return st;
    nvfp4mla::ResizeArgs a;
    a.page_table = page_table;
    a.table_stride = table_stride;
    a.width = max_pages;
    a.shift = page_shift_of(page_size);
    a.seq_lens = seq_lens;
    a.new_lens = new_lens;
    a.batch = batch;
    a.page_refs = page_refs;
    a.num_pages = static_cast<int>(num_pages);
    a.slots = slots;
    a.max_new = max_new;
    int32_t* w = static_cast<int32_t*>(workspace);
    a.offset = w;
    a.cow_src = w + batch;
    a.cow_dst = w + 2 * static_cast<int64_t>(batch);
    a.cow_records = w + 3 * static_cast<int64_t>(batch);
    a.free_list = w + 4 * static_cast<int64_t>(batch);
    a.status = dev_status;
    const nvfp4mla::PoolArgs pool = {caches, num_caches, a.num_pages, a.shift, record_width(record_bytes)};
    const cudaError_t e = nvfp4mla::launch_resize(a, pool, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_mla_compact_pages(uint8_t* const* caches, int32_t num_caches, int32_t record_bytes,
                                          const int32_t* page_table, int64_t table_stride, int32_t* table_out,
                                          int64_t table_out_stride, int32_t max_pages, const int32_t* seq_lens,
                                          int32_t batch, const int32_t* page_refs, int32_t* refs_out,
                                          int64_t num_pages, int32_t page_size, int32_t* page_map, int32_t* live,
                                          void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                          void* stream) {
    int st = check_pages(batch, max_pages, num_pages, page_size, table_stride);
    if (st == NVFP4_MLA_OK) st = check_caches(caches, num_caches, record_bytes);
    if (st != NVFP4_MLA_OK) return st;
    if (table_out_stride < max_pages || !live || !aligned(live, 4)) return NVFP4_MLA_ERR_INVALID_ARG;
    // in place, the old and the new table are the same rows
    if (page_table == table_out && table_stride != table_out_stride) return NVFP4_MLA_ERR_INVALID_ARG;
    if (num_pages > 0 && (!page_refs || !refs_out || !page_map)) return NVFP4_MLA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(batch) * max_pages > 0 && (!page_table || !table_out || !seq_lens)) return NVFP4_MLA_ERR_INVALID_ARG;
    if (!aligned(page_table, 4) || !aligned(table_out, 4) || !aligned(seq_lens, 4) || !aligned(page_map, 4) ||
        !aligned(page_refs, 16) || !aligned(refs_out, 16))
        return NVFP4_MLA_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, round256(4 * compact_words(num_pages)));
    if (st != NVFP4_MLA_OK) return st;
    const int sms = device_sm_count(&st);
    if (sms <= 0) return st;
    nvfp4mla::CompactArgs a;
    a.page_table = page_table;
    a.table_stride = table_stride;
    a.table_out = table_out;
    a.table_out_stride = table_out_stride;
    a.width = max_pages;
    a.shift = page_shift_of(page_size);
    a.seq_lens = seq_lens;
    a.batch = batch;
    a.page_refs = page_refs;
    a.refs_out = refs_out;
    a.num_pages = static_cast<int>(num_pages);
    a.page_map = page_map;
    a.live = live;
    int32_t* w = static_cast<int32_t*>(workspace);
    const int64_t half = num_pages / 2;
    a.moves = w;
    a.mover = w + 1;
    a.mover_refs = a.mover + half;
    a.hole = a.mover_refs + half;
    a.status = dev_status;
    const nvfp4mla::PoolArgs pool = {caches, num_caches, a.num_pages, a.shift, record_width(record_bytes)};
    const cudaError_t e = nvfp4mla::launch_compact(a, pool, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_mla_absorb_query(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* kv_b,
                                         int64_t kv_b_row_stride, int64_t kv_b_head_stride, const int64_t* positions,
                                         const float* cos_table, const float* sin_table, int64_t num_positions,
                                         int32_t rotate_half, int64_t num_tokens, int32_t h_q, void* out,
                                         uint32_t* dev_status, void* stream) {
    int st = check_heads(num_tokens, h_q);
    if (st != NVFP4_MLA_OK) return st;
    if (num_positions < 0 || (rotate_half != 0 && rotate_half != 1)) return NVFP4_MLA_ERR_INVALID_ARG;
    if (num_tokens == 0) return NVFP4_MLA_OK;
    if (!strides_ok(q, num_tokens, h_q, 192, &q_token_stride, &q_head_stride) || !strides_ok(kv_b, h_q, 256, 512, &kv_b_head_stride, &kv_b_row_stride))
        return NVFP4_MLA_ERR_INVALID_ARG;
    if (!out || !aligned(out, 32) || !aligned(positions, 8) || !aligned(cos_table, 16) || !aligned(sin_table, 16)) return NVFP4_MLA_ERR_INVALID_ARG;
    if (positions && (!cos_table || !sin_table)) return NVFP4_MLA_ERR_INVALID_ARG;
    const int sms = device_sm_count(&st);
    if (sms <= 0) return st;
    nvfp4mla::HeadProductArgs p = {};
    p.in = q;
    p.in_token_stride = q_token_stride;
    p.in_head_stride = q_head_stride;
    p.tokens = num_tokens;
    p.heads = h_q;
    p.kv_b = kv_b;
    p.w_row_stride = kv_b_row_stride;
    p.w_head_stride = kv_b_head_stride;
    p.positions = positions;
    p.cos_table = cos_table;
    p.sin_table = sin_table;
    p.num_positions = num_positions;
    p.rotate_half = rotate_half;
    p.out = out;
    p.status = dev_status;
    const cudaError_t e = nvfp4mla::launch_head_product(p, true, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_mla_project_values(const void* latent, int64_t latent_token_stride, int64_t latent_head_stride,
                                           const void* kv_b, int64_t kv_b_row_stride, int64_t kv_b_head_stride,
                                           int64_t num_tokens, int32_t h_q, void* out, uint32_t* dev_status, void* stream) {
    int st = check_heads(num_tokens, h_q);
    if (st != NVFP4_MLA_OK) return st;
    if (num_tokens == 0) return NVFP4_MLA_OK;
    if (!strides_ok(latent, num_tokens, h_q, 512, &latent_token_stride, &latent_head_stride) ||
        !strides_ok(kv_b, h_q, 256, 512, &kv_b_head_stride, &kv_b_row_stride) || !out || !aligned(out, 32))
        return NVFP4_MLA_ERR_INVALID_ARG;
    const int sms = device_sm_count(&st);
    if (sms <= 0) return st;
    nvfp4mla::HeadProductArgs p = {};
    p.in = latent;
    p.in_token_stride = latent_token_stride;
    p.in_head_stride = latent_head_stride;
    p.tokens = num_tokens;
    p.heads = h_q;
    p.kv_b = kv_b;
    p.w_row_stride = kv_b_row_stride;
    p.w_head_stride = kv_b_head_stride;
    p.out = out;
    p.status = dev_status;
    const cudaError_t e = nvfp4mla::launch_head_product(p, false, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_paged_mla_expand(const uint8_t* cache, int64_t num_pages, int32_t page_size, int32_t record_bytes,
                                         const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                         const int32_t* cu_seqlens, int32_t batch, const void* kv_b, int64_t kv_b_row_stride,
                                         int64_t kv_b_head_stride, int32_t h_q, void* kv, void* k_pe, int64_t num_rows,
                                         uint32_t* dev_status, void* stream) {
    int st = check_pages(batch, max_pages, num_pages, page_size, table_stride);
    if (st == NVFP4_MLA_OK) st = check_heads(num_rows, h_q);
    if (st != NVFP4_MLA_OK) return st;
    if (!record_ok(record_bytes) || record_width(record_bytes) == 656) return NVFP4_MLA_ERR_UNSUPPORTED;
    if (batch == 0 || num_rows == 0) return NVFP4_MLA_OK;
    if (!cu_seqlens || !kv || !k_pe || (max_pages > 0 && !page_table) || (num_pages > 0 && !cache)) return NVFP4_MLA_ERR_INVALID_ARG;
    if (!aligned(cache, 16) || !aligned(page_table, 4) || !aligned(cu_seqlens, 4) || !aligned(kv, 32) || !aligned(k_pe, 16))
        return NVFP4_MLA_ERR_INVALID_ARG;
    if (!strides_ok(kv_b, h_q, 256, 512, &kv_b_head_stride, &kv_b_row_stride)) return NVFP4_MLA_ERR_INVALID_ARG;
    const int sms = device_sm_count(&st);
    if (sms <= 0) return st;
    nvfp4mla::ExpandArgs p = {};
    p.cache = cache;
    p.num_pages = static_cast<int>(num_pages);
    p.page_shift = page_shift_of(page_size);
    p.record_bytes = record_width(record_bytes);
    p.block_scales = block_scales(record_bytes);
    p.page_table = page_table;
    p.table_stride = table_stride;
    p.width = max_pages;
    p.starts = cu_seqlens;
    p.batch = batch;
    p.kv_b = kv_b;
    p.w_row_stride = kv_b_row_stride;
    p.w_head_stride = kv_b_head_stride;
    p.heads = h_q;
    p.rows = num_rows;
    p.kv = kv;
    p.k_pe = k_pe;
    p.status = dev_status;
    const cudaError_t e = nvfp4mla::launch_paged_expand(p, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_ragged_mla_attention_workspace_size(size_t* bytes) {
    if (!bytes) return NVFP4_MLA_ERR_INVALID_ARG;
    *bytes = round256(nvfp4mla::ragged_workspace_bytes());
    return NVFP4_MLA_OK;
}

NVFP4_MLA_API int nvfp4_ragged_mla_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t num_q,
                                             const void* kv, int64_t kv_token_stride, int64_t kv_head_stride, const void* k_pe,
                                             int64_t k_pe_stride, int64_t num_k, const int32_t* cu_seqlens_q,
                                             const int32_t* cu_seqlens_k, int32_t batch, int32_t h_q, float sm_scale,
                                             const float* attn_sink, void* out, float* lse, void* workspace,
                                             size_t workspace_bytes, uint32_t* dev_status, void* stream) {
    int st = check_heads(num_q, h_q);
    if (st == NVFP4_MLA_OK) st = check_heads(num_k, h_q);
    if (st != NVFP4_MLA_OK) return st;
    // (a tile's keys, and the lengths of the batch, have to be through within the second that a wait may take)
    if (batch < 0 || batch > (1 << 20) || num_k >= (int64_t(1) << 26)) return NVFP4_MLA_ERR_INVALID_ARG;
    if (batch == 0 || num_q == 0) return NVFP4_MLA_OK;
    if (!cu_seqlens_q || !cu_seqlens_k || !out || !lse) return NVFP4_MLA_ERR_INVALID_ARG;
    if (!aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4) || !aligned(attn_sink, 4) || !aligned(out, 32) || !aligned(lse, 4))
        return NVFP4_MLA_ERR_INVALID_ARG;
    if (!strides_ok(q, num_q, h_q, 192, &q_token_stride, &q_head_stride)) return NVFP4_MLA_ERR_INVALID_ARG;
    if (num_k == 0) {   // nothing is read of them: any address that TMA accepts
        kv = k_pe = q;
        kv_token_stride = kv_head_stride = 256;
        k_pe_stride = 64;
    }
    int64_t one = 1;
    if (!strides_ok(kv, num_k, h_q, 256, &kv_token_stride, &kv_head_stride) || !strides_ok(k_pe, num_k, 1, 64, &k_pe_stride, &one))
        return NVFP4_MLA_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, round256(nvfp4mla::ragged_workspace_bytes()));
    if (st != NVFP4_MLA_OK) return st;
    const int sms = device_sm_count(&st);
    if (sms <= 0) return st;
    nvfp4mla::RaggedArgs p = {};
    p.q = q;
    p.q_token_stride = q_token_stride;
    p.q_head_stride = q_head_stride;
    p.rows_q = num_q;
    p.kv = kv;
    p.kv_token_stride = kv_token_stride;
    p.kv_head_stride = kv_head_stride;
    p.k_pe = k_pe;
    p.pe_stride = k_pe_stride;
    p.rows_k = num_k;
    p.starts_q = cu_seqlens_q;
    p.starts_k = cu_seqlens_k;
    p.batch = batch;
    p.heads = h_q;
    p.sm_scale = sm_scale;
    p.attn_sink = attn_sink;
    p.out = out;
    p.lse = lse;
    p.status = dev_status;
    const cudaError_t e = nvfp4mla::launch_ragged_attention(p, workspace, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API int nvfp4_mla_selftest_wait_timeout(uint32_t* dev_status, uint64_t* elapsed_ns, void* stream) {
    if (!dev_status || !elapsed_ns || !aligned(elapsed_ns, 8)) return NVFP4_MLA_ERR_INVALID_ARG;
    int status = NVFP4_MLA_OK;
    if (device_sm_count(&status) <= 0) return status;
    const cudaError_t e =
        nvfp4mla::launch_wait_timeout_probe(dev_status, elapsed_ns, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NVFP4_MLA_OK : NVFP4_MLA_ERR_CUDA;
}

NVFP4_MLA_API const char* nvfp4_mla_status_string(int status) {
    switch (status) {
        case NVFP4_MLA_OK: return "ok";
        case NVFP4_MLA_ERR_INVALID_ARG: return "invalid argument (null pointer, size, stride or alignment)";
        case NVFP4_MLA_ERR_UNSUPPORTED: return "unsupported (record width, head count, or device is not sm_103)";
        case NVFP4_MLA_ERR_CUDA: return "CUDA runtime error";
        case NVFP4_MLA_ERR_WORKSPACE: return "workspace missing, too small or not 256-byte aligned";
        default: return "unknown status";
    }
}

NVFP4_MLA_API int nvfp4_mla_version(void) { return 100; }

}  // extern "C"

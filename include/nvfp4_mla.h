/*
 * nvfp4_mla.h -- C ABI of the NVFP4 MLA KV-cache library for GB300 (sm_103a).
 *
 * Two operations, as the pages state the problem:
 *
 *  1. nvfp4_mla_quantize_append: quantize each token's 512-dim MLA latent (NoPE) and 64-dim
 *     RoPE key into one self-describing record and scatter it to its cache slot.
 *     - 352-byte "nvfp4.fp8rope" record: FlashMLA PR 18 "W4A16 DSA: NVFP4 KV cache format for
 *       SM100 sparse decode", format block "nvfp4.fp8rope (352 B/token)": bytes [0,256) hold
 *       512 e2m1 values two per byte, [256,320) 64 unscaled e4m3 RoPE values, [320,352) 32
 *       e4m3 scales, one per 16 values, the scale of block s at byte 320 + 8*(s&3) + (s>>2).
 *     - 432-byte "nvfp4_ds_mla" record: vLLM PR 82 "kv: nvfp4_ds_mla - 4-bit NVFP4 KV cache for
 *       B12X sparse MLA (SM120)", Problem and Fix / Write side: 256 B e2m1 NoPE, 32 B e4m3
 *       scales in block order, 16 zero bytes, 128 B bf16 RoPE copied verbatim.
 *     - Scale rule (vLLM PR 82, Tests): scale = E4M3(group_amax / 6); values are rounded to
 *       the nearest e2m1 grid point after division by the decoded scale.
 *     - 656-byte fp8 record, the one the NVFP4 records are measured against (vLLM PR 82,
 *       Problem: "512 B fp8 NoPE + 16 B fp32 tile scales + 128 B BF16 RoPE"): bytes [0,512)
 *       e4m3 NoPE codes, [512,528) four little-endian fp32 scales (scale t covers NoPE values
 *       [128t, 128t+128)), [528,656) bf16 RoPE copied verbatim. The page gives no fp8 scale
 *       rule; this library uses scale = amax / 448 and code = e4m3(x / scale) (fp32 quotients;
 *       a zero tile stores scale 0), and the decode's keys are bf16(e4m3 * scale). The decode
 *       takes V in f16, so NoPE magnitudes must stay below 65536 (the append flags larger
 *       ones with NVFP4_MLA_DEV_FP8_RANGE and stores them anyway).
 *
 *  (Attention over whole sequences through a page table, and operations on the pages, follow further
 *  down: nvfp4_paged_mla_decode, nvfp4_mla_copy_pages, nvfp4_mla_fork_sequences,
 *  nvfp4_mla_resize_sequences, nvfp4_mla_compact_pages. The pages have no counterpart to them.)
 *
 *  2. nvfp4_sparse_mla_decode: DeepSeek-style sparse MLA decode over one shared latent KV
 *     head: for each query row (b, i) and head h, the keys are the records its top-k index
 *     list selects (FlashMLA PR 18, "Kernel:" paragraph: keys dequantized to bf16, QK^T over
 *     576 = 512 NoPE + 64 RoPE dims, PV over the 512 NoPE dims, bf16 MMAs with fp32
 *     accumulation, attention sink and invalid indices per its validation list).
 *
 * Conventions shared by every call
 *  - All data pointers are DEVICE pointers unless stated; the caller owns every buffer.
 *    No call allocates device memory. The only device memory the library owns is the
 *    fixed scratch array of nvfp4_sparse_mla_decode_no_alloc (see there).
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream). Work is enqueued on it
 *    and the call returns without synchronizing. Stream order is kept as usual: every kernel
 *    of the library is launched as a programmatic dependent of the preceding work on the
 *    stream, so its prologue (for the decode: barrier setup, tensor-memory allocation) may
 *    overlap the preceding kernel's tail, but it reads and writes no memory before that kernel
 *    has completed and its writes are visible. The append and decode kernels let the next
 *    kernel on the stream start its prologue early in the same way; the decode's split merge
 *    does not (a waiting successor would hold the SMs the merge runs on).
 *  - Every argument check runs on the host before any launch; a failed check returns a
 *    status below and launches nothing. Kernels never trap: problems found on the device
 *    are OR-ed into *dev_status (if non-NULL) as NVFP4_MLA_DEV_* bits, readable after the
 *    stream has been synchronized.
 *  - The library is built for sm_103a only; calls on any other device return
 *    NVFP4_MLA_ERR_UNSUPPORTED.
 */
#ifndef NVFP4_MLA_H_
#define NVFP4_MLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define NVFP4_MLA_API __attribute__((visibility("default")))

/* Return codes of every call. */
typedef enum {
    NVFP4_MLA_OK = 0,
    NVFP4_MLA_ERR_INVALID_ARG = 1,   /* null pointer, bad size, stride or alignment      */
    NVFP4_MLA_ERR_UNSUPPORTED = 2,   /* record width, head count or device not supported */
    NVFP4_MLA_ERR_CUDA = 3,          /* a CUDA runtime call failed (launch, attribute)   */
    NVFP4_MLA_ERR_WORKSPACE = 4      /* workspace missing, too small or misaligned        */
} nvfp4_mla_status;

/*
 * Record layout. Every call's `record_bytes` is 352, 432 or 656, or
 * (352 | NVFP4_MLA_SCALES_BLOCK_ORDER): a 352-byte record equal to "nvfp4.fp8rope" except that its
 * 32 scales are stored in block order, block s at byte 320 + s. No page defines that record; it
 * is the unpermuted side of the scale-layout comparison (FlashMLA PR 18, format block, credits
 * the permuted placement with 10-12% of decode latency). A cache is read with the value it was
 * written with; its rows are (record_bytes & 0xFFFF) bytes wide. Any other value returns
 * NVFP4_MLA_ERR_UNSUPPORTED.
 */
#define NVFP4_MLA_SCALES_BLOCK_ORDER 0x10000

/* Bits the kernels OR into *dev_status. */
#define NVFP4_MLA_DEV_SLOT_OUT_OF_RANGE 0x1u  /* quantize_append: slot >= num_slots (skipped) */
#define NVFP4_MLA_DEV_INDEX_OUT_OF_RANGE 0x2u /* decode: index >= num_slots (masked); a page,
                                                 sequence or length outside its table          */
#define NVFP4_MLA_DEV_TIMEOUT 0x4u            /* decode: a pipeline wait gave up; out invalid */
#define NVFP4_MLA_DEV_FP8_RANGE 0x8u          /* quantize_append, 656 B: a NoPE |x| >= 65536  */
#define NVFP4_MLA_DEV_POSITION_OUT_OF_RANGE 0x10u /* norm_rope_quantize_append: position outside
                                                     [0, num_positions) (token skipped)         */
#define NVFP4_MLA_DEV_PAGES_EXHAUSTED 0x20u   /* resize_sequences: too few free pages (no sequence
                                                 grew; those that shrink did)                  */
#define NVFP4_MLA_DEV_LENGTH_OUT_OF_RANGE 0x40u /* resize_sequences: a new length below 0 or beyond
                                                   the page table (that sequence unchanged)    */

/*
 * Quantize-and-append (write side).
 *   kv_latent          bf16 [num_tokens, 512], row stride latent_row_stride ELEMENTS, inner
 *                      stride 1; base 16-byte aligned, latent_row_stride % 8 == 0.
 *   k_rope             bf16 [num_tokens, 64], its own row stride rope_row_stride ELEMENTS
 *                      (may differ from the latent's); base 16-byte aligned, stride % 8 == 0.
 *   slot_mapping       int64 [num_tokens]: record slot of each token. A negative slot skips
 *                      the token (padding); a slot >= num_slots is skipped and sets
 *                      NVFP4_MLA_DEV_SLOT_OUT_OF_RANGE. Slots should be distinct; if two tokens
 *                      share a slot, which record lands there is unspecified.
 *   cache              uint8 [num_slots, record_bytes & 0xFFFF], 16-byte aligned. Only the
 *                      slots named by slot_mapping are written; every other byte is untouched.
 *   record_bytes       352, 432 or 656, or 352 | NVFP4_MLA_SCALES_BLOCK_ORDER (see above).
 *   dev_status         nullable device uint32 (see NVFP4_MLA_DEV_*).
 * num_tokens == 0 is valid and launches nothing.
 */
NVFP4_MLA_API int nvfp4_mla_quantize_append(const void* kv_latent, int64_t latent_row_stride,
                                            const void* k_rope, int64_t rope_row_stride,
                                            const int64_t* slot_mapping, int64_t num_tokens,
                                            uint8_t* cache, int64_t num_slots, int32_t record_bytes,
                                            uint32_t* dev_status, void* stream);

/*
 * Fused producer: RMSNorm of the latent, rotary embedding of k_pe, quantize and append, in one
 * kernel. SGLang PR 38646 "[SM120] Add opt-in NVFP4 sparse-MLA KV cache format for
 * DeepSeek-V4", "Limitations": the NVFP4 path lacks the fused norm+rope+quantize+store kernel and
 * pays a bf16 intermediate plus a separate quantize kernel per layer; "Stores": the existing
 * fused store kernels emit only the fp8 layout. The pages fix none of the stages' parameters, so
 * they are arguments here:
 *   kv_latent          bf16 [num_tokens, 512] BEFORE the norm (layout as in quantize_append).
 *   norm_weight        bf16 [512], 16-byte aligned: y_i = norm_weight[i] * x_i /
 *                      sqrt(mean_j x_j^2 + eps).
 *   eps                the norm's epsilon (>= 0).
 *   k_pe               bf16 [num_tokens, 64] BEFORE the rotary embedding (layout as k_rope).
 *   positions          int64 [num_tokens], 8-byte aligned: each token's position p. A position
 *                      outside [0, num_positions) skips the token and sets
 *                      NVFP4_MLA_DEV_POSITION_OUT_OF_RANGE.
 *   cos_table,         fp32 [num_positions, 32] each, 8-byte aligned: cos and sin of frequency f
 *   sin_table          at position p. The pair (a, b) of frequency f becomes (a c - b s, b c + a s).
 *   rotate_half        1: the pair of frequency f is (k_pe[f], k_pe[f + 32]); 0: (k_pe[2f],
 *                      k_pe[2f + 1]) ("interleaved").
 *   slot_mapping, cache, num_slots, record_bytes, dev_status: as in quantize_append.
 * Both stages compute in fp32 and round each result once to bf16, the value an unfused path
 * stores in its bf16 intermediate; the records are then those quantize_append writes for these
 * bf16 values. A result within about 2^-19 (relative to its terms) of a bf16 rounding midpoint may
 * round to either neighbour. num_tokens == 0 is valid and launches nothing.
 */
NVFP4_MLA_API int nvfp4_mla_norm_rope_quantize_append(const void* kv_latent, int64_t latent_row_stride,
                                                      const void* norm_weight, float eps, const void* k_pe,
                                                      int64_t rope_row_stride, const int64_t* positions,
                                                      const float* cos_table, const float* sin_table,
                                                      int64_t num_positions, int32_t rotate_half,
                                                      const int64_t* slot_mapping, int64_t num_tokens,
                                                      uint8_t* cache, int64_t num_slots, int32_t record_bytes,
                                                      uint32_t* dev_status, void* stream);

/*
 * Scratch size of nvfp4_sparse_mla_decode for a problem (host-only, no CUDA call).
 *   num_splits: the top-k list of each query row is cut into num_splits consecutive parts
 *   computed in parallel and merged by a second kernel (launched as a programmatic dependent
 *   of the first on the same stream); 0 lets the library choose from the problem size and the
 *   SM count of the current device (then this call reads the device attribute). The workspace
 *   holds each part's normalized partial output (f16, [rows, parts, h_q, 512]) and fp32
 *   log-sum-exp; it is 0 bytes when a single part is used.
 * Returns NVFP4_MLA_OK and sets *bytes, or an error code for an invalid problem.
 */
NVFP4_MLA_API int nvfp4_sparse_mla_decode_workspace_size(int32_t batch, int32_t s_q, int32_t h_q,
                                                         int32_t topk, int32_t record_bytes,
                                                         int32_t num_splits, size_t* bytes);

/*
 * How a decode of this shape runs on the current device (no launch, no device memory): the split
 * count it uses (num_splits, or the library's choice when 0) and how many kernels one call
 * launches (1: the decode grid alone, which also merges its 2-4 splits per row when they share a
 * cluster; 2: decode grid + merge grid; 0: nothing to do). Errors as ..._workspace_size, plus
 * NVFP4_MLA_ERR_UNSUPPORTED without a usable sm_103 device. (A service of this library; the pages
 * have no counterpart.)
 */
NVFP4_MLA_API int nvfp4_sparse_mla_decode_plan(int32_t batch, int32_t s_q, int32_t h_q, int32_t topk,
                                               int32_t record_bytes, int32_t num_splits, int32_t* splits,
                                               int32_t* kernels);

/*
 * Sparse MLA decode (read side).
 *   q            bf16 [batch, s_q, h_q, 576], contiguous, 16-byte aligned. Dims [0,512) are
 *                the NoPE (latent) part, [512,576) the RoPE part.
 *   cache        uint8 [num_slots, record_bytes & 0xFFFF], 16-byte aligned, as written by
 *                nvfp4_mla_quantize_append with the same record_bytes.
 *   indices      int32 [batch, s_q, topk], contiguous: the cache slots each query row attends.
 *                An entry < 0 is masked (padding); an entry >= num_slots is masked and sets
 *                NVFP4_MLA_DEV_INDEX_OUT_OF_RANGE. Repeated entries count once per occurrence.
 *   h_q          64 or 128. topk >= 1 (any value; the tail tile is masked).
 *   sm_scale     softmax scale applied to q.k (e.g. 1/sqrt(576)).
 *   attn_sink    nullable fp32 [h_q]: per-head extra logit that enters the softmax
 *                denominator of `out` only (no value vector) and not `lse`.
 *   out          bf16 [batch, s_q, h_q, 512], contiguous, 16-byte aligned:
 *                out = sum_j e^{z_j} V_j / (sum_j e^{z_j} + e^{sink_h}), z_j = sm_scale q.K_j
 *   lse          fp32 [batch, s_q, h_q]: natural-log log-sum-exp of the z_j of the used
 *                entries (sink excluded). A row with no used entry gets out = 0, lse = -inf.
 *   num_splits   0 = library choice, else 1..64 (see ..._workspace_size).
 *   workspace    device scratch of at least the size ..._workspace_size reports for the same
 *                arguments, 256-byte aligned; may be NULL when that size is 0. Its contents
 *                need no initialization.
 *   dev_status   nullable device uint32 (see NVFP4_MLA_DEV_*).
 * Precision: dequantized NVFP4 keys are exact in f16 and enter both contractions as f16, with q
 * as f16 times a per-head power of two (the same products as bf16 q for every element within
 * 2^28 of its head's largest |q|; the bf16 RoPE of 432-byte records and its q part stay bf16);
 * fp8 keys are e4m3 * scale rounded in fp32 and then to bf16 (QK^T) or f16 (PV); the
 * contractions run on tcgen05 16-bit MMAs with fp32 accumulation (P enters PV as f16); softmax
 * in fp32; `out` is rounded to bf16 once, after the parts' f16 partial outputs (relative error
 * <= 2^-11 each) are merged in fp32 when the top-k list is split.
 */
NVFP4_MLA_API int nvfp4_sparse_mla_decode(const void* q, const uint8_t* cache, int64_t num_slots,
                                          int32_t record_bytes, const int32_t* indices,
                                          int32_t batch, int32_t s_q, int32_t h_q, int32_t topk,
                                          float sm_scale, const float* attn_sink, void* out,
                                          float* lse, int32_t num_splits, void* workspace,
                                          size_t workspace_bytes, uint32_t* dev_status,
                                          void* stream);

/*
 * Sparse MLA decode for callers that cannot allocate device memory. (The pages have no
 * counterpart to this call; it is a service of this library.)
 *
 * nvfp4_sparse_mla_decode needs a caller-provided workspace when it splits the top-k lists.
 * Some callers cannot provide one: code that works within a device-memory budget fixed at
 * start-up and may not call cudaMalloc afterwards, code that must avoid cudaMalloc/cudaFree
 * because they can synchronize the device, or a host that lends the library only its input
 * and output buffers. This call takes the same arguments as nvfp4_sparse_mla_decode without
 * the workspace, and keeps its scratch in a library-owned, fixed-size device array of
 * NVFP4_MLA_NO_ALLOC_SCRATCH_BYTES bytes (reserved on every GPU that loads the library until
 * the process exits). It calls no cudaMalloc, cudaFree or allocating routine.
 *  - A problem whose split count (num_splits, or the library's choice when 0) needs more
 *    scratch than that returns NVFP4_MLA_ERR_WORKSPACE and launches nothing; pass a smaller
 *    num_splits (1 needs no scratch).
 *  - A call outside stream capture looks up the array's device address with the device
 *    current and keeps it; a call under capture uses the kept address. So make one call
 *    before any capture, and make one again after cudaDeviceReset or any other reset of the
 *    device's primary context: the reset may move the array, and an address kept from before
 *    it is invalid until an uncaptured call looks the array up again.
 *  - Argument checks come first and match nvfp4_sparse_mla_decode's (same status for the same
 *    bad argument); a failed runtime query leaves no pending CUDA error behind.
 *  - All calls share the array and it keeps the last call's contents (nothing in it needs to
 *    start at zero: each call writes every value it reads). Calls whose kernels may overlap on
 *    the GPU, e.g. on unordered streams, race on it and must be serialized by the caller.
 * Results equal those of nvfp4_sparse_mla_decode with the same num_splits.
 */
#define NVFP4_MLA_NO_ALLOC_SCRATCH_BYTES (((size_t)32) << 20)

NVFP4_MLA_API int nvfp4_sparse_mla_decode_no_alloc(const void* q, const uint8_t* cache, int64_t num_slots,
                                                   int32_t record_bytes, const int32_t* indices, int32_t batch,
                                                   int32_t s_q, int32_t h_q, int32_t topk, float sm_scale,
                                                   const float* attn_sink, void* out, float* lse,
                                                   int32_t num_splits, uint32_t* dev_status, void* stream);

/*
 * ---- Sequences in pages -------------------------------------------------------------------------
 *
 * The calls below see the pool as num_pages pages of page_size records: page p is the slots
 * [p page_size, (p + 1) page_size). page_size is a power of two, 1 to 4096. A batch of sequences is
 *   page_table  int32 [batch, max_pages], rows table_stride elements apart (table_stride >=
 *               max_pages): the pages of each sequence, in order. Entries behind a sequence's last
 *               page are not read; the calls that change the table leave -1 there.
 *   seq_lens    int32 [batch]: tokens of each sequence. Token t of sequence b lies in slot
 *               page_table[b][t / page_size] * page_size + t % page_size, the slot that
 *               nvfp4_mla_quantize_append writes its record to. Lengths are read as clamped to
 *               [0, max_pages * page_size].
 *   page_refs   int32 [num_pages], 16-byte aligned: how many table entries name each page. A page is
 *               free exactly when its count is 0; there is no other free list. A pool starts with
 *               all counts 0, all lengths 0 and all entries -1.
 * All of it lives on the device and is read there: no call needs a length or a page on the host, so
 * every call may be captured into a graph, and a replay follows the lengths of its time. The result of
 * each call depends on its inputs alone. A table entry within a sequence's length that names no page
 * of the pool sets NVFP4_MLA_DEV_INDEX_OUT_OF_RANGE and is passed over (as a key: masked). batch *
 * max_pages, max_pages * page_size and num_pages * page_size must stay below 2^31.
 */

/*
 * Scratch size of nvfp4_paged_mla_decode (host-only, no CUDA call; the same on every device): the
 * parts of query rows whose keys were read by several CTAs, and a plan. One size for up to 16 rows per
 * sequence (s_q * h_q); above that it grows with batch and with s_q * h_q.
 */
NVFP4_MLA_API int nvfp4_paged_mla_decode_workspace_size(int32_t batch, int32_t s_q, int32_t h_q, size_t* bytes);

/*
 * Attention of the last s_q tokens of each sequence over all tokens of the sequence up to their own
 * position, for decoding (s_q = 1), several tokens a step, and chunks of a prompt:
 *   q            bf16 [batch, s_q, h_q, 576], contiguous, 16-byte aligned (512 NoPE dims, 64 RoPE).
 *                Query i of sequence b has position seq_lens[b] - s_q + i; its record and those of
 *                the tokens before it are in the cache already.
 *   cache        uint8 [num_pages * page_size, record_bytes & 0xFFFF], 16-byte aligned.
 *   record_bytes 352, 352 | NVFP4_MLA_SCALES_BLOCK_ORDER or 432. 656-byte fp8 records are refused
 *                (NVFP4_MLA_ERR_UNSUPPORTED): the kernels convert e2m1 codes, and an e4m3 value times its
 *                fp32 scale is no f16 number, which their exact keys rest on.
 *   h_q          1 to 128.
 *   sm_scale, attn_sink, out, lse: as in nvfp4_sparse_mla_decode, the sum running over the tokens
 *                at positions 0 .. seq_lens[b] - s_q + i. A query with a negative position (a
 *                sequence shorter than s_q, an empty one, padding of the batch) gets out = 0,
 *                lse = -inf.
 *   workspace    device scratch of at least ..._workspace_size bytes, 256-byte aligned; needs no
 *                initialization. Calls that may overlap on the GPU need one each.
 * batch * s_q must stay below 2^24.
 * Precision: as nvfp4_sparse_mla_decode on NVFP4 records (parts of a row are normalized outputs in f16,
 * in steps of at least 2^-28, joined in fp32). A weight e^z is held in f16: off by 2^-11 of itself, and at
 * least by 2^-28 of the row's largest weight (down to 2^-37 where that one outweighs whole quarters of
 * its tile of 64 or 128 keys by more than 2^17, as an attention sink does). Over n tokens that is at most
 * 2^-28 sum|V| / (sum of the weights over the largest one), which counts where V is 0 for the few keys
 * that hold most of the weight and n passes some 10^5. A NaN in a query or in a record makes NaN the rows
 * that see it, and only those.
 */
NVFP4_MLA_API int nvfp4_paged_mla_decode(const void* q, const uint8_t* cache, int64_t num_pages, int32_t page_size,
                                         int32_t record_bytes, const int32_t* page_table, int64_t table_stride,
                                         int32_t max_pages, const int32_t* seq_lens, int32_t batch, int32_t s_q,
                                         int32_t h_q, float sm_scale, const float* attn_sink, void* out, float* lse,
                                         void* workspace, size_t workspace_bytes, uint32_t* dev_status, void* stream);

/*
 * Scratch size of fork_sequences, resize_sequences and compact_pages (host-only): enough for each of
 * them with these sizes. num_pairs: pairs of a fork (0 if none is made).
 */
NVFP4_MLA_API int nvfp4_mla_pages_workspace_size(int32_t batch, int32_t max_pages, int64_t num_pages,
                                                 int32_t num_pairs, size_t* bytes);

/*
 * Copies page src[k] to page dst[k] (int32 [n], device) in every cache of a model.
 *   caches       HOST array of num_caches (1..256) device pointers, one cache per layer, each
 *                uint8 [num_pages * page_size, record_bytes & 0xFFFF], 16-byte aligned. Any record
 *                width of this library.
 * A pair with a negative page is skipped (padding); one with a page >= num_pages is skipped and sets
 * NVFP4_MLA_DEV_INDEX_OUT_OF_RANGE. All pairs are copied at once: targets should be distinct, and no
 * page both source and target (else which bytes such a target holds afterwards is unspecified).
 * Page counts are not touched. n == 0 is valid and launches nothing.
 */
NVFP4_MLA_API int nvfp4_mla_copy_pages(uint8_t* const* caches, int32_t num_caches, int64_t num_pages,
                                       int32_t page_size, int32_t record_bytes, const int32_t* src,
                                       const int32_t* dst, int32_t n, uint32_t* dev_status, void* stream);

/*
 * Forks sequences: for every pair k, sequence dst[k] (int32 [num_pairs], device) becomes a copy of
 * sequence src[k]. Nothing is copied but the table row and the length: the pages are shared and
 * counted, and a page is copied when one of its sequences grows into it (resize_sequences). The old
 * pages of dst[k] are given back. All pairs read the state before the call, so a permutation of
 * sequences (a beam-search step) is one call. Of several pairs with the same target the last one
 * counts; a pair with a negative sequence is skipped, one with a sequence >= batch is skipped and
 * sets NVFP4_MLA_DEV_INDEX_OUT_OF_RANGE.
 */
NVFP4_MLA_API int nvfp4_mla_fork_sequences(int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                           int32_t* seq_lens, int32_t batch, int32_t* page_refs, int64_t num_pages,
                                           int32_t page_size, const int32_t* src, const int32_t* dst,
                                           int32_t num_pairs, void* workspace, size_t workspace_bytes,
                                           uint32_t* dev_status, void* stream);

/*
 * Gives each sequence the length new_lens[b] (int32 [batch]).
 *  - A shorter one gives back the pages behind its new end (0 frees the sequence): prompts that have
 *    finished, drafted tokens that were rejected. These pages may be taken by the same call.
 *  - A longer one takes the lowest free pages, sequence by sequence. If its last page is partly
 *    filled and shared, it first takes a page of its own for it, into which the records it holds are
 *    copied in every cache (`caches`, as in copy_pages; num_caches 0: no records are copied). The counts
 *    before the call decide: if all k holders of such a page grow in one call, each takes a page of its
 *    own, k in all, and the shared one is free behind the call (not within it).
 *  - slots (int64 [batch, max_new], 8-byte aligned; unused when max_new is 0) receives the slots of
 *    the first max_new new tokens of each sequence, -1 behind its last one: the slot_mapping of the
 *    append that writes them.
 * If there are fewer free pages than the call needs, no sequence grows, all slots are -1 and
 * NVFP4_MLA_DEV_PAGES_EXHAUSTED is set. A new length below 0 or above max_pages * page_size leaves
 * its sequence unchanged and sets NVFP4_MLA_DEV_LENGTH_OUT_OF_RANGE.
 */
NVFP4_MLA_API int nvfp4_mla_resize_sequences(int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                             int32_t* seq_lens, const int32_t* new_lens, int32_t batch,
                                             int32_t* page_refs, int64_t num_pages, int32_t page_size,
                                             uint8_t* const* caches, int32_t num_caches, int32_t record_bytes,
                                             int64_t* slots, int32_t max_new, void* workspace,
                                             size_t workspace_bytes, uint32_t* dev_status, void* stream);

/*
 * Compacts a pool: afterwards the n pages in use are pages 0 .. n - 1. The i-th used page at or
 * behind page n moves, in every cache, into the i-th free page before it; other pages stay.
 *   table_out, refs_out   the new table and counts; each may be the old one (in place) or a buffer
 *                of its own: then the old table still names intact records until its pages are taken.
 *                refs_out 16-byte aligned.
 *   page_map     int32 [num_pages]: receives the new page of every old one, -1 for a free one.
 *   live         int32 [1]: receives n.
 */
NVFP4_MLA_API int nvfp4_mla_compact_pages(uint8_t* const* caches, int32_t num_caches, int32_t record_bytes,
                                          const int32_t* page_table, int64_t table_stride, int32_t* table_out,
                                          int64_t table_out_stride, int32_t max_pages, const int32_t* seq_lens,
                                          int32_t batch, const int32_t* page_refs, int32_t* refs_out,
                                          int64_t num_pages, int32_t page_size, int32_t* page_map, int32_t* live,
                                          void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                          void* stream);

/*
 * ---- Heads and latents --------------------------------------------------------------------------
 *
 * The calls below stand around the latent attention of one layer. With c the latent (512) of a token, head h's key
 * is W_uk[h] c (128 dims) beside the 64 RoPE dims that all heads share, and its value W_uv[h] c (128 dims).
 *   kv_b  bf16 [h_q, 256, 512]: rows 0-127 of head h are W_uk[h], rows 128-255 W_uv[h].
 * Two forms of the attention give the same result:
 *   absorbed  nvfp4_mla_absorb_query -> nvfp4_paged_mla_decode or nvfp4_sparse_mla_decode ->
 *             nvfp4_mla_project_values. The cache is read as it stands: for single tokens and short chunks.
 *   expanded  nvfp4_paged_mla_expand -> nvfp4_ragged_mla_attention. 640 instead of 2176 FLOP per query, key and head,
 *             after 262144 per key and head: for chunks of some 200 tokens and more.
 * All tensors are bf16, sums run in fp32 and are rounded once; h_q is 1 to 128, other values return
 * NVFP4_MLA_ERR_UNSUPPORTED. Strides are in elements and positive multiples of 8, inner strides 1; inputs are 16-byte aligned, outputs
 * contiguous and 32-byte aligned. The stride of a dimension of one entry is not looked at. Row counts stay below 2^31 - 4096.
 * Sequences lie packed, one behind the other: sequence b has rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (int32
 * [batch + 1], device, from 0 on and not decreasing; entries are read as clamped to [0, rows], and other values give
 * unspecified rows but touch nothing outside the tensors).
 * Rows from cu_seqlens[batch] on are never written and change no result, so buffers may be larger than what a batch fills, and a
 * captured call follows the lengths of its replay. The attention reads whole boxes of rows, though, so inputs up to their last
 * row may be read while a call runs. A pipeline wait that gives up sets NVFP4_MLA_DEV_TIMEOUT.
 */

/*
 * out[t, h, 0:512] = W_uk[h]^T q[t, h, 0:128]; out[t, h, 512:576] = q[t, h, 128:192], rotated where positions is not NULL.
 *   q              [num_tokens, h_q, 192], any token and head stride.
 *   positions      int64 [num_tokens] or NULL; cos_table, sin_table fp32 [num_positions, 32], 16-byte aligned; rotate_half 1:
 *                  pairs (f, f + 32), 0: pairs (2f, 2f + 1), as in nvfp4_mla_norm_rope_quantize_append. A token whose
 *                  position lies outside sets NVFP4_MLA_DEV_POSITION_OUT_OF_RANGE; its RoPE dims of out are left as they were.
 *   out            [num_tokens, h_q, 576]: the q of the decode calls.
 */
NVFP4_MLA_API int nvfp4_mla_absorb_query(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* kv_b,
                                         int64_t kv_b_row_stride, int64_t kv_b_head_stride, const int64_t* positions,
                                         const float* cos_table, const float* sin_table, int64_t num_positions,
                                         int32_t rotate_half, int64_t num_tokens, int32_t h_q, void* out,
                                         uint32_t* dev_status, void* stream);

/*
 * out[t, h, 0:128] = W_uv[h] latent[t, h, 0:512]: the heads' outputs from the decode calls' out.
 */
NVFP4_MLA_API int nvfp4_mla_project_values(const void* latent, int64_t latent_token_stride, int64_t latent_head_stride,
                                           const void* kv_b, int64_t kv_b_row_stride, int64_t kv_b_head_stride,
                                           int64_t num_tokens, int32_t h_q, void* out, uint32_t* dev_status, void* stream);

/*
 * Keys and values of the first cu_seqlens[b + 1] - cu_seqlens[b] tokens of each sequence from their records in pages
 * (see "Sequences in pages"; record_bytes as in nvfp4_paged_mla_decode):
 *   kv     [num_rows, h_q, 256]: W_uk[h] c, then W_uv[h] c.
 *   k_pe   [num_rows, 64], 16-byte aligned: the records' RoPE dims.
 * A token whose table entry names no page of the pool, or that lies behind the table's last entry, sets
 * NVFP4_MLA_DEV_INDEX_OUT_OF_RANGE and gets zeros.
 */
NVFP4_MLA_API int nvfp4_paged_mla_expand(const uint8_t* cache, int64_t num_pages, int32_t page_size, int32_t record_bytes,
                                         const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                         const int32_t* cu_seqlens, int32_t batch, const void* kv_b, int64_t kv_b_row_stride,
                                         int64_t kv_b_head_stride, int32_t h_q, void* kv, void* k_pe, int64_t num_rows,
                                         uint32_t* dev_status, void* stream);

/* Scratch size of nvfp4_ragged_mla_attention: one size for every call. */
NVFP4_MLA_API int nvfp4_ragged_mla_attention_workspace_size(size_t* bytes);

/*
 * Attention of the last lq tokens of each sequence over its lk tokens up to their own position: query i sees the keys
 * 0 .. lk - lq + i of its sequence.
 *   q                [num_q, h_q, 192], RoPE dims last, rotated already; any token and head stride.
 *   kv, k_pe         [num_k, h_q, 256] and [num_k, 64] as from nvfp4_paged_mla_expand; any token and head stride.
 *   sm_scale, attn_sink, lse: as in nvfp4_sparse_mla_decode; lse [num_q, h_q].
 *   out              [num_q, h_q, 128].
 *   workspace        at least ..._workspace_size bytes, 256-byte aligned; needs no initialization. Calls that may overlap on
 *                    the GPU need one each.
 * A query without a visible key gets out = 0, lse = -inf. batch is at most 2^20, num_k below 2^26.
 * Precision: weights e^z are rounded to bf16 (2^-8 of themselves, however small), row sums are of the unrounded ones.
 * A NaN in a query or a key, and a score of +infinity, make NaN the rows that see it; a score of -infinity has the weight 0. A NaN or
 * infinity in a value makes its dim, and may make all dims, of the rows that see it NaN or infinite; rows that do not see it, and
 * log-sum-exps, never.
 * Which of two kernels runs follows the average rows and keys of a sequence (num_q / batch, num_k / batch), as the lengths lie on the
 * device: tensors that fit the batch, without padding sequences, let long chunks take the faster one. Results do not depend on
 * it beyond the order of sums.
 */
NVFP4_MLA_API int nvfp4_ragged_mla_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t num_q,
                                             const void* kv, int64_t kv_token_stride, int64_t kv_head_stride, const void* k_pe,
                                             int64_t k_pe_stride, int64_t num_k, const int32_t* cu_seqlens_q,
                                             const int32_t* cu_seqlens_k, int32_t batch, int32_t h_q, float sm_scale,
                                             const float* attn_sink, void* out, float* lse, void* workspace,
                                             size_t workspace_bytes, uint32_t* dev_status, void* stream);

/*
 * Self-test of the decode's wait bound (no counterpart on the pages). Every pipeline wait in
 * the decode kernel gives up after about one second (then the kernel sets
 * NVFP4_MLA_DEV_TIMEOUT, drains its own work and returns; the context stays usable). This call
 * runs one such wait on an mbarrier that nothing arrives on, on `stream`:
 *   dev_status   device uint32: NVFP4_MLA_DEV_TIMEOUT is OR-ed in when the wait gives up.
 *   elapsed_ns   device uint64: how long the wait lasted, in nanoseconds.
 * Returns NVFP4_MLA_ERR_INVALID_ARG for NULL pointers, NVFP4_MLA_ERR_UNSUPPORTED off sm_103.
 */
NVFP4_MLA_API int nvfp4_mla_selftest_wait_timeout(uint32_t* dev_status, uint64_t* elapsed_ns, void* stream);

/* Static text for a status code (never NULL). */
NVFP4_MLA_API const char* nvfp4_mla_status_string(int status);

/* Library version as 10000*major + 100*minor + patch. */
NVFP4_MLA_API int nvfp4_mla_version(void);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_MLA_H_ */

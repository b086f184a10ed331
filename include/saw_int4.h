/*
 * saw_int4.h -- C ABI of the SAW-INT4 hot path on GB300 (sm_103a).
 *
 * Two operations, from the pages on SAW-INT4 (Jia et al., 2026):
 *
 *  1. saw_quantize_append: each new token's K/V vector of head_dim values
 *     per kv-head is rotated by a block-diagonal Hadamard transform (blocks
 *     of h), quantized token-wise to INT4 with its own scale, and appended
 *     into a paged KV cache without touching any other token.
 *     youngju.dev, "INT4 KV-cache quantization" (English transcription),
 *     "Why Naive INT4 Breaks", "The Rotation Trick -- Block-Diagonal
 *     Hadamard" and the fused-kernel diagram in "The System Is the Design --
 *     A Fused Kernel"; gist.science, "SAW-INT4: System-Aware 4-Bit KV-Cache
 *     Quantization for Real-World LLM Serving", s.2 "Metodologia" (token-wise
 *     quantization, Block-Diagonal Rotation, fused kernel) and s.4 (h = 128,
 *     rotation of K only).
 *
 *  2. saw_paged_decode_int4: decode attention of one query token per
 *     sequence over that INT4 cache, with dequantization fused into the
 *     attention kernel (gist.science s.2 point 3, fusion into decoding).
 *     q is rotated once (q.k = Hq.Hk because H is orthogonal), and the output
 *     is rotated back when V was rotated.
 *
 * Further calls build on these two: saw_decode_step (both in one launch),
 * saw_prefill_attn_int4 (causal attention of a chunk of queries over the
 * same cache), the *_ex forms with binary16 inputs or bfloat16 scale/zero
 * metadata, and a BF16 paged cache with the same decode (saw_bf16_*), the
 * baseline the pages compare INT4 against.  saw_build_tables, saw_rope_table,
 * saw_rope_append and saw_prefix_decode_int4 make the rest of a serving step
 * around the cache: tables and slots from lengths, rotary positions fused
 * with the append, and a decode that reads a shared prefix once per group.
 *
 * Readings taken where the pages are silent: Sylvester ordering of H, the
 * 1/sqrt(h) scale applied after an ascending-stride butterfly, one binary16
 * (scale, zero) pair per (token, kv-head) from the rotated row's min/max
 * (zero rounded toward -inf, scale toward +inf), round-half-even codes 0..15,
 * two codes per byte (even index in the low nibble), and the page layout
 * below.  Each is stated with the function it governs.
 *
 * Common rules for every entry point:
 *  - All buffers are owned by the caller.  The library allocates nothing and
 *    keeps no state between calls (saw_paged_decode_int4_noalloc's fixed
 *    scratch array aside); every call is thread-safe.
 *  - Pointers marked "device" must be device memory of the current device.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream).  Work is
 *    enqueued asynchronously on it.  The return value reports argument
 *    checks and launch errors only.
 *  - `dev_status` is an optional device int32 (may be NULL).  A kernel that
 *    meets a bad index or a wait that runs out writes a nonzero
 *    saw_status code into it (the first one wins); it never traps.  The
 *    caller zeroes it and reads it after the stream has finished.
 */
#ifndef SAW_INT4_H
#define SAW_INT4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum saw_status {
  SAW_OK = 0,
  SAW_ERR_INVALID_ARG = 1,    /* a null pointer, a bad size, a misaligned buffer */
  SAW_ERR_UNSUPPORTED = 2,    /* a shape this build has no kernel for */
  SAW_ERR_CUDA = 3,           /* a CUDA runtime error at launch */
  SAW_ERR_DEVICE_INDEX = 4,   /* device-side: a slot, page id or length out of range (skipped) */
  SAW_ERR_DEVICE_TIMEOUT = 5, /* device-side: a bounded wait on a copy ran out */
  SAW_ERR_DEVICE_PAGES = 6    /* device-side: the list of free pages ran out (saw_build_tables) */
} saw_status;

/* Human-readable name of a status code.  Never NULL. */
const char* saw_status_string(int32_t status);

/*
 * Bytes of one cache tensor (K or V of one layer):
 *   [num_pages][num_kv_heads][chunk],  chunk = page_size*head_dim/2 + 4*page_size.
 * Inside a chunk: token offset o's packed codes at o*head_dim/2 (byte j holds
 * code 2j in the low nibble and 2j+1 in the high nibble), then, from
 * page_size*head_dim/2, one 4-byte word per offset: binary16 scale, binary16
 * zero, little-endian.  A row dequantizes as code*scale + zero.  The layout
 * is a reading: the pages require only a paged, token-wise layout.
 * Returns 0 for a negative or zero argument.
 */
size_t saw_cache_bytes(int32_t num_pages, int32_t page_size, int32_t num_kv_heads,
                       int32_t head_dim);

/*
 * Rotate, quantize and append num_tokens tokens of K (and V) into the paged
 * caches (youngju.dev "The System Is the Design -- A Fused Kernel";
 * gist.science s.2 and s.3 point 3).
 *
 * k, v          device bfloat16 [num_tokens][num_kv_heads][head_dim], rows of
 *               a token contiguous; token stride k_token_stride /
 *               v_token_stride elements (>= num_kv_heads*head_dim, multiple
 *               of 8).  v may be NULL: K only (v_cache is then ignored).
 * slot_mapping  device int32 [num_tokens]: slot = page*page_size + offset.
 *               -1 marks padding and is skipped; any other value outside
 *               [0, num_pages*page_size) is skipped and reported through
 *               dev_status as SAW_ERR_DEVICE_INDEX.
 * k_cache, v_cache  device, saw_cache_bytes() each, 16-byte aligned.
 * rotate_k, rotate_v  0 or 1: apply the block-diagonal Hadamard rotation
 *               before quantizing.  The gist.science page (s.4) reports that
 *               rotating K only matches rotating both.
 * block_h       rotation block size h: 16, 32, 64, 128 or 256, at most
 *               head_dim (ignored when neither tensor is rotated).
 *
 * Per row, exactly: widen to binary32; if rotated, an in-place butterfly per
 * h-block with strides 1, 2, ..., h/2 (each a+b, a-b rounded to nearest),
 * then multiply by binary32(1/sqrt(h)); mn/mx over the row; zero =
 * binary16 round-down(mn), scale = binary16 round-up((mx - zero)/15), both
 * saturating at +-65504 and writing zero as +0; r = 1/scale (0 if scale is
 * 0); code = clamp(round-half-even((y - zero)*r), 0, 15).  Each operation is
 * one binary32 round-to-nearest step, so the bytes are fully determined.
 * Inputs are expected finite; non-finite inputs give unspecified codes.
 *
 * Supported: head_dim 64, 128 or 256 (128 runs the tiled bulk kernel, 64
 * and 256 a warp-per-row kernel; the bytes follow the same rule); page_size
 * 16, 32 or 64; num_kv_heads >= 1.  Other sizes: SAW_ERR_UNSUPPORTED.
 * Rows whose slot is written by two tokens of the same call race.
 */
int32_t saw_quantize_append(const void* k, const void* v, int64_t k_token_stride,
                            int64_t v_token_stride, const int32_t* slot_mapping,
                            int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                            void* k_cache, void* v_cache, int32_t num_pages, int32_t page_size,
                            int32_t rotate_k, int32_t rotate_v, int32_t block_h,
                            int32_t* dev_status, void* stream);

/*
 * How many splits of the context the decode will use, and how many pages
 * each split covers, for these sizes on the current device
 * (pages_per_split = 0 picks them from the SM count; > 0 forces it).  The
 * plan is the same at every head dimension.
 * Writes *num_splits and *pages_per_split_out; returns a saw_status.
 */
int32_t saw_decode_plan(int32_t num_seqs, int32_t num_kv_heads, int32_t page_size,
                        int32_t max_seq_len, int32_t pages_per_split, int32_t* num_splits,
                        int32_t* pages_per_split_out);

/*
 * Workspace bytes saw_paged_decode_int4 needs for these sizes with the same
 * pages_per_split argument, on the current device (0 when the plan has one
 * split, which writes the output directly).  Returns 0 on bad arguments.
 * The workspace holds the split partials and, first, two counter words per
 * (sequence, kv-head) that the merge uses: zero-fill a new workspace once
 * (e.g. cudaMemset) before its first use; every call leaves those words at
 * zero again.
 */
size_t saw_decode_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t page_size, int32_t max_seq_len,
                                  int32_t pages_per_split);

/*
 * Decode attention for one query token per sequence over the INT4 pages
 * (gist.science s.2 point 3: the rotation and dequantization live inside
 * the decode kernel; youngju.dev "The Rotation Trick": H is orthogonal, so
 * attention can run in the rotated domain).
 *
 * q             device bfloat16 [num_seqs][num_q_heads][head_dim].
 * k_cache, v_cache  device caches written by saw_quantize_append with the
 *               same num_kv_heads, head_dim, page_size, rotate_* and block_h
 *               (the caller's contract; a mismatch gives wrong numbers).
 * block_tables  device int32 [num_seqs][max_blocks_per_seq]: logical page i
 *               of a sequence -> physical page id.  Ids outside
 *               [0, num_pages) are skipped and reported as
 *               SAW_ERR_DEVICE_INDEX.
 * seq_lens      device int32 [num_seqs]: tokens to attend over (including a
 *               token just appended).  0 gives a zero output row.  A value
 *               below 0 or above max_seq_len is reported as
 *               SAW_ERR_DEVICE_INDEX and treated as 0.
 * max_seq_len   host upper bound on seq_lens; fixes the split plan.
 *               max_blocks_per_seq must be >= ceil(max_seq_len / page_size).
 * num_q_heads   a multiple of num_kv_heads with at most 8 q-heads per
 *               kv-head; q-head j reads kv-head j / (num_q_heads/num_kv_heads).
 * sm_scale      softmax scale on q.k; 0 means 1/sqrt(head_dim).
 * out           device float32 [num_seqs][num_q_heads][head_dim].
 * workspace     device, >= saw_decode_workspace_bytes(...) bytes, 16-byte
 *               aligned (may be NULL when that is 0), zero-filled before its
 *               first use (calls leave it reusable).  The last split to
 *               finish for a (sequence, kv-head) merges the partials, so one
 *               launch covers the whole decode.  Calls sharing a workspace
 *               must be ordered (one stream).
 * pages_per_split  0 = automatic; > 0 forces the split size (tests).
 *
 * Computes, per (sequence, q-head): q' = (1/sqrt(h)) H q if K was rotated;
 * t_j = sm_scale * q'.(code_j*s_j + z_j); p = softmax(t); o' = sum_j p_j
 * (code_j*s_j + z_j) over V; o = (1/sqrt(h)) H o' if V was rotated.  The
 * GQA group of a kv-head is served by one pass over its pages.  Arithmetic
 * (head_dim 64, 128 and 256 alike): q' and p*s in binary16 on the tensor
 * cores with binary32 accumulation, softmax in binary32; results match a
 * float64 evaluation to about 1e-3 of the output's largest magnitude.
 * Up to 8 q-heads per kv-head; head_dim 64, 128 or 256 (else
 * SAW_ERR_UNSUPPORTED).
 */
int32_t saw_paged_decode_int4(const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables, int32_t max_blocks_per_seq,
                              const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                              int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                              int32_t num_pages, int32_t page_size, int32_t rotate_k,
                              int32_t rotate_v, int32_t block_h, float sm_scale, float* out,
                              void* workspace, size_t workspace_bytes, int32_t pages_per_split,
                              int32_t* dev_status, void* stream);

/*
 * One decode step of a layer, fused into one launch: for every sequence b,
 * quantize-append the new token's K and V rows at position seq_lens[b] - 1
 * (slot = block_tables[b][(L-1)/page_size]*page_size + (L-1)%page_size),
 * then attend over all seq_lens[b] tokens -- the per-token path of the
 * fused-kernel diagram in youngju.dev "The System Is the Design -- A Fused
 * Kernel" (rotate, quantize, append to the paged block) followed by the
 * decode of gist.science s.2 point 3.
 *
 * k_new, v_new  device bfloat16 [num_seqs][num_kv_heads][head_dim],
 *               contiguous, 16-byte aligned: the new token of each sequence.
 * k_cache, v_cache  written (the new rows) and read.
 * seq_lens      lengths INCLUDING the new token (>= 1).  A length of 0
 *               appends nothing and gives a zero output row.
 * flags         0, or SAW_STEP_EARLY_PAGES: the caller guarantees that the
 *               kernel issued just before this call on `stream` writes none
 *               of block_tables, seq_lens, k_cache and v_cache.  The kernel
 *               may then read them and start its page copies while that
 *               kernel finishes (programmatic dependent launch); it still
 *               waits for it before reading q, k_new, v_new or writing.
 * Other arguments as saw_paged_decode_int4.  The appended bytes equal those
 * of saw_quantize_append on the same row, and the output equals
 * saw_quantize_append followed by saw_paged_decode_int4.  head_dim 128 only
 * (SAW_ERR_UNSUPPORTED otherwise).
 */
#define SAW_STEP_EARLY_PAGES 1
int32_t saw_decode_step(const void* q, const void* k_new, const void* v_new, void* k_cache,
                        void* v_cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                        const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                        int32_t num_pages, int32_t page_size, int32_t rotate_k, int32_t rotate_v,
                        int32_t block_h, float sm_scale, float* out, void* workspace,
                        size_t workspace_bytes, int32_t pages_per_split, int32_t flags,
                        int32_t* dev_status, void* stream);

/*
 * saw_paged_decode_int4_noalloc -- the same decode as saw_paged_decode_int4
 * for callers that cannot allocate device memory.  The pages have no
 * counterpart: this is a deployment convenience of this library.
 *
 * Who needs it: a plugin or custom op whose host framework owns every device
 * allocation (it may not call cudaMalloc itself), or a latency-critical loop
 * that cannot afford cudaMalloc/cudaFree's device synchronisation.  The split-K scratch comes
 * from a fixed 4 MiB array in device memory declared by the library itself;
 * the caller passes only inputs and outputs (arguments as in
 * saw_paged_decode_int4, without the workspace).
 *
 *  - Limit: the plan's scratch (saw_decode_workspace_bytes) must be at most
 *    4 MiB; a larger plan returns SAW_ERR_UNSUPPORTED before any launch
 *    (use saw_paged_decode_int4, or a larger pages_per_split).
 *  - Memory: every GPU that loads the library holds the 4 MiB until the
 *    process exits.  No cudaMalloc/cudaFree is ever called.
 *  - Set-up: the first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress, with that device current) and keeps it.
 *  - Sharing: all calls on a device share the array, so calls whose kernels
 *    may overlap on the GPU (different streams without ordering) race.
 *    Each call first clears the merge's counter words in it
 *    (cudaMemsetAsync on `stream`); the rest needs no clearing.
 */
int32_t saw_paged_decode_int4_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* seq_lens, int32_t num_seqs,
                                      int32_t max_seq_len, int32_t num_q_heads,
                                      int32_t num_kv_heads, int32_t head_dim, int32_t num_pages,
                                      int32_t page_size, int32_t rotate_k, int32_t rotate_v,
                                      int32_t block_h, float sm_scale, float* out,
                                      int32_t pages_per_split, int32_t* dev_status, void* stream);

/*
 * saw_prefill_attn_int4 -- chunked-prefill attention over the INT4 cache.
 *
 * Pages: youngju.dev "INT4 KV-cache quantization", "Why the KV Cache Is the
 * Real Bottleneck", and gist.science "SAW-INT4", s.1: the method has to work
 * inside engines that run fused attention over paged KV.  Reading: the
 * query of the token at position p of its sequence attends causally to that
 * sequence's cached tokens 0..p; dequantization, q rotation and the inverse
 * V rotation are those of saw_paged_decode_int4.  Append the chunk's K/V
 * with saw_quantize_append first (same stream).
 *
 *  q             device bfloat16 [total_q][num_q_heads][head_dim]: the query
 *                rows of every sequence's chunk, sequence after sequence.
 *  cu_q_lens     device int32 [num_seqs + 1]: rows cu_q_lens[b] ..
 *                cu_q_lens[b+1] - 1 belong to sequence b and are its last
 *                q_len_b = cu_q_lens[b+1] - cu_q_lens[b] tokens, so row i sits
 *                at position seq_lens[b] - q_len_b + (i - cu_q_lens[b]).
 *  seq_lens      device int32 [num_seqs]: cached tokens, the chunk included.
 *  max_q_len     a bound on every q_len_b (sizes the grid; <= max_seq_len).
 *  k/v caches, block tables, rotation and block_h, sm_scale (0 = 1/sqrt(D)):
 *                as in saw_paged_decode_int4.
 *  out           device float32 [total_q][num_q_heads][head_dim].
 *
 * No workspace.  head_dim 128 and page_size 16/32/64 (else
 * SAW_ERR_UNSUPPORTED); any number of q-heads per kv-head.  A sequence
 * whose q_len, seq_len or cu_q_lens entries are inconsistent (q_len < 0,
 * q_len > seq_len, q_len > max_q_len, seq_len > max_seq_len, rows beyond
 * total_q) is skipped and
 * SAW_ERR_DEVICE_INDEX is stored in *dev_status; a bad page id is skipped
 * and reported the same way; a copy that never lands ends the wait after
 * about a second with SAW_ERR_DEVICE_TIMEOUT.  Asynchronous on `stream`.
 */
int32_t saw_prefill_attn_int4(const void* q, const int32_t* cu_q_lens, const void* k_cache,
                              const void* v_cache, const int32_t* block_tables,
                              int32_t max_blocks_per_seq, const int32_t* seq_lens,
                              int32_t num_seqs, int32_t total_q, int32_t max_q_len,
                              int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t head_dim, int32_t num_pages, int32_t page_size,
                              int32_t rotate_k, int32_t rotate_v, int32_t block_h, float sm_scale,
                              float* out, int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * Format variants.  The fused-kernel diagram of youngju.dev ("The System Is
 * the Design -- A Fused Kernel") feeds the kernel binary16 ("fp16") K and V;
 * engines also run in bfloat16.  The pages fix one scale per token but not
 * the storage format of the (scale, zero) pair.  The *_ex calls below are
 * the calls above with one extra argument, `formats`, an OR of:
 *
 *   SAW_FMT_F16_INPUT  q, K and V (and k_new, v_new) are binary16 instead of
 *                      bfloat16.  Both widen to binary32 exactly, so every
 *                      rule after that step is unchanged.
 *   SAW_FMT_BF16_META  the caches' per-row words hold {scale, zero} as
 *                      bfloat16 instead of binary16 (same place, same
 *                      order).  zero = bfloat16 round-down(min), scale =
 *                      bfloat16 round-up((max - zero)/15), both saturating
 *                      at +-(2^128 - 2^120), a zero stored as +0, and a
 *                      nonzero scale raised to at least 2^-126 (so that
 *                      1/scale is finite); codes as before.  A cache must be
 *                      written and read with the same metadata format.
 *
 * formats 0 is the plain call.  Any other bit: SAW_ERR_INVALID_ARG, before
 * anything is enqueued.
 * Supported shapes are those of the plain calls (all head dims for append
 * and decode; head_dim 128 for the decode step and the prefill).
 * Precision note: the head_dim-128 decode and the prefill carry p * scale_V
 * as a binary16 MMA operand, as they do for binary16 metadata, so their
 * error bound assumes V scales below 65504 (rows spanning less than about
 * 9.8e5); the head_dim 64/256 decode computes in binary32 throughout.
 * ------------------------------------------------------------------------ */
#define SAW_FMT_F16_INPUT 1
#define SAW_FMT_BF16_META 2

int32_t saw_quantize_append_ex(const void* k, const void* v, int64_t k_token_stride,
                               int64_t v_token_stride, const int32_t* slot_mapping,
                               int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                               void* k_cache, void* v_cache, int32_t num_pages,
                               int32_t page_size, int32_t rotate_k, int32_t rotate_v,
                               int32_t block_h, int32_t formats, int32_t* dev_status,
                               void* stream);

int32_t saw_paged_decode_int4_ex(const void* q, const void* k_cache, const void* v_cache,
                                 const int32_t* block_tables, int32_t max_blocks_per_seq,
                                 const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t num_pages, int32_t page_size, int32_t rotate_k,
                                 int32_t rotate_v, int32_t block_h, float sm_scale, float* out,
                                 void* workspace, size_t workspace_bytes,
                                 int32_t pages_per_split, int32_t formats, int32_t* dev_status,
                                 void* stream);

int32_t saw_decode_step_ex(const void* q, const void* k_new, const void* v_new, void* k_cache,
                           void* v_cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                           const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                           int32_t num_pages, int32_t page_size, int32_t rotate_k,
                           int32_t rotate_v, int32_t block_h, float sm_scale, float* out,
                           void* workspace, size_t workspace_bytes, int32_t pages_per_split,
                           int32_t flags, int32_t formats, int32_t* dev_status, void* stream);

int32_t saw_paged_decode_int4_noalloc_ex(const void* q, const void* k_cache,
                                         const void* v_cache, const int32_t* block_tables,
                                         int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                         int32_t num_seqs, int32_t max_seq_len,
                                         int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t num_pages, int32_t page_size,
                                         int32_t rotate_k, int32_t rotate_v, int32_t block_h,
                                         float sm_scale, float* out, int32_t pages_per_split,
                                         int32_t formats, int32_t* dev_status, void* stream);

int32_t saw_prefill_attn_int4_ex(const void* q, const int32_t* cu_q_lens, const void* k_cache,
                                 const void* v_cache, const int32_t* block_tables,
                                 int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                 int32_t num_seqs, int32_t total_q, int32_t max_q_len,
                                 int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim, int32_t num_pages, int32_t page_size,
                                 int32_t rotate_k, int32_t rotate_v, int32_t block_h,
                                 float sm_scale, float* out, int32_t formats,
                                 int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * A serving step around the cache.  The pages (gist.science s.1) place the
 * method inside engines with paged KV and continuous batching; the four calls
 * below are the steps of such an engine next to the append and the attention.
 * ------------------------------------------------------------------------ */

/*
 * saw_build_tables -- block tables, slot mapping, positions, lengths and row
 * offsets of a batch, from the requests' lengths and a list of free pages.
 *
 * For request b with c = cached_lens[b] cached and n = new_lens[b] new tokens:
 *   old = ceil(c / page_size), need = ceil((c + n) / page_size) - old,
 *   off = the sum of need over the requests before b;
 *   block_tables[b][e] = src row's entry e for e < old, free_pages[off + e -
 *   old] for old <= e < old + need; later entries are left as they were;
 *   token i < n: position c + i, slot = entry * page_size + offset;
 *   seq_lens[b] = c + n; cu_q_lens = exclusive sums of n (saw_prefill_attn_int4).
 * slot_mapping and positions past the last token are -1 and 0, so a batch
 * padded to max_tokens can be appended as it is.
 *
 * src_tables    device int32 [num_src_rows][src_blocks]: the requests' tables
 *               so far, or NULL when nothing is cached.  May be block_tables
 *               itself (then src_rows is NULL, src_blocks equals
 *               max_blocks_per_seq and num_src_rows >= num_seqs): only new
 *               entries are written.  Must not overlap it otherwise.
 * src_rows      device int32 [num_seqs]: row of src_tables of each request
 *               (several may name the same row: a fork of its first
 *               ceil(cached/page_size) pages; the last of these must be full
 *               if two requests go on to write).  NULL: row b.
 * cached_lens, new_lens  device int32 [num_seqs]; cached_lens NULL: all 0.
 * free_pages    device int32 [max_free], taken from the front; num_free:
 *               device int32 [1], how many of them are free (NULL: max_free).
 * positions, pages_taken  may be NULL.  *pages_taken: pages used of the list.
 *
 * A request whose pages are not all in the list gets none: its slots are -1,
 * its positions 0, its seq_lens entry cached_lens[b], and
 * SAW_ERR_DEVICE_PAGES is reported; later requests that need no page are
 * served.  A request with a negative length, a length beyond
 * max_blocks_per_seq pages, or cached tokens without a source row is refused
 * the same way with seq_lens 0 and SAW_ERR_DEVICE_INDEX (its new tokens, if
 * the count is not negative, keep their rows).  A page id outside [0,
 * num_pages) gives slot -1 and SAW_ERR_DEVICE_INDEX (a free one is stored as
 * -1); so do more tokens than max_tokens (the rows behind are dropped).
 * page_size 16, 32 or 64; at most 65535 requests; num_pages * page_size and
 * max_blocks_per_seq * page_size below 2^31 (else SAW_ERR_UNSUPPORTED).  The
 * outputs must not overlap the inputs (src_tables aside).
 */
int32_t saw_build_tables(const int32_t* src_tables, int32_t num_src_rows, int32_t src_blocks,
                         const int32_t* src_rows, const int32_t* cached_lens,
                         const int32_t* new_lens, const int32_t* free_pages, int32_t max_free,
                         const int32_t* num_free, int32_t num_seqs, int32_t max_tokens,
                         int32_t num_pages, int32_t page_size, int32_t* block_tables,
                         int32_t max_blocks_per_seq, int32_t* seq_lens, int32_t* cu_q_lens,
                         int32_t* slot_mapping, int32_t* positions, int32_t* pages_taken,
                         int32_t* dev_status, void* stream);

/*
 * saw_rope_table -- the table that saw_rope_append reads: cos_sin[p][i] =
 * a cos(p w_i), cos_sin[p][rope_dim/2 + i] = a sin(p w_i), i < rope_dim/2, for
 * positions p < max_pos.  device float32 [max_pos][rope_dim], 16-byte aligned.
 * Build it once per model.
 *
 * w_i = base^(-2i/rope_dim), changed by `scaling` for contexts `factor` times
 * longer than the model's:
 *   SAW_ROPE_NONE    as it is
 *   SAW_ROPE_LINEAR  w_i / factor
 *   SAW_ROPE_NTK     base * factor^(rope_dim/(rope_dim-2)) for base
 *   SAW_ROPE_YARN    w_i for pairs that turn more than `high` times within
 *                    orig_max_pos positions, w_i / factor for those below
 *                    `low`, a linear ramp over the pair index between (its
 *                    ends rounded outwards); a = 0.1 ln(factor) + 1, or 1
 *                    for factor < 1
 *   SAW_ROPE_BANDS   the same ends, a linear ramp over the number of turns
 * low = high = 0 means 1 and 32 (YARN) or 1 and 4 (BANDS).  a is 1 except for
 * YARN; att_scale > 0 sets it.  w_i is a binary64: its 2^-52 moves the angle
 * of position p by p w_i 2^-52 radians, 2^-28 at 16 million positions.  Beside
 * that, values are within 2^-22 a of the true ones at every position.
 * rope_dim a multiple of 16, at most 256 (else SAW_ERR_UNSUPPORTED).
 */
#define SAW_ROPE_NONE 0
#define SAW_ROPE_LINEAR 1
#define SAW_ROPE_NTK 2
#define SAW_ROPE_YARN 3
#define SAW_ROPE_BANDS 4
int32_t saw_rope_table(float* cos_sin, int32_t max_pos, int32_t rope_dim, double base,
                       int32_t scaling, double factor, int32_t orig_max_pos, double low,
                       double high, float att_scale, void* stream);

/*
 * saw_rope_append -- rotary positions on q and k, then saw_quantize_append of
 * k and v, in one launch.
 *
 * q, k, v       device bfloat16 (binary16 with SAW_FMT_F16_INPUT)
 *               [num_tokens][heads][head_dim] with token strides in elements
 *               (multiples of 8, >= heads * head_dim): slices of a fused
 *               projection's output will do.  q may be NULL (or num_q_heads
 *               0): k and v only.  v may be NULL: q and k only.
 * positions     device int32 [num_tokens], each in [0, max_pos); a token with
 *               any other is skipped (q_out row too) and reported as
 *               SAW_ERR_DEVICE_INDEX.
 * cos_sin       device float32 [max_pos][rope_dim]: cosines of the
 *               rope_dim/2 pairs, then sines (saw_rope_table).
 * rope_dim      a multiple of 16 (else SAW_ERR_UNSUPPORTED), at most head_dim:
 *               the first rope_dim elements of a head are turned.
 * interleaved   0: pair i is elements (i, i + rope_dim/2); 1: (2i, 2i + 1).
 * q_out         [num_tokens][num_q_heads][head_dim], token stride
 *               q_out_token_stride; may be q itself with the same stride, and
 *               must not overlap q, k or v otherwise.
 * Other arguments as saw_quantize_append_ex.  A slot of -1 appends nothing;
 * the token's q is turned all the same.  Of two tokens with one slot either may
 * be stored, or codes of one with the scale of the other.  At most 65535 q-heads and kv-heads,
 * and 2^30 - 1 rows of q, k and v together (else SAW_ERR_UNSUPPORTED).
 *
 * Per pair, in binary32 with products rounded separately: y0 = x0 c - x1 s,
 * y1 = x1 c + x0 s.  k is not rounded in between: its binary32 values go into
 * the butterfly and the quantizer by saw_quantize_append's rule, so the bytes
 * are fully determined.  q_out is rounded once to the input type.
 */
int32_t saw_rope_append(const void* q, int64_t q_token_stride, const void* k,
                        int64_t k_token_stride, const void* v, int64_t v_token_stride,
                        const int32_t* positions, const float* cos_sin, int32_t max_pos,
                        int32_t rope_dim, int32_t interleaved, const int32_t* slot_mapping,
                        int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                        int32_t head_dim, void* q_out, int64_t q_out_token_stride, void* k_cache,
                        void* v_cache, int32_t num_pages, int32_t page_size, int32_t rotate_k,
                        int32_t rotate_v, int32_t block_h, int32_t formats, int32_t* dev_status,
                        void* stream);

/*
 * Workspace bytes of saw_prefix_decode_int4 for these sizes and `mode` on the
 * current device; 0 when it needs none or the sizes are bad.  Zero-fill a workspace
 * before its first use; each call leaves it ready for the next, of whatever
 * sizes (up to 131072 (sequence, kv-head) pairs; a larger batch wants one of
 * its own).  It is not one for the other decode calls, whose layouts differ.
 */
size_t saw_prefix_decode_workspace_bytes(int32_t num_seqs, int32_t num_groups,
                                         int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t page_size,
                                         int32_t max_prefix_len, int32_t max_own_len,
                                         int32_t mode);

/*
 * saw_prefix_decode_int4 -- saw_paged_decode_int4 for a batch in which groups
 * of neighbouring sequences share their first pages (a system prompt, a
 * document, samples of one prompt): the shared pages are read once per group
 * instead of once per sequence.
 *
 * cu_group_seqs device int32 [num_groups + 1], ascending: group g is sequences
 *               cu_group_seqs[g] .. cu_group_seqs[g+1] - 1.  A sequence in no
 *               group shares nothing.
 * prefix_lens   device int32 [num_groups]: the group's first prefix_lens[g]
 *               tokens are the same for all its sequences.  Whole pages count
 *               (the rest of the last page is read per sequence).  The table
 *               rows of the group's sequences that reach that far hold the same
 *               ids there (the caller's contract; any of them may be the one
 *               read; one that is idle or refused may hold anything).
 * seq_lens      device int32 [num_seqs]: all tokens, the prefix included.  0:
 *               an idle row, its output zero.  A length below the prefix's
 *               whole pages, beyond max_blocks_per_seq pages, or of more than
 *               max_own_len tokens behind the prefix, is reported as
 *               SAW_ERR_DEVICE_INDEX and treated as 0.
 * max_prefix_len, max_own_len  host bounds on prefix_lens and on the tokens
 *               behind a prefix's whole pages (for a sequence in no group: on
 *               its length).  max_blocks_per_seq pages must hold max_prefix_len.
 * out           [num_seqs][num_q_heads][128]: float32, or with
 *               SAW_FMT_OUT_INPUT in `formats` the input type (one rounding).
 * workspace     saw_prefix_decode_workspace_bytes(...) bytes, 16-byte
 *               aligned, zero-filled before its first use.  Calls sharing one
 *               must be ordered (one stream).
 * mode          SAW_PREFIX_AUTO: by size, whichever should be faster (short
 *               prefixes and few sequences are not worth a pass of their own).
 *               It goes by the bounds given here, as if every sequence had a
 *               prefix of max_prefix_len; and as the two forms round
 *               differently, a row's last bits can change with the batch it is
 *               in.  SAW_PREFIX_SHARE, SAW_PREFIX_SEPARATE: always, never --
 *               for a caller that knows better, or wants one rounding.
 * formats       SAW_FMT_F16_INPUT, SAW_FMT_BF16_META, SAW_FMT_OUT_INPUT.
 *
 * Arithmetic of the prefix pass: scores to about 2^-22 of their terms (codes
 * exact, q' in two binary16 parts; a |q'| whose product with the softmax scale
 * and log2 e exceeds 4094 saturates), dequantized V and p rounded once to
 * binary16 (V beyond +-65504 saturates; p of 2^7 at the row's maximum, so a key
 * fainter than 2^-32 of the heaviest adds to the denominator only), sums and
 * softmax in binary32.  A sequence's result does not depend on which of its
 * splits ends first: the same call gives the same bits.
 *
 * A group with inconsistent entries -- out of range, descending, a prefix beyond
 * max_prefix_len, or reaching back over an earlier group's sequences -- is
 * reported as SAW_ERR_DEVICE_INDEX and shares nothing; the others do.  Other arguments and errors as saw_paged_decode_int4;
 * head_dim 128, at most 8 q-heads per kv-head and 65535 groups (else
 * SAW_ERR_UNSUPPORTED).
 */
#define SAW_FMT_OUT_INPUT 4
#define SAW_PREFIX_AUTO 0
#define SAW_PREFIX_SHARE 1
#define SAW_PREFIX_SEPARATE 2
int32_t saw_prefix_decode_int4(const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_tables, int32_t max_blocks_per_seq,
                               const int32_t* seq_lens, const int32_t* cu_group_seqs,
                               const int32_t* prefix_lens, int32_t num_groups, int32_t num_seqs,
                               int32_t max_prefix_len, int32_t max_own_len, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t head_dim, int32_t num_pages,
                               int32_t page_size, int32_t rotate_k, int32_t rotate_v,
                               int32_t block_h, float sm_scale, void* out, void* workspace,
                               size_t workspace_bytes, int32_t mode, int32_t formats,
                               int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * A sparse decode step: at long contexts a query attends over a few pages
 * that a cheap score picks for it, so that a step reads a summary of the cache
 * (1/17 to 1/65 of K) and the chosen pages instead of all of it.  A page is the block.
 * Models that norm q and k per head append with saw_norm_rope_append;
 * saw_page_summary keeps the mean key of every complete page, whichever call
 * appended it; saw_select_pages and saw_sparse_decode_int4 follow per layer.
 * ------------------------------------------------------------------------ */

/*
 * saw_norm_rope_append -- a norm of every q and k head, then saw_rope_append.
 *
 * q_weight, k_weight  device [head_dim], 16-byte aligned: gains of the input type, or of
 *               float32 with SAW_FMT_F32_WEIGHT in `formats`.  NULL: all 1
 *               (weight_offset is then not used).
 * weight_offset finite; added to every gain: 0, or 1 for gains kept as w - 1.
 * eps           at least 2^-100, finite.
 * q_out may be q itself, as in saw_rope_append, whose other arguments, limits
 * and errors hold.  v is not normed.
 *
 * Per row x of q or k, in binary32, each step rounded once: ss = the sum of
 * the squares by a binary tree over the element index (neighbours, then pairs
 * of neighbours, ...), r = 1 / sqrt(ss / head_dim + eps), y = (x r) g with g =
 * w + weight_offset (no second product without weights).  The whole head is normed, also
 * where only part of it is turned.  y is not rounded to 16 bits before the turn, and the
 * rest is saw_rope_append's rule, so the bytes are fully determined.  Squares have to be
 * within binary32.
 */
#define SAW_FMT_F32_WEIGHT 8
int32_t saw_norm_rope_append(const void* q, int64_t q_token_stride, const void* k,
                             int64_t k_token_stride, const void* v, int64_t v_token_stride,
                             const void* q_weight, const void* k_weight, float weight_offset,
                             float eps, const int32_t* positions, const float* cos_sin,
                             int32_t max_pos, int32_t rope_dim, int32_t interleaved,
                             const int32_t* slot_mapping, int32_t num_tokens, int32_t num_q_heads,
                             int32_t num_kv_heads, int32_t head_dim, void* q_out,
                             int64_t q_out_token_stride, void* k_cache, void* v_cache,
                             int32_t num_pages, int32_t page_size, int32_t rotate_k,
                             int32_t rotate_v, int32_t block_h, int32_t formats,
                             int32_t* dev_status, void* stream);

/*
 * Bytes of the summaries of one layer's pages: [num_pages][stride], stride =
 * num_kv_heads * (head_dim/2 + 4) rounded up to 16.  A page's summary holds
 * every kv-head's packed codes (head_dim/2 bytes each), then every kv-head's
 * {scale, zero} word, in the cache's metadata format; a row dequantizes as
 * code*scale + zero, like a cache row.  0 for a nonpositive argument.
 */
size_t saw_summary_bytes(int32_t num_pages, int32_t num_kv_heads, int32_t head_dim);

/*
 * saw_page_summary -- the mean key of every page that a step completed.  Call
 * it after the step's append (any of them), with the same lengths.
 *
 * seq_lens      device int32 [num_seqs]: cached tokens, the new ones included.
 * new_lens      device int32 [num_seqs]: tokens that the step appended, or NULL
 *               (all of them; a count above seq_lens counts as all too).
 * max_new_len   host bound on the smaller of the two; sizes the grid for every sequence, so
 *               that a long prompt beside many single tokens wants a call of its own.
 * summary       device, saw_summary_bytes(...), 16-byte aligned.  Summaries go by physical
 *               page, so forks of a sequence share them.
 * Pages floor((L - n) / page_size) to floor(L / page_size) - 1 of a sequence
 * are written; a page that is not full has no summary (and none is needed: the
 * last page is always taken).
 *
 * Per (page, kv-head): A_d = sum of code*scale, Z = sum of the zeros, each the
 * even tokens in order plus the odd tokens in order; mean_d = (A_d + Z) /
 * page_size; the row is quantized by saw_quantize_append's rule (unrotated: it
 * is in the cache's domain already).  Each step is one binary32 rounding, so the bytes are
 * fully determined.
 *
 * formats: SAW_FMT_BF16_META or 0.  A length below 0 or beyond
 * max_blocks_per_seq pages, or more new tokens than max_new_len: the sequence
 * is skipped and SAW_ERR_DEVICE_INDEX reported; so is a page id out of range.
 * head_dim 64, 128 or 256; page_size 16, 32 or 64; at most 65535 sequences and
 * kv-heads, and 2^30 pages x kv-heads of a step's sequence (else SAW_ERR_UNSUPPORTED).
 */
int32_t saw_page_summary(const void* k_cache, const int32_t* block_tables,
                         int32_t max_blocks_per_seq, const int32_t* seq_lens,
                         const int32_t* new_lens, int32_t num_seqs, int32_t max_new_len,
                         int32_t num_kv_heads, int32_t head_dim, int32_t num_pages,
                         int32_t page_size, void* summary, int32_t formats, int32_t* dev_status,
                         void* stream);

/*
 * saw_select_pages -- for each (sequence, kv-head), the pages that its queries
 * attend over: the first first_pages and the last last_pages, and of the
 * others those with the best scores, max_selected in all.  A sequence of at
 * most max_selected pages keeps them all.
 *
 * q             device bfloat16 (binary16 with SAW_FMT_F16_INPUT)
 *               [num_seqs][num_q_heads][head_dim], 16-byte aligned.
 * summary       saw_page_summary's, of every page but the last of each sequence.
 * max_seq_len   host bound on seq_lens; max_blocks_per_seq pages must hold it.  It sizes
 *               shared memory: a loose one leaves less room for other work.
 * last_pages    at least 1; first_pages + last_pages at most max_selected.
 * sel_tables    device int32 [num_seqs][num_kv_heads][max_selected]: physical
 *               ids from block_tables, in the order of the sequence, -1 behind
 *               the last: a block table per (sequence, kv-head).
 * sel_pages     the same as page numbers of the sequence, or NULL.
 * sel_lens      device int32 [num_seqs][num_kv_heads]: tokens in those pages.
 *
 * Per q-head: q' = H q / sqrt(h) by saw_quantize_append's butterfly (q itself with rotate_k
 * 0), qs = max|q'| / 127, m_d = round-half-even(q'_d (1/qs)) in -127 .. 127 (0 where qs is
 * below 2^-126); with the summary's codes n, scale s and zero z: score = qs (s (sum m n) +
 * z (sum m)), the largest over the kv-head's q-heads.  The sums are whole numbers and
 * exact, every other step one binary32 rounding, so the lists are fully determined: equal
 * scores (-0 and 0 are equal, a NaN counts as -infinity) go to the lower page.
 *
 * A length below 0 or above max_seq_len is treated as 0 (an empty list) and
 * reported as SAW_ERR_DEVICE_INDEX; a page id outside [0, num_pages) among
 * the scored pages scores -infinity and is reported; ids are passed on as they
 * are.  Outputs must not overlap inputs.
 * formats: SAW_FMT_F16_INPUT, SAW_FMT_BF16_META.  head_dim 64, 128 or 256;
 * page_size 16, 32 or 64; at most 8 q-heads per kv-head, 65535 sequences and
 * kv-heads and 262144 pages in max_seq_len (else SAW_ERR_UNSUPPORTED).
 */
int32_t saw_select_pages(const void* q, const void* summary, const int32_t* block_tables,
                         int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs,
                         int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads,
                         int32_t head_dim, int32_t num_pages, int32_t page_size, int32_t rotate_k,
                         int32_t block_h, int32_t max_selected, int32_t first_pages,
                         int32_t last_pages, int32_t* sel_tables, int32_t* sel_pages,
                         int32_t* sel_lens, int32_t formats, int32_t* dev_status, void* stream);

/*
 * Workspace bytes of saw_sparse_decode_int4 for these sizes on the current
 * device; 0 when it needs none or the sizes are bad.  Zero-fill a workspace
 * before its first use; each call leaves it ready for the next, of whatever
 * sizes (up to 131072 (sequence, kv-head) pairs; a larger batch wants one of
 * its own).  It is not one for the other decode calls, whose layouts differ.
 */
size_t saw_sparse_decode_workspace_bytes(int32_t num_seqs, int32_t num_q_heads,
                                         int32_t num_kv_heads, int32_t head_dim,
                                         int32_t page_size, int32_t max_sel_len);

/*
 * saw_sparse_decode_int4 -- saw_paged_decode_int4 with a list of pages per
 * (sequence, kv-head) instead of one per sequence.
 *
 * sel_tables    device int32 [num_seqs][num_kv_heads][max_selected] page ids
 *               (saw_select_pages, or the caller's own; a page listed twice
 *               counts twice).
 * sel_lens      device int32 [num_seqs][num_kv_heads]: tokens, all pages full
 *               but the last.  0: a zero output row for the kv-head's q-heads.
 * max_sel_len   host bound on sel_lens, at most max_selected * page_size.
 * out           [num_seqs][num_q_heads][head_dim]: float32, or with
 *               SAW_FMT_OUT_INPUT in `formats` the input type (one rounding).
 *               p*s have 22 bits, with a bfloat16 output of more than 4
 *               q-heads per kv-head 11: where those are too few, ask for float32.
 * workspace     saw_sparse_decode_workspace_bytes(...) bytes, 16-byte aligned.
 *               Calls sharing one must be ordered (one stream).
 * Other arguments and the errors as saw_paged_decode_int4_ex, and the arithmetic but
 * for p*s: as binary16 numbers they are times a power of two that follows the scales,
 * so that the error is the same for V of any size (bfloat16 scales 2^-43 to 2^75).
 */
int32_t saw_sparse_decode_int4(const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* sel_tables, int32_t max_selected,
                               const int32_t* sel_lens, int32_t num_seqs, int32_t max_sel_len,
                               int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                               int32_t num_pages, int32_t page_size, int32_t rotate_k,
                               int32_t rotate_v, int32_t block_h, float sm_scale, void* out,
                               void* workspace, size_t workspace_bytes, int32_t formats,
                               int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * BF16 baseline.  gist.science "SAW-INT4: System-Aware 4-Bit KV-Cache
 * Quantization for Real-World LLM Serving", s.4 measures SAW-INT4's serving
 * throughput against an unquantized BF16 KV cache.  These two calls are that
 * baseline at the kernel level: the same paging and split-K decode, over a
 * cache of bfloat16 rows, so that INT4 and BF16 can be timed side by side.
 *
 * Cache layout, per layer and tensor (K and V separately):
 *   [num_pages][num_kv_heads][page_size][head_dim] bfloat16, rows of 256 B
 *   (head_dim 128).  Token t of a sequence lives in page block_tables[b][t /
 *   page_size], row t % page_size.  Owned by the caller; 16-byte aligned.
 * ------------------------------------------------------------------------ */

/* Bytes of one BF16 cache tensor; 0 for a nonpositive size. */
size_t saw_bf16_cache_bytes(int32_t num_pages, int32_t page_size, int32_t num_kv_heads,
                            int32_t head_dim);

/*
 * saw_bf16_append -- copy the bfloat16 rows k[t][h][:] (and v, if not NULL)
 * to slot slot_mapping[t] of the BF16 cache, unchanged.  Argument meaning,
 * strides (in elements, multiples of 8), the -1 padding slot and the
 * out-of-range rule (skipped, SAW_ERR_DEVICE_INDEX in *dev_status) are those
 * of saw_quantize_append.  head_dim must be 128 and page_size 16, 32 or 64
 * (else SAW_ERR_UNSUPPORTED).  Asynchronous on `stream`.
 */
int32_t saw_bf16_append(const void* k, const void* v, int64_t k_token_stride,
                        int64_t v_token_stride, const int32_t* slot_mapping, int32_t num_tokens,
                        int32_t num_kv_heads, int32_t head_dim, void* k_cache, void* v_cache,
                        int32_t num_pages, int32_t page_size, int32_t* dev_status, void* stream);

/*
 * Bytes of device workspace saw_paged_decode_bf16 needs for this shape (its
 * own split plan: one CTA per SM, at least 1024 tokens per split); 0 if it
 * needs none or the shape is invalid.  Zero-fill it before its first use;
 * each call leaves it ready for the next.
 */
size_t saw_decode_bf16_workspace_bytes(int32_t num_seqs, int32_t num_q_heads,
                                       int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                                       int32_t max_seq_len);

/*
 * saw_paged_decode_bf16 -- out[b][h][:] = softmax(sm_scale * K_b q_bh) V_b
 * over the seq_lens[b] cached tokens of kv-head h / (num_q_heads /
 * num_kv_heads), K and V read from the BF16 cache (no rotation, no
 * quantization).  q: bfloat16 [num_seqs][num_q_heads][128]; out: float32,
 * same shape.  Other arguments, sequences of length 0 (output zero), the
 * device-side index and timeout reports, and the return codes are those of
 * saw_paged_decode_int4.  Asynchronous on `stream`.
 */
int32_t saw_paged_decode_bf16(const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables, int32_t max_blocks_per_seq,
                              const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                              int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                              int32_t num_pages, int32_t page_size, float sm_scale, float* out,
                              void* workspace, size_t workspace_bytes, int32_t* dev_status,
                              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SAW_INT4_H */

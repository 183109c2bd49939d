/*
 * bsattn.h -- C ABI of the GB300 (sm_103a) block-sparse attention library.
 *
 * Sources of the operations (page title, section):
 *   [BSA] "TileLang 块稀疏 Flash-Attention 内核实现与实战指南" (TileLang block-sparse
 *         Flash-Attention kernel guide): 3.1 top-k mask, 3.2 threshold mask, 4.1-4.7 the
 *         prefill kernel, 5 the reference check, 6.1-6.3 GQA varlen sparse decode and the
 *         split heuristic, 7 paged KV decode.
 *   [FA]  "使用 TileLang 实现 FlashAttention ... 完整实战指南" (TileLang FlashAttention
 *         guide): online softmax, bottom-right causal alignment when seq_kv > seq_q.
 *   [XA]  "XAttention 算法实现指南" (XAttention algorithm guide): block selection
 *         (find_blocks_chunked) and its worked example.
 *
 * Conventions for every call:
 *   - Pointers marked (device) are caller-owned device memory; (host) caller-owned host
 *     memory.  The library never allocates, frees or retains any of them.
 *   - Tensors are dense, row-major (last index fastest), with no padding between rows.
 *   - GPU calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *     stream).  The return value only reports host-side argument checks and launch
 *     errors; faults found on the device (a bounded wait that expired, an out-of-range
 *     block index) are OR-ed into the status word at the start of the workspace and are
 *     read (and cleared) with bsattn_get_device_status().
 *   - Workspaces must be zero-filled once before their first use; every call leaves them
 *     ready for the next call (counters are reset by the kernels themselves).  After a
 *     call reports BSATTN_ERR_TIMEOUT the workspace must be zero-filled again, but for the
 *     paged-serving calls at the end of this file.
 *   - Block size is 64 tokens (bsattn_prefill_bs also takes 128-token prefill masks);
 *     head dimension d is 64 or 128; dtype fp16 or bf16.
 */
#ifndef BSATTN_H_
#define BSATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BSATTN_F16 = 0, BSATTN_BF16 = 1 } bsattn_dtype;

typedef enum {
    BSATTN_OK = 0,
    BSATTN_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misaligned or too-small buffer */
    BSATTN_ERR_UNSUPPORTED = 2,  /* head dim / dtype / shape outside what is built */
    BSATTN_ERR_CUDA = 4,         /* a CUDA runtime / driver call failed */
    BSATTN_ERR_TIMEOUT = 8,      /* device: a bounded wait expired (the kernel bailed out) */
    BSATTN_ERR_BAD_INDEX = 16,   /* device: a block index past the sequence was skipped */
    BSATTN_ERR_NO_SPACE = 32     /* device: a request got no pages or slots (bsattn_paged_plan) */
} bsattn_status;

#define BSATTN_BLOCK 64

/* Human-readable name of a status value (or of an OR of device status bits). */
const char* bsattn_status_string(int status);

/* Library version string. */
const char* bsattn_version(void);

/*
 * Block-sparse attention forward (prefill) -- [BSA] 4.1-4.7.
 *
 * For every (batch b, head h, 64-row query block qb) only key blocks kb with
 * block_mask[b][h][qb][kb] != 0 are visited; when is_causal, only key positions
 * j <= i + (Sk - Sq) are visible to query position i (bottom-right alignment, [FA]); keys
 * j >= Sk are never visible.  Computes out_i = softmax_j(q_i . k_j / sqrt(d)) v_j over the
 * visible keys with an exp2 online softmax in fp32, P rounded to the input dtype for the
 * second product; a query row with no visible key gets exactly 0.
 *
 *   q           (device) [B, H, Sq, d]  dtype
 *   k, v        (device) [B, H, Sk, d]  dtype
 *   block_mask  (device) [B, H, ceil(Sq/64), ceil(Sk/64)] uint8, nonzero = visit
 *   out         (device) [B, H, Sq, d]  dtype, fully written (rows with no work = 0)
 *   workspace   (device) >= 256 bytes, zero-filled once, 16-byte aligned: scheduler counters
 *               and the status word.  With bsattn_prefill_workspace_size() bytes (64 MiB) and
 *               rows that can span 1024+ key blocks, a row visiting more than 96 key blocks is
 *               split into 64-block parts run by different CTAs and merged by log-sum-exp
 *               (2048 partial slots; rows that do not fit run whole, so results are
 *               bit-reproducible only while the slots suffice).
 * q, k, v, out must be 16-byte aligned.  Returns BSATTN_OK or an error status; Sk beyond
 * 4096 key blocks at d = 64, or 2672 key blocks (171008 keys) at d = 128, returns
 * BSATTN_ERR_UNSUPPORTED (the per-CTA shared memory holds each item's mask-row list).
 */
int bsattn_prefill(const void* q, const void* k, const void* v, const uint8_t* block_mask,
                   int is_causal, void* out, int B, int H, int Sq, int Sk, int d,
                   bsattn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * bsattn_prefill with a block mask of 64- or 128-token blocks -- [BSA] 4.1-4.7 with the
 * block size of [XA] "BSA (Block Sparse Attention)", block size requirement (the block-sparse
 * library that consumes XAttention's selection takes 128-token blocks only).
 *
 *   block_size  64 or 128 (else BSATTN_ERR_UNSUPPORTED)
 *   block_mask  (device) [B, H, ceil(Sq/block_size), ceil(Sk/block_size)] uint8: entry
 *               [qb][kb] != 0 makes query rows [qb*bs, qb*bs+bs) see keys [kb*bs, kb*bs+bs)
 *               (subject to the causal rule and to Sk, as in bsattn_prefill).
 * Every other argument, the result and the error behaviour are those of bsattn_prefill, which
 * is this call with block_size = 64.  The kernel works on 64-token tiles either way: a
 * 128-token entry stands for the four 64 x 64 tiles it covers.
 */
int bsattn_prefill_bs(const void* q, const void* k, const void* v, const uint8_t* block_mask,
                      int block_size, int is_causal, void* out, int B, int H, int Sq, int Sk,
                      int d, bsattn_dtype dtype, void* workspace, size_t workspace_bytes,
                      void* stream);

/* Workspace bytes that enable splitting long rows (256 bytes is the minimum). */
size_t bsattn_prefill_workspace_size(int B, int H, int Sq, int Sk);

/*
 * GQA variable-length sparse decode -- [BSA] 6.1-6.2.
 *
 * One query token per sequence.  Query head h reads kv head g = h / (Hq / Hkv).  The keys
 * of (b, g) are the union over the slots t of block_indices[b][g][:] with t >= 0 of the
 * tokens [64 t, 64 t + 64) clipped to cache_seqlens[b]; out[b][h] = softmax attention of
 * q[b][h] over those keys (exactly 0 when there are none).  The selected blocks of each
 * (b, g) are cut into num_splits contiguous slices ([BSA] 6.2: the first len % num_splits
 * slices get one extra block) processed by separate CTAs and merged by log-sum-exp.
 *
 *   q              (device) [B, Hq, d]            dtype
 *   k, v           (device) [B, Smax, Hkv, d]     dtype (BSHD)
 *   cache_seqlens  (device) [B] int32, each in [0, Smax]
 *   block_indices  (device) [B, Hkv, max_sel] int32; -1 = empty slot; valid entries are
 *                  distinct and < ceil(cache_seqlens[b] / 64), in any order.  Entries at or
 *                  past the sequence end are skipped and flagged BSATTN_ERR_BAD_INDEX.
 *   num_splits     >= 1, or 0 to let the library choose (bsattn_decode_default_splits)
 *   out            (device) [B, Hq, d] dtype
 *   workspace      (device) >= bsattn_decode_workspace_size(B, Hq, Hkv, d, max_sel, num_splits)
 *                  bytes, zero-filled once.
 * Requires Hq % Hkv == 0, 1 <= Hq / Hkv <= 8, d in {64, 128}; q, k, v, out 16-byte aligned.
 */
int bsattn_decode_varlen(const void* q, const void* k, const void* v,
                         const int32_t* cache_seqlens, const int32_t* block_indices,
                         int num_splits, void* out, int B, int Hq, int Hkv, int Smax, int d,
                         int max_sel, bsattn_dtype dtype, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * bsattn_decode_varlen without a workspace argument, for callers that cannot allocate
 * device memory when they attend (code running inside a custom allocator or memory pool,
 * runtimes that forbid allocation after start-up, hosts that only pass pointers to buffers
 * they own).  The pages have no counterpart: this is a deployment variant of the decode
 * above, with the same arguments (minus the workspace) and the same results.
 *
 * Its scratch is one fixed 8 MiB device array inside the library (held by every GPU that
 * loads the library until the process exits); shapes whose decode workspace
 * (bsattn_decode_workspace_size) exceeds it return BSATTN_ERR_UNSUPPORTED.  It allocates
 * nothing: no cudaMalloc / cudaFree, no allocating library routine.  The first call on a
 * device looks up the array's device address (cudaGetSymbolAddress) with that device
 * current; make that first call before any stream capture.  CUDA loads a library's device
 * code lazily by default, and that first call is also what loads this file's code and
 * reserves the array on the device: make one call per device before entering a context
 * that must not allocate (or run with CUDA_MODULE_LOADING=EAGER).  `stream` must belong to
 * the current device (else BSATTN_ERR_INVALID_ARG).  Each call clears the array's status
 * word and merge tickets with cudaMemsetAsync on `stream`.  All calls share the array, so
 * calls that overlap on the GPU (different streams, or threads) race and must be serialised
 * by the caller.  Device-detected conditions (a skipped out-of-range index, an expired
 * wait) go to the array's status word: read them with bsattn_decode_noalloc_status.
 */
int bsattn_decode_varlen_noalloc(const void* q, const void* k, const void* v,
                                 const int32_t* cache_seqlens, const int32_t* block_indices,
                                 int num_splits, void* out, int B, int Hq, int Hkv, int Smax,
                                 int d, int max_sel, bsattn_dtype dtype, void* stream);

/*
 * Reads and clears the device status word of bsattn_decode_varlen_noalloc on the current
 * device, after synchronising `stream` (which must belong to that device, else
 * BSATTN_ERR_INVALID_ARG).  Each allocation-free call clears the word when it starts, so the
 * result is the OR of the BSATTN_ERR_* bits (BSATTN_ERR_BAD_INDEX, BSATTN_ERR_TIMEOUT) that
 * the most recent call recorded (0 = none), or BSATTN_ERR_CUDA if the read itself failed.
 * It allocates nothing: a 4-byte copy into a host word.
 */
int bsattn_decode_noalloc_status(void* stream);

/*
 * GQA varlen sparse decode, block-mask form -- [BSA] 6 (the `_mask` example).  Identical to
 * bsattn_decode_varlen except that the selected blocks of (b, g) are given as
 *   block_mask (device) [B, Hkv, num_blocks] uint8, nonzero = block j selected;
 * slot j of the mask is block j, and the num_blocks slots are cut into num_splits slices as in
 * [BSA] 6.2.  Set entries at or past the sequence end select no tokens (not flagged).
 * Workspace: bsattn_decode_workspace_size(B, Hq, Hkv, d, num_blocks, num_splits) bytes.
 */
int bsattn_decode_varlen_mask(const void* q, const void* k, const void* v,
                              const int32_t* cache_seqlens, const uint8_t* block_mask,
                              int num_splits, void* out, int B, int Hq, int Hkv, int Smax, int d,
                              int num_blocks, bsattn_dtype dtype, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * GQA varlen sparse decode over a paged KV cache -- [BSA] 7.  As bsattn_decode_varlen, but
 *   k_pages, v_pages (device) [num_pages, page_size, Hkv, d] dtype
 *   block_table      (device) [B, max_pages_per_seq] int32: logical page p of sequence b is
 *                    physical page block_table[b][p]
 * Logical token position P of sequence b lives in page block_table[b][P / page_size], row
 * P % page_size.  page_size must be a multiple of 64 (a 64-token block never straddles two
 * pages; [BSA] 7 asserts the same).  Blocks whose page is out of range are skipped and flagged
 * BSATTN_ERR_BAD_INDEX.  Workspace as for bsattn_decode_varlen.
 */
int bsattn_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                        const int32_t* cache_seqlens, const int32_t* block_indices,
                        const int32_t* block_table, int num_splits, void* out, int B, int Hq,
                        int Hkv, int num_pages, int page_size, int max_pages_per_seq, int d,
                        int max_sel, bsattn_dtype dtype, void* workspace, size_t workspace_bytes,
                        void* stream);

/* Workspace bytes bsattn_decode_varlen needs (num_splits 0 = the library's choice). */
size_t bsattn_decode_workspace_size(int B, int Hq, int Hkv, int d, int max_sel, int num_splits);

/*
 * The split count bsattn_decode_varlen uses when num_splits == 0: the decode is bound by HBM
 * bandwidth, so it takes as many splits as fill exactly one wave of resident CTAs (resident
 * CTAs per SM for head dim d x num_sms, divided over the B * Hkv groups), capped by max_sel
 * and 64.  num_sms <= 0 queries the current device.
 */
int bsattn_decode_default_splits(int B, int Hkv, int max_sel, int d, int num_sms);

/*
 * The split-count rule of [BSA] 6.3, bit-exact: if total_mblocks >= 0.8 num_SMs return 1
 * (or, when one kv head exceeds the assumed 50 MB L2, num_m_blocks > 2 num_SMs and not
 * causal/local, ceil(size / L2) capped at max_splits); if num_n_blocks <= 4 return 1;
 * otherwise the smallest s in [1, min(max_splits, num_SMs, num_n_blocks)] whose wave
 * efficiency w / ceil(w), w = total_mblocks s / num_SMs, is >= 0.85 of the best.
 * Pure host function.
 */
int bsattn_num_splits_heuristic(int total_mblocks, int num_SMs, int num_n_blocks,
                                int num_m_blocks, long long size_one_kv_head,
                                int is_causal_or_local, int max_splits);

/*
 * Host-side block-mask builders -- [BSA] 3.1 and 3.2.  scores (host) fp32
 * [B, H, nq, nk]; mask_out (host) uint8 of the same shape, fully written with 0 / 1.
 *   top-k:     per row keep the min(topk, nk) highest scores (ties: lower column first).
 *   threshold: keep score > threshold (strict).
 * Then, if use_dense_for_last_block, the last min(2, nq) rows are set all-1; then, if
 * apply_tril, entries with column > row are cleared.  NaN scores -> BSATTN_ERR_INVALID_ARG.
 */
int bsattn_mask_from_topk(const float* scores, int B, int H, int nq, int nk, int topk,
                          int use_dense_for_last_block, int apply_tril, uint8_t* mask_out);
int bsattn_mask_from_threshold(const float* scores, int B, int H, int nq, int nk,
                               float threshold, int use_dense_for_last_block, int apply_tril,
                               uint8_t* mask_out);

/*
 * Cumulative-threshold block mask -- [XA] "block selection (find_blocks_chunked)".  attn_sum
 * (host) fp32 [B, H, nq, nk] holds per (query block, key block) attention weight sums.  Per
 * row: block 0 (the sink) is kept and, when causal, the diagonal block i (if i < nk); the other
 * blocks are visited from the largest weight down (ties: lower column first) and taken while
 * the sum of the weights already taken is below threshold * (row total), so the block whose
 * addition reaches the threshold is taken too.  Sums are in double, left to right.
 * mask_out (host) uint8 [B, H, nq, nk].  NaN weights -> BSATTN_ERR_INVALID_ARG.
 */
int bsattn_mask_from_cumulative_threshold(const float* attn_sum, int B, int H, int nq, int nk,
                                          double threshold, int causal, uint8_t* mask_out);

/*
 * ---------------------------------------------------------------------------------------------
 * Paged serving: a page plan, a 4-bit cache, and attention with a sliding window.  The calls below
 * have no counterpart in the pages; their definitions are given in full here.
 *
 * Their workspaces: the plan, append, gather and window prefill use only the status word (256 bytes,
 * 16-byte aligned); they set bits of it and read nothing, so calls may share one (the status is then
 * that of all of them).  The stream decodes
 * (bsattn_decode_window, bsattn_decode_window_paged, bsattn_decode_paged_kv4) also keep merge tickets
 * and partial results in theirs: its first 4352 bytes must be zero before the first use, any shapes
 * may follow one another on it, and calls that can overlap on the GPU (streams, replayed graphs) need
 * one each.  A stream decode that reports BSATTN_ERR_TIMEOUT leaves its tickets at zero too (the
 * workspace need not be zero-filled again), and every row that lacks some of its tokens is NaN.
 */

/*
 * Block-table rows and slot map of a step, from request lengths.  Sequence b holds cached_lens[b]
 * tokens and brings new_lens[b]; the new tokens of all sequences are packed in that order.
 *
 *   cached_lens, new_lens  (device) [B] int32
 *   free_pages   (device) [free_capacity] int32: the first *free_count entries are free pages; they
 *                are taken from the end, in the order of the sequences
 *   free_count   (device) int32
 *   block_table  (device) [B, max_pages_per_seq] int32, updated: the entries of new pages are written,
 *                all others are left as they were
 *   slots        (device) [max_tokens] int64, fully written: page * page_size + row of each packed
 *                token's place, -1 for a token that got none and past the last token
 *   starts       (device) [B + 1] int32: starts[b] = new_lens[0] + ... + new_lens[b - 1] (sums past
 *                INT32_MAX stay there)
 *   seqlens      (device) [B] int32: cached_lens[b] + new_lens[b], or cached_lens[b] if not served
 *   free_left    (device) int32: the free pages that remain
 * A sequence is not served (no page, slots -1, BSATTN_ERR_NO_SPACE in the status word) if its table
 * row or `slots` is too short for it, or if it needs pages and those asked for up to and including it
 * exceed *free_count.  A negative length is not served and counts as 0 tokens (BSATTN_ERR_BAD_INDEX);
 * a token whose page is mapped to a negative number gets slot -1 (BSATTN_ERR_BAD_INDEX).  No output
 * may overlap another output or an input (BSATTN_ERR_INVALID_ARG), so that a call can be repeated.
 * page_size >= 1; B <= 8192 (else BSATTN_ERR_UNSUPPORTED).
 */
int bsattn_paged_plan(const int32_t* cached_lens, const int32_t* new_lens, const int32_t* free_pages,
                      const int32_t* free_count, int32_t* block_table, int64_t* slots, int32_t* starts,
                      int32_t* seqlens, int32_t* free_left, int B, int page_size, int max_pages_per_seq,
                      int free_capacity, int max_tokens, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * The 4-bit cache.  16 consecutive channels of a token's head are a group; a group is 16 e2m1 codes
 * c_i and one e4m3 scale s and stands for the values e2m1(c_i) * s * unit, where the unit (k_scale for
 * all keys, v_scale for all values) is a power of two in [2^-16, 2^16].
 *
 *   k_codes, v_codes    (device) [num_pages, Hkv, page_size, d / 2] uint8: channel 2 i in the low half
 *                       of byte i, channel 2 i + 1 in the high half
 *   k_scales, v_scales  (device) [num_pages, Hkv, page_size, d / 16] uint8
 * all 16-byte aligned.  Writing x: s = e4m3(max |x| / (6 unit)), c = e2m1(x / (s unit)), each rounded to
 * nearest with ties to even and saturated (448, 6), c = 0 where s = 0 and for every value that rounds to
 * 0; the bytes are those of exact arithmetic.  A group with an infinity or a NaN gets the NaN scale 0x7f and reads as NaN.
 *
 * Append rounds T rows of k and v, (device) [T, Hkv, d] dtype with contiguous channels and the given
 * strides (elements, multiples of 8; any value for a dimension of one entry), into the rows that
 * slots (device) [T] int64 names.  Negative slots are skipped; slots at or past num_pages * page_size
 * are skipped and flagged BSATTN_ERR_BAD_INDEX; the others must be distinct.  Other rows are not
 * touched.  Gather writes the rows that slots names to k and v, (device) [T, Hkv, d] dtype, dense,
 * rounded to nearest; a skipped slot gives zeros, a slot may be named more than once.
 */
int bsattn_kv4_append(const void* k, const void* v, long long k_token_stride, long long k_head_stride,
                      long long v_token_stride, long long v_head_stride, const int64_t* slots,
                      uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales,
                      float k_scale, float v_scale, int T, int Hkv, int num_pages, int page_size, int d,
                      bsattn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);
int bsattn_kv4_gather(const int64_t* slots, const uint8_t* k_codes, const uint8_t* k_scales,
                      const uint8_t* v_codes, const uint8_t* v_scales, float k_scale, float v_scale,
                      void* k, void* v, int T, int Hkv, int num_pages, int page_size, int d,
                      bsattn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One query token per sequence over the paged 4-bit cache.  As bsattn_decode_paged: query head h of
 * sequence b attends to kv head h / (Hq / Hkv) over the visible ones of its cache_seqlens[b] tokens,
 * out = softmax(q . k / sqrt(d)) v, 0 where nothing is visible.  Visible are
 *   - with block_indices (device) [B, Hkv, max_sel] int32: the tokens of the chosen 64-token blocks
 *     (-1 = empty slot, distinct, any order; a block at or past the end is skipped and flagged
 *     BSATTN_ERR_BAD_INDEX); window must be 0;
 *   - with block_indices NULL and window > 0: token j with j < sinks or j >= cache_seqlens[b] - window;
 *   - with block_indices NULL and window 0: every token.
 * q, out (device) [B, Hq, d] dtype; block_table as in bsattn_decode_paged, page_size a multiple of 64.
 * Tokens on pages out of range, and any past the table, are skipped and flagged BSATTN_ERR_BAD_INDEX;
 * a negative length is flagged and taken as 0.  Masked tokens and rows past the end may hold anything.
 * The products run in fp16 with 32-bit sums: cache values are exact there, weights are rounded to fp16.
 * Requires Hq % Hkv == 0, Hq / Hkv <= 8, Hkv <= 1024, d in {64, 128}.  out may be q itself; otherwise it
 * shares no memory with q or the cache (BSATTN_ERR_INVALID_ARG).  The result does not depend on the
 * order in which CTAs run.
 */
int bsattn_decode_paged_kv4(const void* q, const uint8_t* k_codes, const uint8_t* k_scales,
                            const uint8_t* v_codes, const uint8_t* v_scales, float k_scale, float v_scale,
                            const int32_t* cache_seqlens, const int32_t* block_indices,
                            const int32_t* block_table, int window, int sinks, void* out, int B, int Hq,
                            int Hkv, int num_pages, int page_size, int max_pages_per_seq, int d,
                            int max_sel, bsattn_dtype dtype, void* workspace, size_t workspace_bytes,
                            void* stream);
size_t bsattn_decode_kv4_workspace_size(int Hq, int Hkv, int d);

/*
 * Sliding-window decode with sinks over a 16-bit cache: as bsattn_decode_varlen (contiguous k, v
 * [B, Smax, Hkv, d]) and bsattn_decode_paged ([num_pages, page_size, Hkv, d] and a block table), with
 * token j of sequence b visible iff j < cache_seqlens[b] and (j < sinks or j >= cache_seqlens[b] -
 * window), window >= 1.  A length past Smax is flagged BSATTN_ERR_BAD_INDEX and taken as Smax; bad
 * lengths and pages otherwise as in bsattn_decode_paged_kv4, and the same limits.
 */
int bsattn_decode_window(const void* q, const void* k, const void* v, const int32_t* cache_seqlens,
                         int window, int sinks, void* out, int B, int Hq, int Hkv, int Smax, int d,
                         bsattn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);
int bsattn_decode_window_paged(const void* q, const void* k_pages, const void* v_pages,
                               const int32_t* cache_seqlens, const int32_t* block_table, int window,
                               int sinks, void* out, int B, int Hq, int Hkv, int num_pages, int page_size,
                               int max_pages_per_seq, int d, bsattn_dtype dtype, void* workspace,
                               size_t workspace_bytes, void* stream);
size_t bsattn_decode_window_workspace_size(int Hq, int Hkv, int d);

/*
 * Causal attention with a sliding window and sinks, forward.  Query row i of Sq stands at position
 * p = i + (Sk - Sq) and sees key j iff j <= p and (j < sinks or j > p - window); query head h reads kv
 * head h / (Hq / Hkv); out_i = softmax_j(q_i . k_j / sqrt(d)) v_j, 0 for a row that sees no key
 * (and for one all of whose scores are -infinity; so in the decodes above).
 *
 *   q, out   (device) [B, Hq, Sq, d] dtype;  k, v (device) [B, Hkv, Sk, d] dtype; 16-byte aligned
 *   strides  (host) 12 element strides: batch, head, row of q, of k, of v, of out (positive multiples
 *            of 8, out's at least d; any value for a dimension of one entry), or NULL for dense tensors
 * window >= 1, sinks >= 0, d in {64, 128}, any Hq % Hkv == 0.  P is rounded to dtype before the second
 * product.  What stands at keys that a row does not see has no effect on it, infinities and NaN
 * included; a row that sees one in v may be NaN in every channel.  (Rows that share a 128-key tile with
 * one that they do not see are worked out again, which takes longer.)  out may be q itself, with q's
 * strides; otherwise its rows share no memory with q, k, v or one another (BSATTN_ERR_INVALID_ARG).  The
 * wait budget is that of an item (128 or 256 rows), not of the whole call.
 */
int bsattn_prefill_window(const void* q, const void* k, const void* v, int window, int sinks, void* out,
                          int B, int Hq, int Hkv, int Sq, int Sk, int d, const int64_t* strides,
                          bsattn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * ---------------------------------------------------------------------------------------------
 * Choosing key blocks on the GPU.  The summary of a block of up to 64 rows is its mean in 8 bits: the rows'
 * 32-bit sum, taken in halves (row i + row i + 32, then i + 16, ... i + 1, absent rows being 0), divided by
 * their number; scale = max |mean| / 127 and code_c = mean_c / scale, each quotient rounded to nearest in 32
 * bits, the code then to a whole number (ties to even, at most 127 in magnitude; 0 where the scale is 0).  A
 * mean with a channel that is not finite has codes 0 and scale +infinity.  A query or a query block is
 * summarised likewise (one row, or the block's).
 * The score of a key block for query summaries h = 1 .. G is
 *     (max_h ((sum_c code_hc code_c) scale_h)) scale,
 * a whole number, exact, times two factors, each product rounded to nearest in 32 bits; +infinity where
 * the key's scale is, and a query whose own scale is infinite counts as scale 0.  Nothing in it depends on the
 * order of additions, and of blocks with equal scores the lower one comes first: a choice is the same
 * wherever and however it is made.  These calls have no counterpart in the pages; the block scores stand for
 * the given ones of bsattn_mask_from_topk.
 */

/*
 * Summarises again, for every sequence b, each 64-token block that holds one of its last new_lens[b] tokens,
 * from the rows in the cache (so tokens are appended first, in one step or in many).
 *
 *   k_pages        (device) [num_pages, page_size, Hkv, d] dtype, as in bsattn_decode_paged; page_size a
 *                  multiple of 64
 *   cache_seqlens  (device) [B] int32: lengths with the new tokens;  new_lens (device) [B] int32
 *   block_table    (device) [B, max_pages_per_seq] int32
 *   codes          (device) [num_pages, page_size / 64, Hkv, d] int8, updated
 *   scales         (device) [num_pages, page_size / 64, Hkv] fp32, updated
 * k_pages, codes and scales 16-byte aligned.  Entries of other blocks are left as they were; rows past a
 * sequence's end have no effect.  Blocks on pages out of range and lengths past the table are skipped, a
 * negative length or new_lens[b] counts as 0, one past the length as the length; all are flagged
 * BSATTN_ERR_BAD_INDEX.  Sequences that share a block must agree about its rows.  codes and scales share no
 * memory with the inputs (BSATTN_ERR_INVALID_ARG).  Workspace: a status word (256 bytes), as for the plan.
 */
int bsattn_index_update(const void* k_pages, const int32_t* cache_seqlens, const int32_t* new_lens,
                        const int32_t* block_table, int8_t* codes, float* scales, int B, int Hkv, int num_pages,
                        int page_size, int max_pages_per_seq, int d, bsattn_dtype dtype, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * The key blocks of one query token per sequence, for bsattn_decode_paged and bsattn_decode_paged_kv4 (or,
 * with a table of consecutive pages, bsattn_decode_varlen): for sequence b and kv head g the first `sinks` and
 * the last `recent` blocks of its cache_seqlens[b] tokens, then those with the highest scores for its
 * G = Hq / Hkv query heads, max_sel in all or as many as there are.
 *
 *   q              (device) [B, Hq, d] dtype;  codes, scales, block_table as above
 *   block_indices  (device) [B, Hkv, max_sel] int32, fully written: the chosen blocks in rising order, then -1
 * sinks + recent <= max_sel (else BSATTN_ERR_INVALID_ARG).  Blocks on pages out of range are not chosen, a
 * length past the table is taken as the table's, a negative one as 0; all are flagged BSATTN_ERR_BAD_INDEX.
 * Requires Hq / Hkv <= 8, d in {64, 128}, max_pages_per_seq * page_size <= 3000000.  block_indices shares no
 * memory with the inputs.  Workspace: a status word.
 */
int bsattn_decode_select(const void* q, const int8_t* codes, const float* scales, const int32_t* cache_seqlens,
                         const int32_t* block_table, int sinks, int recent, int32_t* block_indices, int B, int Hq,
                         int Hkv, int num_pages, int page_size, int max_pages_per_seq, int d, int max_sel,
                         bsattn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * A block mask for bsattn_prefill from the summaries of q's and k's 64-row blocks (of the rows there are, at the
 * end).  Query block r sees the key blocks up to that of its last row's position min(64 r + 63, Sq - 1) + Sk -
 * Sq (bottom-right alignment), or all of them if not is_causal.  Of these it gets the first `sinks` and the last
 * `recent`, then those with the highest scores until it has topk (forced blocks stay, however many), or all of
 * them if use_dense_for_last_block and r is one of the last two.  Under the causal rule `recent` 1 is the
 * diagonal block; where Sk - Sq is not a multiple of 64 a block's rows begin in the block before it, and 2 has
 * all of them see themselves.
 *
 *   q         (device) [B, Hq, Sq, d] dtype;  k (device) [B, Hkv, Sk, d] dtype; 16-byte aligned.  Query head h
 *             is scored against kv head h / (Hq / Hkv)
 *   strides   (host) 6 element strides: batch, head, row of q, of k (multiples of 8, not negative; any value
 *             for a dimension of one entry; channels contiguous), or NULL for dense tensors
 *   mask_out  (device) [B, Hq, ceil(Sq/64), ceil(Sk/64)] uint8, fully written with 0 / 1
 *   workspace (device) >= bsattn_mask_from_qk_workspace_size bytes, 16-byte aligned; need not be zero-filled.
 *             Calls that can overlap on the GPU need one each.
 * d in {64, 128}; Sk <= 450560 (else BSATTN_ERR_UNSUPPORTED).  mask_out and workspace share no memory with one
 * another, q or k (BSATTN_ERR_INVALID_ARG).
 */
int bsattn_mask_from_qk(const void* q, const void* k, int topk, int sinks, int recent,
                        int use_dense_for_last_block, int is_causal, uint8_t* mask_out, int B, int Hq, int Hkv,
                        int Sq, int Sk, int d, const int64_t* strides, bsattn_dtype dtype, void* workspace,
                        size_t workspace_bytes, void* stream);
size_t bsattn_mask_from_qk_workspace_size(int B, int Hq, int Hkv, int Sq, int Sk, int d);

/*
 * One query token per sequence over a prefix that sequences share and the sequence's own tokens after it, from a
 * 16-bit paged cache: out = softmax(q . k / sqrt(d)) v over both.  The prefix is read once for all the
 * sequences that share it (for 256 query rows of a kv head at a time), not once for each.
 *
 *   q, out         (device) [B, Hq, d] dtype;  k_pages, v_pages (device) [num_pages, page_size, Hkv, d] dtype
 *   prefix_lens    (device) [P] int32: tokens of prefix p, any number
 *   prefix_table   (device) [P, max_pages_per_prefix] int32: its pages
 *   group_starts   (device) [P + 1] int32: sequences group_starts[p] .. group_starts[p + 1] - 1 share prefix p;
 *                  rising from 0 to B
 *   cache_seqlens  (device) [B] int32: a sequence's own tokens, which may be none
 *   block_table    (device) [B, max_pages_per_seq] int32: their pages
 * No visible token gives 0.  Tokens on pages out of range, and any past a table, are skipped, a negative length
 * is taken as 0; these and group_starts that do not rise from 0 to B are flagged BSATTN_ERR_BAD_INDEX (the
 * rows of groups that overlap or run backwards are then undefined; a sequence outside all groups has no prefix).
 * Rows past a length may hold anything.  P is rounded to dtype before the second product.  A wait that expires
 * makes every row NaN that lacks some of its tokens.  The result does not depend on the order in which CTAs run.
 * P >= 1, Hq / Hkv <= 8, Hkv <= 1024, d in {64, 128}, page_size a multiple of 64, at most 2^30 tokens a prefix or
 * sequence.  out may be q itself; otherwise it shares no memory with q or the cache.  Workspace:
 * bsattn_decode_shared_workspace_size bytes, 16-byte aligned; its first 256 bytes are the status word's, the rest
 * need not be zero and serves any shape that fits.  Calls that can overlap on the GPU need one each.
 */
int bsattn_decode_shared(const void* q, const void* k_pages, const void* v_pages, const int32_t* prefix_lens,
                         const int32_t* prefix_table, const int32_t* group_starts, const int32_t* cache_seqlens,
                         const int32_t* block_table, void* out, int B, int P, int Hq, int Hkv, int num_pages,
                         int page_size, int max_pages_per_prefix, int max_pages_per_seq, int d, bsattn_dtype dtype,
                         void* workspace, size_t workspace_bytes, void* stream);
size_t bsattn_decode_shared_workspace_size(int B, int P, int Hq, int Hkv, int d);

/*
 * Reads and clears the device status word at the start of `workspace` (device), after
 * synchronising `stream`.  Returns the OR of the BSATTN_ERR_* bits the kernels recorded
 * since the last read (0 = none), or BSATTN_ERR_CUDA if the read itself failed.  Only the
 * bits returned are cleared: one that a call on another stream sets meanwhile is returned
 * by the next read.  Where several calls share a workspace a bit may be of any of them.
 */
int bsattn_get_device_status(void* workspace, void* stream);

/*
 * Makes the paged-serving calls that this host thread makes from now on record what their kernels
 * find in the 4 bytes at `word` (memory of the device they run on, 16-byte aligned, zero; read like a
 * workspace's) and not at the start of their workspace; NULL ends that.  For calls captured into a graph whose workspace
 * is not the caller's to read afterwards.
 */
int bsattn_set_status_word(void* word);

/*
 * Budget, in nanoseconds, of every bounded wait inside the kernels launched after this
 * call (default 2e9).  Exists so tests can make a wait expire on purpose and check that
 * the kernel reports BSATTN_ERR_TIMEOUT and leaves the context usable.  It runs from the
 * start of the wait in the stream decodes, of the item in bsattn_prefill_window, of the
 * CTA in the other kernels.
 */
void bsattn_set_wait_budget_ns(unsigned long long ns);

#ifdef __cplusplus
}
#endif

#endif /* BSATTN_H_ */

/*
 * sls.h - C ABI of the GB300 sparse decode-attention library (libsls.so).
 *
 * One decode step of sparse long-context attention:
 *
 *   select   sls_select_pages   Quest-style page bound + per-KV-head top-k
 *            sls_select_delta   2-bit thumbnail scan + top-delta
 *   attend   sls_sparse_decode_attend   split-K online softmax over the
 *                                       selected pages (flash-decoding)
 *   combine  sls_combine_splits         log-sum-exp merge of the splits,
 *                                       with the optional sink
 *
 * plus the selector metadata kept next to the KV cache (page min/max keys,
 * 2-bit thumbnails), built in bulk or updated on append; and, around a cache
 * held in 8 bits, what fills, reads and bounds it:
 *
 *   sls_qk_norm_rope        per-head norm and rotation of the projected heads
 *   sls_kv8_append          tokens into the 8-bit cache
 *   sls_kv8_decode_attend   decode attention over it, dense or over page lists
 *   sls_kv8_evict           the blocks with the most attention weight kept
 *
 * and a cache whose pages lie in a pool, handed out as sequences grow:
 *
 *   sls_paged_append         tokens into pages taken from the pool
 *   sls_paged_select_pages   page bound + top-k over the pool's summaries
 *   sls_paged_decode_attend  decode attention, dense or over page lists
 *   sls_paged_fork           sequences shared, reordered, cut and freed
 *   sls_paged_compact        the pool's used pages moved to its front
 *
 * Conventions shared by every call
 * --------------------------------
 * - Every pointer argument is a DEVICE pointer owned by the caller, unless
 *   stated otherwise.  The library allocates no memory; scratch comes from a
 *   caller buffer whose size a *_workspace_size() call reports.
 * - Queries, K/V caches, page metadata (kmin/kmax), thumbnail codes, scales
 *   and residuals, appended keys/values and split partials (o_part) are read
 *   in 16-byte vectors: their pointers must be 16-byte aligned, or the call
 *   fails with SLS_EINVAL before launching anything.
 * - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *   stream).  Calls only enqueue work: they never synchronise the device
 *   and never read device memory from the host, so they can be captured in
 *   a CUDA graph.
 * - Every call returns an sls_status.  Arguments are validated on the host
 *   before anything is launched; on error nothing is enqueued and
 *   sls_last_error() describes the problem (thread-local string).
 * - KV cache layout: K and V are [B, Hkv, Cap, D] row-major, element type
 *   desc->dtype.  Row r = b*Hkv + h of the cache is the contiguous slice of
 *   request (b, kv head h); seen as a page pool it holds Cap/P pages of P
 *   tokens, page p covering positions [p*P, p*P+P) ("perf(core): fused
 *   sparse-attention decode via page indirection", section "The reduction":
 *   a dense [B, H, Cap, D] allocation viewed as a pool by a pure reshape,
 *   with the KV-head axis folded into the request axis).
 * - Query heads: q is [B, Hq, D]; query head hq belongs to KV head
 *   hq / (Hq/Hkv) (grouped-query attention), and every page list is shared
 *   by the G = Hq/Hkv query heads of its KV head.
 * - ctx_len[b] is the number of valid positions of sequence b; positions
 *   >= ctx_len[b] are never read by selection and never attended.  Values
 *   outside [0, Cap] are clamped to that range on the device.
 * - Page indices in page lists are LOGICAL page numbers within the row
 *   (0 .. Cap/P - 1); -1 marks an empty slot that is skipped.
 */
#ifndef SLS_H
#define SLS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
typedef int sls_status;
#define SLS_OK            0
#define SLS_EINVAL       -1  /* null pointer, bad size or out-of-range parameter */
#define SLS_EUNSUPPORTED -2  /* valid but unsupported combination (dtype, D, G, P) */
#define SLS_EOVERFLOW    -3  /* a size product overflows the index range */
#define SLS_EWORKSPACE   -4  /* workspace missing or too small */
#define SLS_ECUDA        -5  /* a CUDA launch or attribute call failed */
#define SLS_ETIMEOUT     -6  /* a pipelined kernel gave up waiting for its own copies */
#define SLS_EDEVICE      -7  /* a kernel met page-list entries it could not use (skipped) */

/* ---- element types ----------------------------------------------------- */
#define SLS_DTYPE_F32  0
#define SLS_DTYPE_BF16 1

/* ---- descriptor flags -------------------------------------------------- */
/* Use the CUDA-core kernels even where a tensor-core kernel exists (for
 * comparison; results agree within the same tolerances). */
#define SLS_FLAG_CUDA_CORES 1
/* Feed the bf16 tensor-core attend kernel from registers (16-byte loads)
 * instead of the shared-memory ring filled by tensor-map copies (for
 * comparison; results agree within the same tolerances). */
#define SLS_FLAG_NO_TMA 2
/* Test hook of the bounded waits, not for production: in the tensor-map fed
 * kernels (sls_sparse_decode_attend[_combine] on bf16 pages of >= 16 tokens,
 * the one-launch sls_quest_decode_step, sls_kv8_decode_attend and
 * sls_paged_decode_attend), the first CTA of the launch (of the last two, the
 * first one that has tokens) announces 16 bytes on its first attend stage that it never requests, and
 * that CTA's waits poll a short while only.  The waits on that stage
 * give up, the first row's outputs become NaN (and those of the rows that the
 * same CTA works on after it), and the next
 * sls_pipeline_check() returns SLS_ETIMEOUT.  No copy is issued for the
 * announced bytes, so nothing faults and nothing waits forever. */
#define SLS_FLAG_TEST_WAIT_TIMEOUT 4

/*
 * Shapes and element type of one attention layer's decode step.
 *   batch        B >= 1
 *   num_q_heads  Hq >= 1
 *   num_kv_heads Hkv >= 1, Hq % Hkv == 0, G = Hq/Hkv <= 8
 *   head_dim     D in {64, 128}
 *   page_size    P, a power of two in [1, 256]; Cap % P == 0
 *   capacity     Cap >= 1 cache slots per (b, kv head)
 *   dtype        SLS_DTYPE_F32 or SLS_DTYPE_BF16: K, V, q, page min/max,
 *                thumbnail scales and the combined output use this type
 *   flags        bitwise OR of SLS_FLAG_* (0 by default)
 *   scale        softmax scale applied to q.k; 0 selects 1/sqrt(D)
 *                ("Attention: Undivided & Uncompressed", Notation:
 *                S = QK^T / sqrt(d))
 */
typedef struct sls_attn_desc {
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t capacity;
  int32_t dtype;
  int32_t flags;
  float scale;
} sls_attn_desc;

/* ---- metadata: Quest page min/max -------------------------------------- */

/*
 * Per-page, per-channel min and max of the keys ("Don't read the haystack",
 * Part two: for each page keep the elementwise min and max of its keys).
 *   k_cache  [B, Hkv, Cap, D]  dtype            (read)
 *   ctx_len  [B] int32                          (read)
 *   kmin     [B, Hkv, Cap/P, D] dtype           (written)
 *   kmax     [B, Hkv, Cap/P, D] dtype           (written)
 * Pages p < ceil(ctx_len[b]/P) are written; a partial last page summarises
 * only its positions < ctx_len[b]; later pages are left untouched.  The
 * stored values are exact copies of key elements.
 */
sls_status sls_pagemeta_build(const sls_attn_desc* desc, const void* k_cache,
                              const int32_t* ctx_len, void* kmin, void* kmax,
                              void* stream);

/*
 * Fold one appended key per sequence into its page's min/max ("Don't read
 * the haystack", Part two: summaries maintained incrementally as tokens
 * append).  The caller has already written the key at position pos[b] of
 * every kv head of sequence b.  When pos[b] % P == 0 the page is reset to
 * that key; otherwise min/max are taken with the stored values.  pos[b] < 0
 * skips sequence b; pos[b] >= Cap is clamped away (skipped) on the device.
 *   k_cache [B, Hkv, Cap, D] (read), pos [B] int32 (read),
 *   kmin, kmax [B, Hkv, Cap/P, D] (read-modify-write)
 */
sls_status sls_pagemeta_update(const sls_attn_desc* desc, const void* k_cache,
                               const int32_t* pos, void* kmin, void* kmax,
                               void* stream);

/*
 * Append one decoded token per sequence, entirely on the device, so that a
 * captured decode step can be replayed step after step: the new key and
 * value of every KV head are written at position ctx_len[b], the key is
 * folded into its page's min/max as sls_pagemeta_update does ("Don't read
 * the haystack", Part two: summaries maintained as tokens append), and
 * ctx_len[b] advances by one.  A sequence already at capacity is left
 * unchanged.
 *   k_new, v_new  [B, Hkv, D] dtype (read)
 *   k_cache, v_cache  [B, Hkv, Cap, D] dtype (row ctx_len[b] written)
 *   kmin, kmax    page metadata to keep current, or both NULL (page size 1,
 *                 or a selector without it)
 *   ctx_len       [B] int32 (read and advanced)
 *   pos_out       [B] int32 receiving the written position (-1 at capacity),
 *                 e.g. for sls_thumb_update; may be NULL
 */
sls_status sls_decode_append(const sls_attn_desc* desc, const void* k_new, const void* v_new,
                             void* k_cache, void* v_cache, void* kmin, void* kmax,
                             int32_t* ctx_len, int32_t* pos_out, void* stream);

/* ---- metadata: 2-bit key thumbnails ------------------------------------ */

/*
 * 2-bit symmetric zero-free (mid-rise) thumbnails of every complete block
 * of `block` tokens ("Faster Than Flash", Methodology 1): per block and
 * channel s = max|k|; each key element gets a 2-bit code for the levels
 * -0.75s, -0.25s, +0.25s, +0.75s (codes 0..3) with thresholds -s/2, 0,
 * +s/2, a value on a threshold taking the upper level.
 *   k_cache [B, Hkv, Cap, D] dtype (read), ctx_len [B] (read)
 *   block   power of two in [16, 256], Cap % block == 0
 *   codes   [B, Hkv, Cap, D/4] uint8 (written): channel c of a token is
 *           bits 2*(c%4) of byte c/4
 *   scales  [B, Hkv, Cap/block, D] dtype (written; exact, since max|k| is
 *           a key magnitude)
 * Only blocks that are complete (all positions < ctx_len[b]) are written.
 */
sls_status sls_thumb_build(const sls_attn_desc* desc, const void* k_cache,
                           const int32_t* ctx_len, int32_t block,
                           uint8_t* codes, void* scales, void* stream);

/*
 * Quantise the block that the key at position pos[b] completes, if any
 * (pos[b] % block == block - 1).  pos[b] < 0 skips sequence b.  Same
 * layouts as sls_thumb_build.
 */
sls_status sls_thumb_update(const sls_attn_desc* desc, const void* k_cache,
                            const int32_t* pos, int32_t block,
                            uint8_t* codes, void* scales, void* stream);

/*
 * Thumbnails plus 8-bit residuals ("Faster Than Flash", Methodology 1: the
 * key splits into the 2-bit thumbnail and an 8-bit residual that recovers
 * the precision the thumbnail drops).  The codes and scales are those of
 * sls_thumb_build; the residual of element (t, c) is
 *   r = clamp(rint(((k - k^) * 508) / s), -127, 127),   0 when s == 0,
 * each step one IEEE float32 operation (k^ = (code - 1.5) * s / 2 exactly),
 * so that the refined key k~ = k^ + r * s / 508 is within s / 1016 of k.
 *   res  [B, Hkv, Cap, D] int8 (written for complete blocks only)
 * The _update form quantises the block that position pos[b] completes, as
 * sls_thumb_update does.  Errors: SLS_EINVAL for a null pointer or a block
 * that is not a power of two in [16, 256] dividing Cap.
 */
sls_status sls_thumb_residual_build(const sls_attn_desc* desc, const void* k_cache,
                                    const int32_t* ctx_len, int32_t block, uint8_t* codes,
                                    void* scales, int8_t* res, void* stream);
sls_status sls_thumb_residual_update(const sls_attn_desc* desc, const void* k_cache,
                                     const int32_t* pos, int32_t block, uint8_t* codes,
                                     void* scales, int8_t* res, void* stream);

/* ---- selection --------------------------------------------------------- */

/*
 * Quest page selection with a fixed budget ("Don't read the haystack",
 * Part two): for every (b, kv head) row and query head g of its group,
 * U[g,p] = sum_c max(q[g,c]*kmin[p,c], q[g,c]*kmax[p,c]); the row's page
 * score is max_g U[g,p] (one list per KV head, shared by its query heads).
 * Forced pages: the first n_sink_pages pages and every page holding one of
 * the last n_local_tokens positions.  The list holds the forced pages plus
 * the top (k - #forced) other pages by score, ties to the lower page
 * index, sorted ascending.  When the row has <= k pages all of them are
 * listed and the rest of the list is -1.
 * The summaries may hold infinities: a channel adds q kmax where q > 0, q kmin
 * where q < 0 and nothing where q is 0 or NaN.  A page one of whose heads has a
 * U that is no number (infinities of both signs, a NaN summary) ranks above every
 * score and below the forced pages, ties to the lower page index.
 *   q        [B, Hq, D] dtype (read)
 *   kmin     [B, Hkv, Cap/P, D] dtype (read); kmax likewise.  With P == 1
 *            a page is one token, its min and max are the key itself:
 *            pass the K cache as kmin and kmax == kmin (read once).
 *   ctx_len  [B] int32 (read)
 *   k        budget in pages, 1 <= k <= Cap/P, and k must cover the forced
 *            pages: k >= n_sink_pages + ceil(n_local_tokens/P) + 1
 *   page_idx [B*Hkv, k] int32 (written)
 *   workspace >= sls_select_pages_workspace_size() bytes of device memory
 *            (one 32-bit key per page of every row, and for rows of more
 *            than 8192 pages the candidates of the scoring CTAs: 12.5 more
 *            bytes per page; contents on entry are ignored and on exit
 *            unspecified)
 * The score is computed in fp32; two pages whose scores differ by less
 * than the fp32 rounding of the sum may rank either way.  Rows may hold at
 * most 262144 pages (Cap/P); larger capacities return SLS_EUNSUPPORTED.
 */
sls_status sls_select_pages(const sls_attn_desc* desc, const void* q,
                            const void* kmin, const void* kmax,
                            const int32_t* ctx_len, int32_t k,
                            int32_t n_sink_pages, int32_t n_local_tokens,
                            int32_t* page_idx, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Bytes of workspace sls_select_pages needs for this descriptor (0 if the
 * descriptor is invalid or its rows hold too many pages). */
size_t sls_select_pages_workspace_size(const sls_attn_desc* desc);

/*
 * sls_select_pages without a workspace argument, for callers that cannot
 * allocate device memory for one (for example a plugin whose host framework
 * only passes it input and output tensors, or a process whose memory is all
 * reserved up front so that a cudaMalloc during decoding would fail or stall
 * the device).  It is not an operation of the source pages: only the origin
 * of the scratch differs.  The per-page keys go to a 4 MiB array compiled
 * into the library (held on every device that loads it, until exit) instead
 * of a caller buffer; the call allocates nothing.
 *   Arguments, results and validation: as sls_select_pages.
 *   Shapes whose keys need more than 4 MiB (sls_select_pages_workspace_size)
 *   return SLS_EWORKSPACE and enqueue nothing.
 *   The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before capturing a stream.  The address is cached with the id of the
 *   device's CUDA context: after a cudaDeviceReset (a new context, the
 *   array at a new address) the next call looks it up again, so make that
 *   call outside stream capture too.
 *   All calls share the array: calls whose kernels may overlap on the GPU
 *   (other streams, other host threads) race on it and must be serialised
 *   by the caller.  No part of it needs to be zero.
 */
sls_status sls_select_pages_static(const sls_attn_desc* desc, const void* q,
                                   const void* kmin, const void* kmax,
                                   const int32_t* ctx_len, int32_t k,
                                   int32_t n_sink_pages, int32_t n_local_tokens,
                                   int32_t* page_idx, void* stream);

/* Bytes of workspace sls_select_delta needs for this descriptor/block. */
size_t sls_select_delta_workspace_size(const sls_attn_desc* desc, int32_t block);

/*
 * Top-delta block selection over 2-bit thumbnails ("Faster Than Flash",
 * Methodology 2, eqs. 1-3, with eq. 4's 1/sqrt(d) scaling):
 *   m~[g]  = max over the tokens of block 0 and of the newest block
 *            (partial or not) of the exact score scale * q[g] . k
 *   a complete block b other than those two is kept when
 *            max_g max_{t in b} (scale * q[g] . k^[t] - m~[g]) >= -delta
 *            with k^ the thumbnail levels;
 *   block 0 and the newest block are always kept.
 * Output: count[r] kept blocks, block_idx[r, 0..count[r]) the kept block
 * numbers ascending (entries past count[r] are unspecified).
 *   q [B, Hq, D], k_cache [B, Hkv, Cap, D], codes/scales as written by
 *   sls_thumb_build with the same block; ctx_len [B]
 *   idx_stride >= Cap/block
 *   workspace  >= sls_select_delta_workspace_size() bytes
 * Scores are computed in fp32.
 */
sls_status sls_select_delta(const sls_attn_desc* desc, const void* q,
                            const void* k_cache, const uint8_t* codes,
                            const void* scales, const int32_t* ctx_len,
                            int32_t block, float delta, int32_t* count,
                            int32_t* block_idx, int32_t idx_stride,
                            void* workspace, size_t workspace_bytes,
                            void* stream);

/* ---- attention --------------------------------------------------------- */

/*
 * Split-K sparse decode attention, stage one of two-stage flash-decoding
 * ("Don't read the haystack", Part one; the sparse twin of Part two walks
 * a page list instead of a range).  For every row r = (b, h), the page list
 * page_idx[r*idx_stride + i], i < n_r (n_r = count[r] if count != NULL,
 * else k_fixed) is cut into num_splits contiguous slices; slice s of every
 * query head g of the group produces
 *   m = max x, l = sum exp(x - m), acc = sum exp(x - m) v
 * over the valid tokens of its pages (position < ctx_len[b]), with
 * x = scale * q.k.  The sink is NOT applied here (see combine).
 * page_idx == NULL attends every page 0..ceil(ctx_len/P)-1 (dense decode).
 *   q [B, Hq, D], k_cache/v_cache [B, Hkv, Cap, D] dtype (read)
 *   o_part [B, Hq, num_splits, D] f32, m_part/l_part [B, Hq, num_splits]
 *   f32 (written; m in natural-log units; an empty slice gives m = -inf,
 *   l = 0, acc = 0)
 *   1 <= num_splits <= 1024
 */
sls_status sls_sparse_decode_attend(const sls_attn_desc* desc, const void* q,
                                    const void* k_cache, const void* v_cache,
                                    const int32_t* page_idx, int32_t idx_stride,
                                    const int32_t* count, int32_t k_fixed,
                                    const int32_t* ctx_len, int32_t num_splits,
                                    float* o_part, float* m_part, float* l_part,
                                    void* stream);

/*
 * Stage two: merge the splits with the log-sum-exp rescale ("Don't read the
 * haystack", Part one) and fold in the optional per-query-head sink as a
 * virtual key with value 0 ("Training-free sparse attention for
 * long-context LLM decode", section 1): with M = max(max_s m_s, sink_h),
 *   L = sum_s l_s e^(m_s - M) + e^(sink_h - M),
 *   out = sum_s acc_s e^(m_s - M) / L,   lse = M + log L.
 * The sink is a raw logit (not scaled).  Rows with no token and no sink
 * give out = 0, lse = -inf.
 *   o_part/m_part/l_part as written by sls_sparse_decode_attend
 *   sink [Hq] f32 or NULL
 *   out [B, Hq, D] dtype (written); lse [B, Hq] f32 or NULL (written)
 */
sls_status sls_combine_splits(const sls_attn_desc* desc, const float* o_part,
                              const float* m_part, const float* l_part,
                              int32_t num_splits, const float* sink, void* out,
                              float* lse, void* stream);

/*
 * A split count for sls_sparse_decode_attend(_combine) that gives about two
 * waves of CTAs on this GPU, each slice holding at least 64 tokens of a
 * list of up to max_entries pages.  Returns 1 for an invalid descriptor.
 */
int32_t sls_attend_default_splits(const sls_attn_desc* desc, int32_t max_entries);

/* Bytes of workspace sls_sparse_decode_attend_combine needs (num_splits 0:
 * the library's own schedule on the current device). */
size_t sls_attend_combine_workspace_size(const sls_attn_desc* desc,
                                         int32_t num_splits);

/*
 * Both stages in one launch: sls_sparse_decode_attend followed, inside the
 * same kernel, by the combine of each row.  num_splits == 0 lets the library
 * pick the split count (sls_attend_default_splits).  Where the tensor-map
 * fed kernel runs (bf16, pages of >= 16 tokens) with at most 16 splits, the
 * splits of a row form one thread-block cluster and combine through
 * distributed shared memory; otherwise every CTA of a row takes an arrival
 * ticket after writing its partials and the CTA that arrives last merges the
 * row's splits exactly as sls_combine_splits does (no CTA ever waits for
 * another).  Arguments as in the two separate calls; the partials live in
 * the workspace, whose first 4*B*Hkv bytes hold the tickets.
 *   workspace  >= sls_attend_combine_workspace_size() bytes; it must be
 *              zero-filled before its first use, and every call leaves the
 *              tickets at zero again.  Calls sharing a workspace must not
 *              run concurrently.
 */
sls_status sls_sparse_decode_attend_combine(const sls_attn_desc* desc, const void* q,
                                            const void* k_cache, const void* v_cache,
                                            const int32_t* page_idx, int32_t idx_stride,
                                            const int32_t* count, int32_t k_fixed,
                                            const int32_t* ctx_len, int32_t num_splits,
                                            const float* sink, void* out, float* lse,
                                            void* workspace, size_t workspace_bytes,
                                            void* stream);

/*
 * Refined top-delta attention ("Faster Than Flash", Methodology 3 step 3,
 * eq. 4): attention over each row's kept blocks in which the tokens of
 * complete blocks are scored with the refined key
 *   k~ = (code - 1.5) * s / 2 + r * s / 508
 * (thumbnail level plus 8-bit residual, sls_thumb_residual_build) instead
 * of the bf16 key; tokens of the newest, partial block are scored with the
 * bf16 key.  Values are the bf16 V.  With codes, scales and res all NULL
 * every token is scored with its bf16 key (plain attention over the lists).
 * The rows' lists, of different lengths, are cut into work items of equal
 * length spread over the GPU; each row's last item merges the row (sink,
 * lse as in sls_combine_splits).
 *   desc.page_size  the thumbnail block (>= 16); bf16, G <= 8, D 64 or 128,
 *                   B*Hkv <= 4096
 *   codes, scales, res  as written by sls_thumb_residual_build/_update
 *   block_idx [B*Hkv, idx_stride] int32, count [B*Hkv] int32: the kept
 *             blocks of each row (sls_select_delta's output); -1 entries
 *             and blocks past the context are skipped
 *   workspace >= sls_refined_decode_attend_workspace_size() bytes, zero-
 *             filled before its first use (every call leaves its arrival
 *             counters at zero); calls sharing it must not run concurrently
 *   |q * s| must stay below 65504 (the products run in fp16 hi/lo parts).
 * Errors: SLS_EUNSUPPORTED for another dtype, G > 8, blocks < 16 tokens or
 * more rows; SLS_EINVAL for null or misaligned pointers or bad sizes;
 * SLS_EWORKSPACE.
 */
size_t sls_refined_decode_attend_workspace_size(const sls_attn_desc* desc);
sls_status sls_refined_decode_attend_combine(const sls_attn_desc* desc, const void* q,
                                             const void* k_cache, const void* v_cache,
                                             const uint8_t* codes, const void* scales,
                                             const int8_t* res, const int32_t* block_idx,
                                             int32_t idx_stride, const int32_t* count,
                                             const int32_t* ctx_len, const float* sink,
                                             void* out, float* lse, void* workspace,
                                             size_t workspace_bytes, void* stream);

/* ---- the whole Quest decode step ---------------------------------------- */

/* Bytes of workspace sls_quest_decode_step needs for this budget and split
 * count (0 on an invalid descriptor). */
size_t sls_quest_decode_step_workspace_size(const sls_attn_desc* desc, int32_t k, int32_t num_splits);

/* CTAs per row (the cluster size) the one-launch Quest step uses for this
 * shape and budget by default; 0 when the shape takes the two-launch path. */
int32_t sls_quest_decode_step_splits(const sls_attn_desc* desc, int32_t k);

/*
 * One Quest decode step: the selection of sls_select_pages (budget k,
 * n_sink_pages, n_local_tokens, same tie rule and list order) and the
 * sparse attention with the combine of sls_sparse_decode_attend_combine
 * over the chosen pages ("Don't read the haystack", Part two).
 *
 * For bf16 caches with pages of >= 16 tokens (k <= 4096, Cap/P <= 131072)
 * this is ONE kernel launch: a
 * thread-block cluster per (sequence, KV head) scores its row's pages from
 * the min/max metadata, selects the top k inside the cluster and attends to
 * them; the scores and the page list never leave shared memory.  Otherwise
 * the call runs sls_select_pages then sls_sparse_decode_attend_combine.
 *   kmin, kmax  [B, Hkv, Cap/P, D] page metadata (sls_pagemeta_build)
 *   page_idx    [B*Hkv, k] int32 receiving the chosen pages (ascending, -1
 *               padded), or NULL
 *   out, lse    as in sls_combine_splits
 *   num_splits  CTAs per row (0: the library's choice; the one-launch kernel
 *               uses at most 16)
 *   min_sparsity  sparsity gate ("perf(core): fused sparse-attention decode
 *               via page indirection", Corrected premise 2): a row whose
 *               context holds fewer than min_sparsity * k * P tokens is
 *               attended densely over its whole context, without selection,
 *               and its page_idx row is left at -1.  0 disables the gate.
 *               The gate needs the one-launch kernel: on the two-launch path
 *               a non-zero value returns SLS_EUNSUPPORTED.
 *   workspace   >= sls_quest_decode_step_workspace_size() bytes, zero-filled
 *               before its first use (the one-launch kernel leaves it alone;
 *               the two-launch path keeps its tickets at zero).
 */
sls_status sls_quest_decode_step(const sls_attn_desc* desc, const void* q, const void* k_cache,
                                 const void* v_cache, const void* kmin, const void* kmax,
                                 const int32_t* ctx_len, int32_t k, int32_t n_sink_pages,
                                 int32_t n_local_tokens, const float* sink, int32_t* page_idx,
                                 void* out, float* lse, int32_t num_splits, float min_sparsity,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* ---- selection quality ------------------------------------------------- */

/* Bytes of workspace sls_selection_recall needs. */
size_t sls_selection_recall_workspace_size(const sls_attn_desc* desc);

/*
 * Attention-mass recall of page lists ("Don't read the haystack", Part
 * three: how much of the true attention mass the selected pages hold): for
 * every query head, the share of its full-context softmax mass (scores
 * scale * q.k over the positions < ctx_len; no sink) that falls on the
 * tokens of its row's listed pages.  A diagnostic beside the decode step: it
 * reads every key of the context.
 *   page_idx, idx_stride, count, k_fixed   as in sls_sparse_decode_attend
 *               (NULL page_idx: every page, recall 1)
 *   recall      [B, Hq] float; an empty context gives 1 (no mass missed)
 *   workspace   >= sls_selection_recall_workspace_size() bytes
 * Capacities above 262144 pages per row return SLS_EUNSUPPORTED.
 */
sls_status sls_selection_recall(const sls_attn_desc* desc, const void* q, const void* k_cache,
                                const int32_t* page_idx, int32_t idx_stride, const int32_t* count,
                                int32_t k_fixed, const int32_t* ctx_len, float* recall, void* workspace,
                                size_t workspace_bytes, void* stream);

/* ---- per-head norm and position rotation ------------------------------- */

/*
 * Shapes of sls_qk_norm_rope.
 *   num_q_heads, num_kv_heads  >= 0, at least one head in all
 *   head_dim     D in {64, 128}
 *   rotary_dim   R: the first R channels of a head are rotated, the others
 *                pass through; a multiple of 16 in [0, D]
 *   interleaved  0: channel i pairs with i + R/2;  1: 2i pairs with 2i + 1
 *   dtype        SLS_DTYPE_F32 or SLS_DTYPE_BF16 (q, k, weights, outputs)
 *   eps          added to the mean square, >= 0
 *   theta        base of the frequencies f_i = theta^(-2i/R), i < R/2, > 0
 *   inv_freq     HOST pointer to R/2 frequencies in radians per position
 *                (each finite), or NULL for those of theta
 */
typedef struct sls_rope_desc {
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t rotary_dim;
  int32_t interleaved;
  int32_t dtype;
  float eps;
  double theta;
  const double* inv_freq;
} sls_rope_desc;

/*
 * Root-mean-square norm of every query and key head and the rotation by the
 * token's position, in one pass.  For token t and head vector x:
 *   y = x * w / sqrt(mean(x^2) + eps)        (w NULL: y = x, no norm)
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
 * for every channel pair (a, b) with the angle positions[t] * f_i.
 * The arithmetic is fp32; angles are reduced modulo one turn in 64-bit fixed
 * point, so far positions lose nothing; results are rounded once.
 *   q [N, Hq, D], k [N, Hkv, D]   read, with strides in elements between
 *        tokens and between heads (>= 0, multiples of 8 for bf16 and 4 for
 *        fp32; channels are contiguous), so the head slices of one packed
 *        projection can be passed as they are
 *   q_weight, k_weight  [D] dtype, or NULL
 *   positions [N] int32; a token with a negative position is skipped (its
 *        outputs are left as they were)
 *   q_out, k_out  written, strides as above and without overlap.  They may
 *        be q and k themselves (same pointer and strides); any other overlap
 *        of inputs and outputs gives unspecified results.
 * q (k) and its output are ignored when num_q_heads (num_kv_heads) is 0;
 * num_tokens 0 does nothing.
 * Errors: SLS_EINVAL for null or misaligned pointers, bad strides or bad
 * values; SLS_EUNSUPPORTED for another head_dim, rotary_dim or dtype.
 */
sls_status sls_qk_norm_rope(const sls_rope_desc* rope, int32_t num_tokens,
                            const void* q, int64_t q_token_stride, int64_t q_head_stride,
                            const void* k, int64_t k_token_stride, int64_t k_head_stride,
                            const void* q_weight, const void* k_weight,
                            const int32_t* positions,
                            void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                            void* k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
                            void* stream);

/* ---- the 8-bit KV cache ------------------------------------------------- */

/* Code formats: the value of a code c is c * s with the block's scale s. */
#define SLS_KV8_INT8 0  /* two's complement integers -127..127, s = max|x| / 127 */
#define SLS_KV8_E4M3 1  /* 4-bit exponent, 3-bit mantissa floats, s = max|x| / 448 */

/*
 * A K/V cache held in 8 bits with one scale for each block of `block` tokens
 * of each KV head (bf16 descriptors only).  The struct lives on the host, the
 * pointers are device memory of the caller.  Blocks are quantised once, when
 * their last token arrives; the tokens of a sequence's newest, partial block
 * wait in bf16 in the tail buffers (token position t at slot t % block).
 * Complete block: amax = max |x| over its block * D elements, and with
 * top = 127 or 448
 *   s = amax / top,  code = round(x * top / amax) to the nearest code, ties
 *   to even (each step one IEEE float32 operation); amax = 0 gives s = 0 and
 *   codes 0; an infinity or NaN in the block gives s = NaN and codes 0, so
 *   that it shows in every output that attends to the block.
 *   format    SLS_KV8_INT8 or SLS_KV8_E4M3
 *   block     power of two in [16, 256], Cap % block == 0, Cap <= 2^30
 *   k_codes, v_codes    [B, Hkv, Cap, D] one byte each
 *   k_scales, v_scales  [B, Hkv, Cap/block] float
 *   k_tail, v_tail      [B, Hkv, block, D] bf16
 * All pointers 16-byte aligned but for the scales (4); six pieces of memory.
 */
typedef struct sls_kv8_cache {
  int32_t format;
  int32_t block;
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scales;
  float* v_scales;
  void* k_tail;
  void* v_tail;
} sls_kv8_cache;

/*
 * Append new tokens of every sequence to its cache: one decoded token, a
 * whole prompt or a piece of one.  Sequence b appends its first new_len[b]
 * (clamped to [0, max_new]; NULL: max_new) tokens at positions ctx_len[b]
 * and up: blocks that become complete are quantised, the tokens of the
 * newest, partial block go to the tail buffers, and ctx_out[b] =
 * ctx_len[b] + the count.  A sequence whose tokens do not all fit is left
 * unchanged (ctx_out[b] = ctx_len[b]).
 *   k_new, v_new  [B, max_new, Hkv, D] bf16 (read), strides in elements
 *                 between sequences, tokens and heads (>= 0, multiples of 8;
 *                 channels contiguous)
 *   kmin, kmax    [B, Hkv, Cap/P, D] bf16 page min/max of the (unquantised)
 *                 keys to keep current as sls_pagemeta_update does, or both
 *                 NULL
 *   mass          [B, Hkv, Cap/block] float: set to 0 for every block that
 *                 becomes complete, or NULL
 *   ctx_len       [B] int32 (read, clamped to [0, Cap]); ctx_out [B] int32
 *                 (written; ctx_len itself or memory of its own)
 *   pos_out       [B] int32 receiving the first written position (-1 when
 *                 nothing was written), or NULL; memory of its own
 * Lengths and outputs share no memory with the cache or each other (ctx_out
 * excepted, as above).
 * max_new 0 appends nothing (ctx_out and pos_out are still written).
 */
sls_status sls_kv8_append(const sls_attn_desc* desc, const sls_kv8_cache* cache,
                          const void* k_new, int64_t k_seq_stride, int64_t k_token_stride, int64_t k_head_stride,
                          const void* v_new, int64_t v_seq_stride, int64_t v_token_stride, int64_t v_head_stride,
                          int32_t max_new, const int32_t* new_len, void* kmin, void* kmax, float* mass,
                          const int32_t* ctx_len, int32_t* ctx_out, int32_t* pos_out, void* stream);

/* Bytes of workspace sls_kv8_decode_attend needs (with_mass: when it is
 * given mass_out); 0 for an invalid or unsupported descriptor or cache. */
size_t sls_kv8_decode_attend_workspace_size(const sls_attn_desc* desc, const sls_kv8_cache* cache,
                                            int32_t with_mass);

/*
 * Decode attention over an 8-bit cache: softmax(scale q.k^) v^ with k^, v^
 * the stored values (codes times scales; bf16 tail tokens as they are), over
 * the positions < ctx_len[b] (page_idx NULL) or over the valid tokens of the
 * listed pages, with the sink as in sls_combine_splits.  Rows of uneven
 * length are cut into equal ranges over the GPU.
 *   desc      bf16, G <= 8, D 64 or 128, B*Hkv <= 4096, B*Hkv*Cap < 2^31;
 *             with page_idx pages of >= 16 tokens (the page size does not
 *             matter otherwise); of the flags only SLS_FLAG_TEST_WAIT_TIMEOUT
 *   page_idx, idx_stride, count, k_fixed   as in sls_sparse_decode_attend
 *             (-1 entries are skipped, bad ones counted for
 *             sls_pipeline_check and skipped)
 *   sink      [Hq] float or NULL;  out [B, Hq, D] bf16 (not q's memory);
 *             lse [B, Hq] float or NULL
 *   mass_in, mass_out  [B, Hkv, Cap/block] float, or mass_out NULL: every
 *             complete block of the context gets mass_out = mass_in (NULL: 0)
 *             + the sum over the group's query heads and the block's tokens
 *             of the softmax weight; the other blocks' entries are left as
 *             they were.  mass_in may be mass_out itself.  Only without
 *             page_idx.
 *             The sums do not depend on the order in which CTAs finish.
 *   workspace >= sls_kv8_decode_attend_workspace_size() bytes, 16-byte
 *             aligned, zero-filled before its first use (every call leaves
 *             its arrival counters at zero).  Calls of this function, of any
 *             shapes, may share one that is large enough for each, but not
 *             run concurrently
 * Outputs and workspace share no memory with each other or with what is read
 * (mass_in excepted).
 * Roundings: scores, softmax statistics and sums are fp32.  In the value
 * product a weight times its block's value scale has 11 bits (tail tokens'
 * weights 16), down to 2^-28 of the largest such product that shares its sums;
 * smaller ones lose bits, and those below 2^-38 of it are dropped.  The
 * output is rounded to bf16.
 * Rows with no token: out = 0, lse = -inf (or the sink alone).
 */
sls_status sls_kv8_decode_attend(const sls_attn_desc* desc, const sls_kv8_cache* cache, const void* q,
                                 const int32_t* page_idx, int32_t idx_stride, const int32_t* count,
                                 int32_t k_fixed, const int32_t* ctx_len, const float* sink, void* out,
                                 float* lse, const float* mass_in, float* mass_out, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * Bound a cache by the attention weight its blocks have drawn.  A sequence
 * with more than keep complete blocks keeps, in every KV head's row, its
 * first n_sink_blocks, its newest n_recent_blocks complete blocks and those
 * with the largest mass of the others, ties to the lower block (NaN counts as
 * the largest), keep in all, in their old order without gaps, so the row
 * looks as if the evicted tokens had never been appended.  The tail stays;
 * ctx_out[b] = min(ctx_len[b]/block, keep) * block + ctx_len[b] % block.
 *   desc, src     the cache to cut; dst_capacity, dst  the cache to write:
 *                 the source itself (dst NULL or equal to src, dst_capacity
 *                 = Cap: in place) or another one with the same format and
 *                 block and no memory in common (every kept block is copied,
 *                 and the valid tail tokens).
 *                 (keep + 1) * block <= dst_capacity, dst_capacity % block
 *                 == 0
 *   keep >= 1, 0 <= n_sink_blocks + n_recent_blocks <= keep
 *   mass          [B, Hkv, Cap/block] float (read); mass_out [B, Hkv,
 *                 dst_capacity/block] the kept blocks' sums, or NULL.  In
 *                 place mass_out must be mass.
 *   kmin, kmax    page min/max to take along, or both NULL, to kmin_out,
 *                 kmax_out [B, Hkv, dst_capacity/P, D] (in place: the same
 *                 buffers); needs P <= block and P dividing dst_capacity
 *   kept_idx      [B*Hkv, keep] int32 (written): the kept blocks' old
 *                 numbers, ascending, -1 padded when the row has fewer;
 *                 memory of its own, as are ctx_len and ctx_out
 *   ctx_len [B] (read), ctx_out [B] (written; ctx_len itself or memory of
 *             its own)
 */
sls_status sls_kv8_evict(const sls_attn_desc* desc, const sls_kv8_cache* src, int32_t dst_capacity,
                         const sls_kv8_cache* dst, int32_t keep, int32_t n_sink_blocks,
                         int32_t n_recent_blocks, const float* mass, float* mass_out, const void* kmin,
                         const void* kmax, void* kmin_out, void* kmax_out, int32_t* kept_idx,
                         const int32_t* ctx_len, int32_t* ctx_out, void* stream);

/* ---- the paged KV cache -------------------------------------------------- */

/*
 * A K/V cache whose pages lie anywhere in a pool and may be held by several
 * sequences.  Of the descriptor, batch is the number of sequences, page_size P
 * in [16, 256], and capacity the most tokens of one sequence (no memory is
 * set aside for it but the table's row).  The struct lives on the host, the
 * pointers are device memory of the caller.
 *   num_pages   N pages of the pool, 1 <= N <= 2^24, N * Hkv * P < 2^31
 *   k_pages, v_pages  [N, Hkv, P, D] dtype
 *   kmin, kmax  [N, Hkv, D] dtype: min and max of every page's keys, kept
 *               current by the calls below, or both NULL
 *   ctx_len     [B] int32 tokens of each sequence
 *   table       [B, Cap/P] int32 the pool's page that holds a logical page, -1
 *               past the sequence's length
 *   refs        [N] int32 sequences that hold each page (0: free)
 *   state       [sls_paged_state_words()] int32, the free pages and scratch of
 *               the calls; its contents are the library's
 * k_pages, v_pages, kmin, kmax and state are 16-byte aligned; no two of the
 * buffers share memory.  Before the first use of a cache (all ctx_len 0), and
 * whenever table or ctx_len were written by the caller, sls_paged_init derives
 * refs and state from them.
 * A page that is not complete (the last one of a sequence whose length is not
 * a multiple of P) belongs to one sequence; complete pages may be shared and are
 * never written.  The calls keep to this; a table that the caller writes has to.
 * Calls on one cache are ordered by the caller: none runs while another that
 * changes it does.  At most 4096 sequences; another P returns
 * SLS_EUNSUPPORTED.  Table entries of a sequence's length that are no page
 * of the pool are counted for sls_pipeline_check() and skipped.
 */
typedef struct sls_paged_cache {
  int32_t num_pages;
  void* k_pages;
  void* v_pages;
  void* kmin;
  void* kmax;
  int32_t* ctx_len;
  int32_t* table;
  int32_t* refs;
  int32_t* state;
} sls_paged_cache;

/* Words of a cache's state; 0 for an invalid descriptor or number of pages. */
size_t sls_paged_state_words(const sls_attn_desc* desc, int32_t num_pages);

/*
 * Derives refs and state from table and ctx_len (read), and sets the table's
 * entries past each length to -1.  The page summaries are the caller's.
 */
sls_status sls_paged_init(const sls_attn_desc* desc, const sls_paged_cache* cache, void* stream);

/*
 * Append new tokens of every sequence: one decoded token, a whole prompt or a
 * piece of one.  Sequence b appends its first new_len[b] (clamped to
 * [0, max_new]; NULL: max_new) tokens at positions ctx_len[b] and up.  It needs
 * ceil((ctx_len[b] + n) / P) - ceil(ctx_len[b] / P) pages: the call takes the
 * lowest-numbered free ones, in the order of sequences and their logical pages.
 * A sequence whose tokens do not fit its capacity needs none and is left
 * unchanged; so is one that needs pages when it and the sequences before it need
 * more in all than are free (a later one that needs none still appends).
 *   k_new, v_new  [B, max_new, Hkv, D] dtype (read), strides in elements
 *                 between sequences, tokens and heads (>= 0, multiples of 8
 *                 for bf16 and 4 for fp32; channels contiguous); no memory of the
 *                 cache
 *   kmin, kmax of the cache: a page's first token sets them, later ones fold in
 *   pos_out       [B] int32 receiving the first written position (-1 when
 *                 nothing was written), or NULL; memory of its own
 * A sequence whose partial page is held by others too (a table the caller
 * wrote) is left unchanged and counted as a bad entry.
 */
sls_status sls_paged_append(const sls_attn_desc* desc, const sls_paged_cache* cache,
                            const void* k_new, int64_t k_seq_stride, int64_t k_token_stride, int64_t k_head_stride,
                            const void* v_new, int64_t v_seq_stride, int64_t v_token_stride, int64_t v_head_stride,
                            int32_t max_new, const int32_t* new_len, int32_t* pos_out, void* stream);

/*
 * sls_select_pages over a paged cache: the summaries are the cache's kmin and
 * kmax (not NULL), found through its table; page_idx [B, Hkv, k] receives
 * LOGICAL pages.  A page whose table entry is bad scores as a summary of zeros.
 *   workspace  >= sls_select_pages_workspace_size() bytes, memory of its own
 *              like page_idx
 */
sls_status sls_paged_select_pages(const sls_attn_desc* desc, const sls_paged_cache* cache, const void* q, int32_t k,
                                  int32_t n_sink_pages, int32_t n_local_tokens, int32_t* page_idx, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Bytes of workspace sls_paged_decode_attend needs; 0 for an invalid or
 * unsupported descriptor. */
size_t sls_paged_decode_attend_workspace_size(const sls_attn_desc* desc);

/*
 * Decode attention over a paged cache: softmax(scale q.k) v over the positions
 * < ctx_len[b] (page_idx NULL) or over the valid tokens of the listed LOGICAL
 * pages, with the sink as in sls_combine_splits.  Rows of uneven length are cut
 * into equal ranges over the GPU.
 *   desc      G <= 8, D 64 or 128, B*Hkv <= 4096, B*Hkv*(Cap/16 + 1) < 2^30;
 *             of the flags only SLS_FLAG_TEST_WAIT_TIMEOUT
 *   page_idx, idx_stride, count, k_fixed   as in sls_sparse_decode_attend
 *             (-1 entries are skipped, bad ones counted and skipped); count
 *             only with page_idx; idx_stride*P < 2^31 and
 *             B*Hkv*idx_stride*(P/16) <= 2^30, else SLS_EOVERFLOW
 *   q [B, Hq, D] dtype; sink [Hq] float or NULL; out [B, Hq, D] dtype; lse
 *             [B, Hq] float or NULL
 *   workspace >= sls_paged_decode_attend_workspace_size() bytes, 16-byte
 *             aligned, zero-filled before its first use (every call leaves
 *             its arrival counters at zero).  Calls of this function, of any
 *             shapes, may share one that is large enough for each, but not
 *             run concurrently
 * Outputs and workspace share no memory with each other or with what is read.
 * Roundings: scores, softmax statistics and sums are fp32; a bf16 cache's
 * weights enter the value product with 16 bits; the output is rounded to dtype.
 * Rows with no token: out = 0, lse = -inf (or the sink alone).
 */
sls_status sls_paged_decode_attend(const sls_attn_desc* desc, const sls_paged_cache* cache, const void* q,
                                   const int32_t* page_idx, int32_t idx_stride, const int32_t* count, int32_t k_fixed,
                                   const float* sink, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* Bytes of workspace sls_paged_fork needs; 0 for an invalid descriptor. */
size_t sls_paged_fork_workspace_size(const sls_attn_desc* desc);

/*
 * Make every sequence a prefix of an old one, all at once: sequence b becomes
 * the first min(ctx_len[parent[b]], keep_len[b]) tokens of what sequence
 * parent[b] was before the call (keep_len NULL: all of them).  parent[b] = b
 * leaves it (or cuts it), -1 frees it, several sequences with one parent fork
 * it, and a permutation reorders.  Complete pages are shared.  A partial last
 * page, other than that of a sequence that stays as it is, is kept by the
 * lowest-numbered sequence that needs it if no sequence holds it otherwise, and
 * copied for the others to the lowest-numbered pages that were free before the
 * call, in the order of sequences; its summary is formed anew.  Pages that no
 * sequence holds any more are free after the call.
 *   parent    [B] int32 (read); a value outside [-1, B) leaves the sequence as
 *             it is and is counted for sls_pipeline_check()
 *   keep_len  [B] int32 (read, negative ones count as 0) or NULL
 *   done      [1] int32 or NULL: 1, or 0 when fewer pages were free than copies
 *             are needed; then nothing has changed
 *   workspace >= sls_paged_fork_workspace_size() bytes, 16-byte aligned
 * parent, keep_len, done and workspace are memory of their own.
 */
sls_status sls_paged_fork(const sls_attn_desc* desc, const sls_paged_cache* cache, const int32_t* parent,
                          const int32_t* keep_len, int32_t* done, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace sls_paged_compact needs; 0 for an invalid number of pages. */
size_t sls_paged_compact_workspace_size(int32_t num_pages);

/*
 * Move the used pages to the front of the pool, so that with U of them the
 * pages from U on are free: the used pages numbered U and up move, in order, to
 * the free pages below U, with their summaries; table and refs follow.
 *   moved     [N] int32: every page's new number, -1 for those that were free;
 *             or NULL
 *   workspace >= sls_paged_compact_workspace_size() bytes, 16-byte aligned
 * moved and workspace are memory of their own.
 */
sls_status sls_paged_compact(const sls_attn_desc* desc, const sls_paged_cache* cache, int32_t* moved, void* workspace,
                             size_t workspace_bytes, void* stream);

/* ---- diagnostics ------------------------------------------------------- */

/* Message of the last failing call on this thread ("" if none). */
const char* sls_last_error(void);

/*
 * Device status of the kernels since the previous check ("perf(core): fused
 * sparse-attention decode via page indirection", Making the selection
 * inspectable: every call has an observable outcome).  Two kinds of events
 * are counted on the device:
 *   - a bounded wait on a copy pipeline that gave up (kernels that stage data
 *     through shared memory poll their copies a bounded number of times; the
 *     affected outputs become NaN);
 *   - a page-list entry that is neither a page of the pool [0, Cap/P) nor the
 *     -1 padding (the attend and recall kernels skip it: it gives no token);
 *     and what the calls of a paged cache count as bad: table entries, partial
 *     pages that are shared, parents that do not exist.
 * This call synchronises the device, reads and clears the counts (one atomic
 * exchange per word, so no count is lost), and returns SLS_ETIMEOUT if any
 * wait gave up, else SLS_EDEVICE if any bad entry was met, else SLS_OK
 * (SLS_ECUDA if the device cannot be read); the message gives the counts.
 * The counts are global to the process: they cover every launch since the
 * previous check, on every stream and host thread, so only calls ordered
 * with the check are attributed to it.
 */
sls_status sls_pipeline_check(void);

/*
 * Which paths the library took ("perf(core): fused sparse-attention decode
 * via page indirection", Proving which path a benchmark arm took: a
 * benchmark must be able to show which kernel it measured).  Host counters
 * count launches by the kernel the library picked; the two row counters are
 * kept on the device by the one-launch step.
 */
typedef struct sls_stats {
  uint64_t quest_step_one_launch;     /* sls_quest_decode_step calls run as one kernel */
  uint64_t quest_step_two_launch;     /* ... run as select + attend (shape outside the kernel) */
  uint64_t step_rows_dense;           /* rows the sparsity gate sent to dense attention */
  uint64_t step_rows_all_keys;        /* rows whose cluster selected from all of the row's keys
                                         (long rows, or the candidate check failed) */
  uint64_t select_pages;              /* sls_select_pages(_static) and sls_paged_select_pages calls */
  uint64_t select_delta_tensor_cores; /* top-delta scans on the tensor cores */
  uint64_t select_delta_cuda_cores;   /* ... on the CUDA cores (fp32, or the CUDA-core flag) */
  uint64_t attend_tma;                /* split-K attends by kernel: tensor-map fed, */
  uint64_t attend_mma;                /* register-fed tensor cores, */
  uint64_t attend_cuda_cores;         /* CUDA cores */
  uint64_t attend_stream_k;           /* stream-K attends over block lists with bf16 keys */
  uint64_t attend_refined;            /* ... with the refined (2-bit + 8-bit) keys */
  uint64_t combine;                   /* separate combine launches */
  uint64_t metadata;                  /* page min/max, thumbnail, residual and append calls, and those of
                                         the norm/rotation, the 8-bit cache's append and eviction, and the
                                         paged cache's append, fork and compaction */
  uint64_t recall;                    /* selection-recall launches */
  uint64_t select_rows_all_keys;      /* rows wider than 8192 pages whose sls_select_pages top-k
                                         ranked all of the row's keys (the candidate check failed) */
  uint64_t attend_stream_k_tma;       /* of attend_stream_k: the tensor-map fed kernel */
  uint64_t attend_refined_tma;        /* of attend_refined: the tensor-map fed kernel */
  uint64_t attend_kv8;                /* attends over an 8-bit cache */
  uint64_t attend_paged;              /* attends over a paged cache */
  uint64_t select_paged_one_launch;   /* of select_pages: selections over a paged cache run as one kernel */
} sls_stats;

/* Fills *out (the sls_stats of this header: counters are added at its end)
 * with the counters (synchronising the device to read the row
 * counters); reset != 0 zeroes them.  SLS_EINVAL for a NULL out. */
sls_status sls_get_stats(sls_stats* out, int32_t reset);

/* Library ABI version (major*10000 + minor*100 + patch). */
int32_t sls_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SLS_H */

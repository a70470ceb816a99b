/*
 * msa.h -- C ABI of libmsa: the hot path of MiniMax Sparse Attention (MSA)
 * on one NVIDIA B200 (sm_100a).
 *
 * The method (web pages, cited by title and section):
 *   [P2] "MiniMax M3模型算力成本大幅降低原因深度解析", sections "索引分支（Index
 *        Branch）" and "稀疏分支（Sparse Branch）": a lightweight single-head
 *        index key with block max-pooling screens the whole context and keeps
 *        the top-K KV blocks; standard GQA then runs over the kept blocks only,
 *        on raw KV.
 *   [P4] "MiniMax M3 深度实战 ...", section 2.2 "KV Outer Gather Q" (each KV
 *        block gathers the queries that selected it and is read once), section
 *        2.3 "MSA 算法实现" (the own/local block is always kept; softmax of
 *        Q K^T / sqrt(d_head) over the gathered keys), section 3.3 (decode:
 *        one new query, at the newest position).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *    never allocates, frees or retains memory and (apart from the
 *    no-allocation decode entry point below) keeps no global mutable state,
 *    so calls on different workspaces may run concurrently.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  Every call is
 *    asynchronous on that stream and returns after enqueueing its kernels.
 *  - Layouts are row-major and contiguous, bf16 means IEEE bfloat16 bits:
 *        q_idx [Bt][n_q][d_idx]  bf16     k_idx [Bt][T][d_idx]   bf16
 *        q     [Bt][n_q][Hq][d]  bf16     k, v  [Bt][T][Hkv][d]  bf16
 *        ids   [Bt][n_q][K]      int32    out   [Bt][n_q][Hq][d] fp32
 *        lse   [Bt][n_q][Hq]     fp32
 *    Query i (0 <= i < n_q) of sequence b sits at position t = T - n_q + i of
 *    its length-T context (prefill: n_q = T; decode: n_q = 1).  Block j holds
 *    keys [j*block, min((j+1)*block, T)); N = ceil(T / block); own(t) = t / block.
 *  - Selection: ids[b][i] lists min(K, own(t)+1) distinct blocks in ascending
 *    order, padded with -1: the own block, plus the top min(K, own+1) - 1 of
 *    the blocks j < own(t) ranked by s(t,j) = max_{i in block j} q_idx[t].k_idx[i]
 *    (descending; ties go to the lower block index).  Scores are accumulated in
 *    fp32, which is exact for the integer-valued index keys of the pages'
 *    workloads (|s| < 2^24).
 *  - Attention: for each query head h (kv head h / (Hq/Hkv)), softmax of
 *    q.k_i / sqrt(d) over the keys i <= t of the blocks in ids, output the
 *    weighted sum of v_i (fp32) and lse = ln sum_i exp(q.k_i / sqrt(d)).
 *  - Supported shapes: d, d_idx in {64, 128}; block in {32, 64} or a
 *    multiple of 128; 1 <= K <= 32; 128 % (Hq/Hkv) == 0; N <= 8192;
 *    Bt*T < 2^31, Bt*n_q*K < 2^31 and Bt*n_q*Hq*d < 2^34 (the attention
 *    calls address q in 16-byte units with 32-bit offsets).  Anything else
 *    returns MSA_ERR_UNSUPPORTED before any work is enqueued.
 *  - Alignment (MSA_ERR_INVALID_ARG otherwise, nothing enqueued): q_idx,
 *    k_idx, q, k, v (and their paged stores) and out must be 16-byte aligned
 *    (they are read or written in 16-byte pieces); ids, lse, row_ptr,
 *    entries and page tables 4-byte aligned.
 *  - Errors found on the host return immediately (nothing enqueued).  Errors a
 *    kernel finds (an id outside [-1, N), a bounded wait that expired) are
 *    OR-ed into a sticky status word at the start of the workspace; kernels
 *    skip the offending work and never trap.  Read it with msa_device_status().
 */
#ifndef MSA_H
#define MSA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MSA_API __attribute__((visibility("default")))
#else
#define MSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum msa_status {
    MSA_OK = 0,
    MSA_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, n_q > T, Hq % Hkv != 0, K < 1 */
    MSA_ERR_UNSUPPORTED = 2, /* valid but outside the supported shapes listed above */
    MSA_ERR_WORKSPACE = 3,   /* workspace pointer null/misaligned or smaller than required */
    MSA_ERR_CUDA = 4,        /* a CUDA runtime call or kernel launch failed */
    MSA_ERR_TIMEOUT = 5,     /* device: a bounded wait inside a kernel expired */
    MSA_ERR_BAD_IDS = 6      /* device: an id outside [-1, N) was seen and skipped */
} msa_status;

/*
 * Bytes of device workspace that msa_index_topk, msa_select_invert and
 * msa_sparse_attn need for these sizes (the maximum over the three; a decode
 * shape, n_q == 1, needs far less than a prefill).  The workspace must be
 * 256-byte aligned.  Its first 256 bytes hold the sticky device status word:
 * zero them once before first use (e.g. cudaMemsetAsync(ws, 0, 256)); the
 * paged-cache attention calls need the whole header of
 * MSA_WORKSPACE_HEADER_BYTES zeroed once.  The rest is scratch that every
 * call overwrites; two calls that overlap in time must not share a workspace.  Returns 0 for arguments the calls would reject.
 *
 * Prefill attention keeps one bf16 partial (and its lse) per (query row,
 * slot, query head) until the log-sum-exp combine; it attends the kv heads in
 * groups and merges each group before the next, so the workspace holds one
 * group's partials.  msa_workspace_size returns the minimum: the largest
 * group (a divisor of Hkv) whose partials fit in about 4 GiB, at least one kv
 * head.  Given a larger workspace, msa_sparse_attn uses the largest group that
 * fits (fewer, longer launches); msa_workspace_size_kv_group gives the size
 * for kv_group kv heads per pass (kv_group = Hkv: a single pass), or 0 if
 * kv_group does not divide Hkv.
 */
#define MSA_WORKSPACE_HEADER_BYTES 2304

MSA_API size_t msa_workspace_size(int Bt, int n_q, int T, int Hq, int Hkv, int d, int d_idx,
                                  int block, int K);

MSA_API size_t msa_workspace_size_kv_group(int Bt, int n_q, int T, int Hq, int Hkv, int d,
                                           int d_idx, int block, int K, int kv_group);

/*
 * Index branch [P2 "索引分支"]: block max-pooled single-head index scores and
 * top-K block selection with the own block forced.  Writes ids (layout above).
 * Prefill (n_q > 1) runs one fused tcgen05 kernel that never materialises the
 * n_q x T score matrix; decode (n_q == 1) streams k_idx once and selects.
 */
MSA_API msa_status msa_index_topk(const void *q_idx, const void *k_idx, int32_t *ids, int Bt,
                                  int n_q, int T, int d_idx, int block, int K, void *workspace,
                                  size_t workspace_bytes, void *stream);

/*
 * Index branch with signed 8-bit index keys: the same selection as
 * msa_index_topk (same layouts and rules) for q_idx [Bt][n_q][d_idx] and
 * k_idx [Bt][T][d_idx] stored as int8 instead of bf16.  The pages' index key
 * is lightweight ([P2 "索引分支"]) and the workloads' keys are small integers,
 * which int8 holds exactly; the scores are then integer dot products,
 * computed exactly (prefill: tcgen05 kind::i8 with s32 accumulation, twice
 * the bf16 tensor-core rate; decode: dp4a over half the bytes of bf16 keys),
 * so the ids equal those of msa_index_topk on the same integer values.
 * Keys that are not integers must go through msa_index_topk instead.
 */
MSA_API msa_status msa_index_topk_i8(const int8_t *q_idx, const int8_t *k_idx, int32_t *ids,
                                     int Bt, int n_q, int T, int d_idx, int block, int K,
                                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * Selection inversion [P4 section 2.2]: the per-query block lists in ids
 * turned into per-block lists of hit queries, in CSR form over the Bt*N
 * (sequence, block) pairs:
 *   row_ptr [Bt*N + 1] int32: list of pair p = b*N + j is
 *           entries[row_ptr[p] .. row_ptr[p+1]);
 *   entries [Bt*n_q*K] int32 (capacity; row_ptr[Bt*N] are used): each entry
 *           is (b*n_q + i)*K + slot with ids[b][i][slot] == j, listed in
 *           ascending query order.
 * msa_sparse_attn performs the same inversion internally (into its
 * workspace); this entry point exposes it on its own.
 */
MSA_API msa_status msa_select_invert(const int32_t *ids, int32_t *row_ptr, int32_t *entries,
                                     int Bt, int n_q, int T, int block, int K, void *workspace,
                                     size_t workspace_bytes, void *stream);

/*
 * Sparse branch [P2 "稀疏分支"; P4 sections 2.2, 2.3]: exact GQA softmax
 * attention over the keys of the selected blocks (causal inside the own block),
 * scale 1/sqrt(d), raw bf16 KV.  Writes out and lse (layouts above).
 * ids must hold, per row, distinct block ids in [0, N) or -1; an id greater
 * than own(t) contributes no key; an id outside [-1, N) is skipped (it
 * contributes no key either) and reported as MSA_ERR_BAD_IDS.  Prefill (n_q > 1): inversion, a
 * KV-block-outer tcgen05 kernel that loads each selected KV block into shared
 * memory and gathers its hit queries, then a log-sum-exp combine of the per
 * slot partials.  With blocks longer than 128 keys, each row's own block is
 * left out of the hit lists and attended by a second, causal launch of the
 * kernel over the consecutive rows of each block, which skips the 128-key
 * sub-tiles past each chunk's last row.  Decode (n_q == 1): a split-K kernel
 * over the selected blocks, then the same combine.
 */
MSA_API msa_status msa_sparse_attn(const void *q, const void *k, const void *v,
                                   const int32_t *ids, float *out, float *lse, int Bt, int n_q,
                                   int T, int Hq, int Hkv, int d, int block, int K,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Paged KV for decode [P4 section 3.2, "MSA 如何降低显存压力": page-managed
 * KV cache; its 4-bit quantisation is not followed, KV stays raw bf16].
 * Same computation as msa_index_topk / msa_sparse_attn for a decode step
 * (n_q = 1, the query at t = T-1), with k_idx, K and V held in pages of
 * `block` rows instead of contiguous [Bt][T] rows:
 *   page_table  [Bt][page_stride] int32 (device): logical block j of
 *               sequence b is physical page page_table[b*page_stride + j],
 *               for j < N = ceil(T / block); page_stride >= N.
 *   k_idx_pages [num_pages][block][d_idx] bf16;
 *   k_pages, v_pages [num_pages][block][Hkv][d] bf16 (16-byte aligned).
 * Rows past T in the last logical block are never read.  The caller owns
 * all buffers; the workspace is msa_workspace_size(Bt, 1, T, ...).  A page id
 * outside [0, num_pages) is skipped and reported as MSA_ERR_BAD_IDS through
 * the status word (msa_device_status).  Host-detected errors as above.
 */
MSA_API msa_status msa_index_topk_paged(const void *q_idx, const void *k_idx_pages,
                                        const int32_t *page_table, int page_stride,
                                        int num_pages, int32_t *ids, int Bt, int T, int d_idx,
                                        int block, int K, void *workspace,
                                        size_t workspace_bytes, void *stream);

MSA_API msa_status msa_sparse_attn_paged(const void *q, const void *k_pages, const void *v_pages,
                                         const int32_t *page_table, int page_stride,
                                         int num_pages, const int32_t *ids, float *out,
                                         float *lse, int Bt, int T, int Hq, int Hkv, int d,
                                         int block, int K, void *workspace,
                                         size_t workspace_bytes, void *stream);

/*
 * Paged cache of a batch: writing it, reading it back, attending over it.
 * ------------------------------------------------------------------------
 * [P4 section 3.2] manages the KV cache in pages.  The calls below keep that
 * cache (the page stores of msa_sparse_attn_paged, or 8-bit ones) and serve
 * the layers around the sparse branch: dense attention of new tokens over
 * their whole context, and attention in a window with first tokens that stay
 * visible.  A step of a batch is described by two device arrays:
 *   cu      [Bt + 1] int32: packed rows cu[b] .. cu[b+1]-1 belong to sequence
 *           b (cu[0] = 0, ascending); rows at or behind cu[Bt] do not matter
 *           and are not written, so a padded buffer needs no copy;
 *   kv_len  [Bt] int32: length of each context, this step's tokens included.
 * Row i of the n_b = cu[b+1] - cu[b] rows of sequence b stands at position
 * t = kv_len[b] - n_b + i.  The arrays are read when the kernels run: a
 * captured step follows the lengths in them.  `total` is the number of rows
 * that the packed buffers hold.  Where a row's position is negative, nothing
 * is cached for it and it sees no key.
 *
 * Page stores: bf16 [num_pages][block][Hkv][d], or int8 codes of that shape
 * with fp32 scales [num_pages][Hkv][block]: a cached row is code * scale.  As
 * it is written, a row x of d values gets (all in fp32)
 *     amax = max |x_i|, inv = 127 / amax, code_i = rint(x_i * inv), scale = amax / 127.
 * Rows with amax < 2^-100 are stored as zeros; a row that holds an infinity
 * or a NaN gets scale NaN, so that it reads back as NaN.  Scales that a
 * caller brings from elsewhere are not negative.
 *
 * Pages are found as in the paged decode calls above: logical block j of
 * sequence b is page_table[b*page_stride + j].  A page id outside
 * [0, num_pages), or a position that the table's row cannot hold, is skipped
 * and reported as MSA_ERR_BAD_IDS in the status word (msa_device_status).
 * Limits (MSA_ERR_UNSUPPORTED): d, d_idx in {64, 128}; block 32, 64 or a
 * multiple of 128; num_pages*block < 2^31; page_stride*block, total < 2^30;
 * total*Hkv*d < 2^33 (append, gather); total*Hq < 2^31; attention: fewer than
 * 2^31 (row tile, kv head, 128 keys) triples, counted with the page table's
 * whole width (or the window).  Any Hq that Hkv divides.  Row strides (elements) are multiples of 8 and at least a row
 * long: k, v and q may be parts of one projection's output.  All base
 * pointers are 16-byte aligned but for int32 arrays and lse (4).  total = 0
 * is a step without rows: MSA_OK, nothing enqueued.
 *
 * msa_cache_workspace_size: bytes of workspace for all calls of this section
 * (0 for arguments that they reject).  256-byte aligned, as msa_workspace_size
 * describes: zero the first MSA_WORKSPACE_HEADER_BYTES once before first use.
 * Behind the status word the header holds counters that every attention call
 * leaves at zero; no other call of this library writes them.  Append and
 * gather use the status word only.
 */
MSA_API size_t msa_cache_workspace_size(int Hq, int Hkv, int d);

/*
 * The step's new rows k, v ([total] rows of Hkv*d bf16 values every k_stride /
 * v_stride elements) into the pages of their positions, and, unless k_idx and
 * k_idx_pages are both NULL, the index keys k_idx ([total] rows of d_idx bf16
 * values) into k_idx_pages [num_pages][block][d_idx].  Rows of the stores that
 * no new row maps to are left as they were.  Two rows of one call must not
 * map to the same place.
 */
MSA_API msa_status msa_kv_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                 const void *k_idx, int64_t k_idx_stride, void *k_pages,
                                 void *v_pages, void *k_idx_pages, const int32_t *page_table,
                                 int page_stride, int num_pages, const int32_t *cu,
                                 const int32_t *kv_len, int Bt, int total, int Hkv, int d,
                                 int d_idx, int block, void *workspace, size_t workspace_bytes,
                                 void *stream);

MSA_API msa_status msa_kv_append_i8(const void *k, int64_t k_stride, const void *v,
                                    int64_t v_stride, const void *k_idx, int64_t k_idx_stride,
                                    int8_t *k_pages, int8_t *v_pages, float *k_scales,
                                    float *v_scales, void *k_idx_pages, const int32_t *page_table,
                                    int page_stride, int num_pages, const int32_t *cu,
                                    const int32_t *kv_len, int Bt, int total, int Hkv, int d,
                                    int d_idx, int block, void *workspace, size_t workspace_bytes,
                                    void *stream);

/*
 * The cached rows of the step's positions as packed bf16 k, v [total][Hkv][d]
 * (n_b = kv_len[b] reads whole contexts back, e.g. for the contiguous prefill
 * calls).  int8: code * scale in fp32, rounded once.  Rows whose position is
 * negative or whose page does not exist are zeros.
 */
MSA_API msa_status msa_kv_gather(const void *k_pages, const void *v_pages,
                                 const int32_t *page_table, int page_stride, int num_pages,
                                 const int32_t *cu, const int32_t *kv_len, void *k, void *v,
                                 int Bt, int total, int Hkv, int d, int block, void *workspace,
                                 size_t workspace_bytes, void *stream);

MSA_API msa_status msa_kv_gather_i8(const int8_t *k_pages, const int8_t *v_pages,
                                    const float *k_scales, const float *v_scales,
                                    const int32_t *page_table, int page_stride, int num_pages,
                                    const int32_t *cu, const int32_t *kv_len, void *k, void *v,
                                    int Bt, int total, int Hkv, int d, int block, void *workspace,
                                    size_t workspace_bytes, void *stream);

/*
 * Attention of the step's rows over their cached contexts (append first: the
 * step's own tokens are read from the pages).  q: [total] rows of Hq*d bf16
 * values every q_stride elements.  A query at position t sees the keys
 *     j <= t  with  window == 0  or  j > t - window  or  j < sinks
 * (window > 0: the last `window` keys, itself among them, and the first
 * `sinks` ones; sinks is ignored without a window).  Scale 1/sqrt(d).  Pages
 * that lie wholly before every window and behind the sinks are not looked up:
 * their table entries may be stale.
 * out [total][Hq][d] bf16 (fp32 sums, rounded once), lse [total][Hq] fp32
 * (natural log); a row that sees no key gets out 0 and lse -inf.
 * max_q: the largest n_b of the step, or 0 if the caller does not know it; it
 * chooses between kernels and changes no result beyond rounding.  Give it: a
 * step of single tokens without it is taken for a chunk of Bt tokens, which
 * finds its way to the right kernel by a longer path (8 heads per kv head, 32
 * contexts of up to 32768 keys: 297 instead of 182 us on int8 pages, 317 instead
 * of 301 on bf16 ones).
 * Precision: scores, weights' sums and outputs are summed in fp32.  Steps of few
 * rows keep 15 bits of the weights (bf16 pages) or 23 below the largest of 128
 * keys (int8 pages), steps of many rows 8 (a bf16).  Few rows on int8 pages:
 * values of q below 2^-12 of their row's largest are rounded to multiples of
 * 2^-19 of it.  Many rows: weights go up to 256 before they are divided by their
 * sum, so values of V beyond 2^100 or so may leave the range of fp32.
 * Cache rows at or past kv_len[b], and rows that no row of the step sees, do
 * not matter, whatever they hold.  A key that one row of the step sees and
 * another does not must have finite values in v_pages (bf16); an infinity on a
 * key that every row sees reaches the outputs as it is.
 */
MSA_API msa_status msa_attn_paged(const void *q, int64_t q_stride, const void *k_pages,
                                  const void *v_pages, const int32_t *page_table, int page_stride,
                                  int num_pages, const int32_t *cu, const int32_t *kv_len,
                                  void *out, float *lse, int Bt, int total, int max_q, int Hq,
                                  int Hkv, int d, int block, int window, int sinks,
                                  void *workspace, size_t workspace_bytes, void *stream);

MSA_API msa_status msa_attn_paged_i8(const void *q, int64_t q_stride, const int8_t *k_pages,
                                     const int8_t *v_pages, const float *k_scales,
                                     const float *v_scales, const int32_t *page_table,
                                     int page_stride, int num_pages, const int32_t *cu,
                                     const int32_t *kv_len, void *out, float *lse, int Bt,
                                     int total, int max_q, int Hq, int Hkv, int d, int block,
                                     int window, int sinks, void *workspace,
                                     size_t workspace_bytes, void *stream);

/*
 * The kernels that msa_attn_paged and msa_attn_paged_i8 launch for a step of
 * these sizes (profiling and tests): MSA_KERNEL_SPLIT, MSA_KERNEL_CHUNK or both,
 * where the chunk kernel takes the sequences with more than 16 rows (n_b * Hq /
 * Hkv) and the split kernel the others; 0 for sizes without work or outside the
 * limits above (but for that on triples, which depends on the device).  Host
 * only: no CUDA call is made.
 */
#define MSA_KERNEL_SPLIT 1
#define MSA_KERNEL_CHUNK 2
MSA_API int msa_attn_paged_kernels(int Bt, int total, int max_q, int Hq, int Hkv, int block,
                                   int page_stride, int window, int sinks);

/*
 * The sparse branch of a decode step on int8 pages: msa_sparse_attn_paged
 * (same ids, same keys) with the 8-bit stores and the output types of this
 * section: out [Bt][1][Hq][d] bf16, lse [Bt][1][Hq] fp32.  K <= 32,
 * K*block < 2^30.
 */
MSA_API msa_status msa_sparse_attn_paged_i8(const void *q, const int8_t *k_pages,
                                            const int8_t *v_pages, const float *k_scales,
                                            const float *v_scales, const int32_t *page_table,
                                            int page_stride, int num_pages, const int32_t *ids,
                                            void *out, float *lse, int Bt, int T, int Hq, int Hkv,
                                            int d, int block, int K, void *workspace,
                                            size_t workspace_bytes, void *stream);

/*
 * Instrumented variants (profiling): the same work as msa_index_topk and
 * msa_sparse_attn, with optional CUDA events recorded on `stream`
 * immediately before (start[i]) and after (stop[i]) the kernels of stage i.
 * Each non-NULL entry must be a cudaEvent_t created on the current device;
 * `events` itself may be NULL.  Stages:
 *   msa_index_topk_ev, msa_index_topk_i8_ev:
 *                       0 = index kernel (prefill) or k_idx scan (decode);
 *                       1 = top-K select (decode only).
 *   msa_sparse_attn_ev: 0 = selection inversion (prefill only);
 *                       1 = attention kernel (KV-block-outer: the hit-list
 *                           launch and, for blocks longer than 128 keys, the
 *                           own-block launch; or split-K);
 *                       2 = log-sum-exp combine.
 *   A prefill that attends its kv heads in several groups (see
 *   msa_workspace_size) records stage 1 from the first group's attention to
 *   the last group's, which spans the combines of all groups but the last,
 *   and stage 2 around the last group's combine.
 */
#define MSA_MAX_STAGES 4
typedef struct msa_stage_events {
    void *start[MSA_MAX_STAGES];
    void *stop[MSA_MAX_STAGES];
} msa_stage_events;

MSA_API msa_status msa_index_topk_ev(const void *q_idx, const void *k_idx, int32_t *ids, int Bt,
                                     int n_q, int T, int d_idx, int block, int K,
                                     void *workspace, size_t workspace_bytes, void *stream,
                                     const msa_stage_events *events);

MSA_API msa_status msa_index_topk_i8_ev(const int8_t *q_idx, const int8_t *k_idx, int32_t *ids,
                                        int Bt, int n_q, int T, int d_idx, int block, int K,
                                        void *workspace, size_t workspace_bytes, void *stream,
                                        const msa_stage_events *events);

MSA_API msa_status msa_sparse_attn_ev(const void *q, const void *k, const void *v,
                                      const int32_t *ids, float *out, float *lse, int Bt,
                                      int n_q, int T, int Hq, int Hkv, int d, int block, int K,
                                      void *workspace, size_t workspace_bytes, void *stream,
                                      const msa_stage_events *events);

/*
 * Decode attention that allocates nothing.  The pages have no counterpart:
 * this entry point is an addition of this library for callers that cannot
 * allocate device memory or hand over a workspace -- for example a serving
 * engine or plugin host that has already given all device memory to its own
 * pool, where a cudaMalloc would fail or stall the whole device, and which
 * has no spare buffer to pass as workspace.
 *
 * It computes exactly what msa_sparse_attn computes for a decode step (n_q = 1,
 * same layouts, same split-K and combine kernels), but its scratch (the
 * per-split partials) is a file-scope static __device__ array of
 * MSA_NOALLOC_SCRATCH_BYTES (16 MiB).  That array is part of the library
 * image: every GPU on which it has been loaded holds it until the process
 * exits.  The caller still owns and passes every input and output.
 *   - Limit: 256 + align256(Bt*K*S*Hq*d*4) + align256(Bt*K*S*Hq*4) bytes must
 *     fit in the array, with S = ceil(block / 64); otherwise the call returns
 *     MSA_ERR_WORKSPACE before enqueueing anything.  (The 4-sequence
 *     1M-context decode, Bt 4, K 8, block 512, Hq 64, d 128, needs 8.5 MB.)
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) and caches it; make that first call before any
 *     stream capture begins.  The cached address belongs to the device's
 *     primary context: after cudaDeviceReset, or when calling from another
 *     driver context on the same device, it is stale and must not be used.
 *   - Every call uses the same array, which keeps the contents of the last
 *     call.  Calls whose kernels overlap on the GPU (two streams, or two host
 *     threads) race on it and must be serialised by the caller.
 *   - status: optional device int.  Kernels OR 2 into it when they skip an id
 *     outside [-1, N).  With NULL those reports are dropped.
 * No cudaMalloc, cudaFree or allocating library routine is called.
 */
#define MSA_NOALLOC_SCRATCH_BYTES (16u << 20)

MSA_API msa_status msa_sparse_attn_decode_noalloc(const void *q, const void *k, const void *v,
                                                  const int32_t *ids, float *out, float *lse,
                                                  int Bt, int T, int Hq, int Hkv, int d,
                                                  int block, int K, int *status, void *stream);

/*
 * Synchronises `stream`, then reads and clears the sticky device status word
 * of `workspace`: MSA_OK, MSA_ERR_TIMEOUT or MSA_ERR_BAD_IDS (the first found,
 * in that order of precedence: timeout first), or MSA_ERR_CUDA if the
 * synchronisation or the copy failed.
 */
MSA_API msa_status msa_device_status(void *workspace, void *stream);

/* Static, NUL-terminated name of a status code ("unknown status" otherwise). */
MSA_API const char *msa_status_string(int status);

/*
 * Tensor-core self-test, not part of the method: C[128][N] = A . B with
 * A [128][Kd] bf16 (K-major) and B either as [N][Kd] (bit 0 of b_mn_major = 0,
 * K-major) or as [Kd][N] (bit 0 = 1), C fp32, through the same TMA,
 * shared-memory descriptor, tcgen05.mma and TMEM read-back code the attention
 * kernels use.  Bit 1 of b_mn_major set: A is first copied into tensor memory
 * and the MMA reads it from there (the layout the attention kernel uses for P).
 * N in {64, 128, 256}, Kd a multiple of 64 up to 256.  Device pointers;
 * `status` is a device int the kernel sets non-zero on a wait timeout.
 */
MSA_API msa_status msa_selftest_umma(const void *A, const void *B, float *C, int N, int Kd,
                                     int b_mn_major, int *status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H */

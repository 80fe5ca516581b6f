/*
 * jgdpa.h - C ABI of libjgdpa.so: jagged Generalized Dot-Product Attention
 * (GDPA) forward and backward on one GB300 GPU (sm_103a).
 *
 * What is computed.  For every segment b and head h, with segment-local query
 * rows i < Lq_b and key/value rows j < Lkv_b, and valid(i,j) = (not causal or
 * j <= i):
 *
 *     x_ij = scale * <q_i, k_j> + bias[h][clamp(i - j, -R, R) + R]
 *     GELU / SiLU mode:  O_i = sum_{valid j} act(x_ij) * v_j   (no normalisation)
 *     SOFTMAX mode:      O_i = sum_{valid j} softmax_j(x_ij) * v_j,
 *                        LSE_i = log sum_{valid j} exp(x_ij)
 *
 * Sources: "GEM Training: How Meta Doubled the Efficiency of Its ..."
 * (globalainews.in), section "What to watch" -- self-attention, PMA and
 * cross-attention are two matrix multiplications with an element-wise
 * activation (GELU or SiLU) in place of softmax, unified in one GDPA kernel;
 * section "What happened" -- Jagged Flash Attention works directly on jagged
 * tensors with custom attention biases, asymmetric query/key-value lengths and
 * a backward pass.  "Meta redesigns AI training infrastructure to solve
 * trillion-parameter ad recommendation bottlenecks" (aiuniverse.news),
 * sections "Eliminating Compute Waste in Asymmetric Workloads" and "Custom
 * Kernels and 5D Parallelism for Trillion-Parameter Scale" -- the jagged
 * masking, the software tile scheduler and the split-dQ backward.
 *
 * The pages print no formula; where they are silent this library reads them
 * as follows: no normalisation in GELU/SiLU mode; GELU means x*Phi(x) (the
 * device evaluates an approximation of it); the bias is a per-head table of
 * bias_len = 2R+1 entries indexed by clamp(i-j, -R, R)+R with segment-local
 * i, j and is added after scaling; causal masking is top-left aligned
 * (j <= i); a query row with no valid key gets O_i = 0 (and LSE_i = -inf).
 *
 * Conventions shared by every call:
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    allocates and frees nothing and keeps no per-call state.
 *  - Calls are asynchronous and ordered on `stream`; they return before the
 *    kernels run.  The stream must belong to the current device.
 *  - Q, K, V, O and their gradients are bf16, packed "THD": [total][H][d],
 *    row-major, with no padding between segments.  The base pointers must be
 *    16-byte aligned.  Segment b owns query rows q_offsets[b] ..
 *    q_offsets[b+1]-1 and key/value rows kv_offsets[b] .. kv_offsets[b+1]-1.
 *  - Offsets are int32 [batch+1] device arrays with offsets[0] = 0,
 *    non-decreasing, and offsets[batch] equal to total_q (total_kv).
 *  - Outputs are overwritten, never accumulated; rows of segments with no keys
 *    (or no queries, for dK/dV) are written as zeros.
 *  - head_dim is 32, 64 or 128; heads >= 1; bias_len is 0 or odd (<= 4095).
 *  - Errors that the host can see are returned before anything is launched.
 *    Errors that only the device can see (bad offsets, an internal wait that
 *    timed out) are recorded in the workspace status word, turn the remaining
 *    kernels into no-ops, and are read back with jgdpa_read_device_status().
 *  - `workspace` is caller-owned device scratch of at least
 *    jgdpa_workspace_bytes(...) bytes, 256-byte aligned; its contents need no
 *    initialisation and are clobbered by every call.  Two calls that overlap
 *    in time must not share a workspace.
 */
#ifndef JGDPA_H
#define JGDPA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define JGDPA_API __attribute__((visibility("default")))
#else
#define JGDPA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* jgdpa_stream_t;  /* a cudaStream_t (NULL = legacy default stream) */

typedef enum {
    JGDPA_ACT_GELU = 0,     /* act(x) = x * Phi(x) */
    JGDPA_ACT_SILU = 1,     /* act(x) = x * sigmoid(x) */
    JGDPA_ACT_SOFTMAX = 2   /* Jagged Flash Attention: softmax over the valid keys */
} jgdpa_act;

typedef enum {
    JGDPA_OK = 0,
    JGDPA_ERR_INVALID_ARGUMENT = 1,   /* null pointer, negative size, bad enum, even bias_len */
    JGDPA_ERR_UNSUPPORTED = 2,        /* head_dim not in {32, 64, 128}, sizes beyond int32 rows */
    JGDPA_ERR_MISALIGNED = 3,         /* a tensor or the workspace is not suitably aligned */
    JGDPA_ERR_WORKSPACE_TOO_SMALL = 4,  /* workspace (or the no-alloc array) too small for the sizes */
    JGDPA_ERR_CUDA = 5,               /* a CUDA runtime call or launch failed */
    JGDPA_ERR_BAD_OFFSETS = 6,        /* device-detected: offsets not monotone / wrong ends */
    JGDPA_ERR_DEVICE_TIMEOUT = 7,     /* device-detected: an internal wait gave up */
    JGDPA_ERR_OUT_OF_PAGES = 8,       /* device-detected: the pool has too few free pages */
    JGDPA_ERR_BAD_PAGE = 9            /* device-detected: a block table entry outside the cache */
} jgdpa_status;

/*
 * Bytes of device workspace that jgdpa_fwd (for_backward = 0) or jgdpa_bwd
 * (for_backward = 1) needs for these sizes.  Depends only on the arguments
 * and on the number of SMs of the current device.  Returns 0 if the arguments
 * are invalid.
 */
JGDPA_API size_t jgdpa_workspace_bytes(int32_t batch, int64_t total_q, int64_t total_kv,
                             int32_t heads, int32_t head_dim, jgdpa_act act,
                             int32_t bias_len, int32_t for_backward);

/*
 * Forward pass.
 *   q        bf16 [total_q][heads][head_dim]
 *   k, v     bf16 [total_kv][heads][head_dim]
 *   scale    the factor s on <q_i, k_j> (typically 1/sqrt(head_dim))
 *   bias_table  fp32 [heads][bias_len], or NULL with bias_len = 0
 *   causal   0 or 1 (top-left aligned: key j is visible to query i iff j <= i)
 *   out      bf16 [total_q][heads][head_dim], written
 *   lse      fp32 [heads][total_q], natural-log log-sum-exp of each row;
 *            required in SOFTMAX mode (needed by jgdpa_bwd), must be NULL
 *            otherwise
 * Work runs in a persistent kernel over (segment, head, pair of 128-row query
 * tiles) units ordered longest first by a scheduling kernel (the software tile
 * scheduler of the GDPA kernel redesign, "Custom Kernels and 5D Parallelism
 * ...", aiuniverse.news).
 */
JGDPA_API jgdpa_status jgdpa_fwd(const void* q, const void* k, const void* v,
                       const int32_t* q_offsets, const int32_t* kv_offsets,
                       int32_t batch, int64_t total_q, int64_t total_kv,
                       int32_t heads, int32_t head_dim, jgdpa_act act, float scale,
                       const float* bias_table, int32_t bias_len, int32_t causal,
                       void* out, float* lse,
                       void* workspace, size_t workspace_bytes, jgdpa_stream_t stream);

/*
 * Forward pass with a sliding window: the same computation, arguments and
 * errors as jgdpa_fwd, plus
 *   window   0 (no window, exactly jgdpa_fwd) or w >= 1: only pairs with
 *            |i - j| < w (segment-local) are attended, on top of the
 *            length and causal conditions; negative -> INVALID_ARGUMENT.
 * Sliding window attention is named for long sequences in "Meta redesigns AI
 * training infrastructure ..." (aiuniverse.news), section "Custom Kernels
 * and 5D Parallelism ...", without a definition; this symmetric band, with
 * the same segment-local indices as the bias and causal rules, is the reading
 * taken.  Key/value tiles wholly outside the band are neither loaded nor
 * computed, and the scheduler costs units by the tiles they visit.  A query
 * row that meets no key gets O = 0 (and LSE = -inf in SOFTMAX mode).
 */
JGDPA_API jgdpa_status jgdpa_fwd_ex(const void* q, const void* k, const void* v,
                       const int32_t* q_offsets, const int32_t* kv_offsets,
                       int32_t batch, int64_t total_q, int64_t total_kv,
                       int32_t heads, int32_t head_dim, jgdpa_act act, float scale,
                       const float* bias_table, int32_t bias_len, int32_t causal, int32_t window,
                       void* out, float* lse,
                       void* workspace, size_t workspace_bytes, jgdpa_stream_t stream);

/*
 * Backward pass: gradients of L = sum(O * dout) with respect to q, k, v and
 * the bias table.
 *   out, lse   the forward's O and LSE; read in SOFTMAX mode only (may be NULL
 *              otherwise)
 *   dout       bf16 [total_q][heads][head_dim]
 *   dq         bf16 [total_q][heads][head_dim], written
 *   dk, dv     bf16 [total_kv][heads][head_dim], written
 *   dbias      fp32 [heads][bias_len], written; NULL to skip (must be NULL
 *              when bias_table is NULL)
 * dK/dV come from a KV-major pass and dQ from a separate Q-major pass, so
 * every output tile has exactly one writer and no atomics touch dQ, dK or dV
 * (the split-dQ, atomics-free backward of "Eliminating Compute Waste in
 * Asymmetric Workloads", aiuniverse.news).
 */
JGDPA_API jgdpa_status jgdpa_bwd(const void* q, const void* k, const void* v,
                       const void* out, const float* lse, const void* dout,
                       const int32_t* q_offsets, const int32_t* kv_offsets,
                       int32_t batch, int64_t total_q, int64_t total_kv,
                       int32_t heads, int32_t head_dim, jgdpa_act act, float scale,
                       const float* bias_table, int32_t bias_len, int32_t causal,
                       void* dq, void* dk, void* dv, float* dbias,
                       void* workspace, size_t workspace_bytes, jgdpa_stream_t stream);

/*
 * Bytes of stored-dS scratch that jgdpa_bwd_ex needs for these segment
 * lengths and window: heads * sum_b nk_b * span_b tiles of 32 KB, with
 * nq_b = ceil(Lq_b/128), nk_b = ceil(Lkv_b/128), and span_b = nq_b, or under
 * a window w > 0 the 2e + 1 query tiles one key tile can meet
 * (e = ceil((w - 1)/128)) when that is fewer.  q_offsets_host /
 * kv_offsets_host are HOST copies of the offsets ([batch + 1] each); window
 * as in jgdpa_bwd_ex.  Returns 0 for invalid arguments (and for batch 0).
 */
JGDPA_API size_t jgdpa_ds_scratch_bytes(const int32_t* q_offsets_host, const int32_t* kv_offsets_host,
                                        int32_t batch, int32_t heads, int32_t window);

/*
 * Backward pass, extended.  The same computation, arguments and errors as
 * jgdpa_bwd, plus:
 *   window
 *       0 (no window) or w >= 1: the sliding window of jgdpa_fwd_ex; pass
 *       the forward's window (and its out / lse in SOFTMAX mode).
 *   ds_scratch, ds_scratch_bytes
 *       optional caller-owned device scratch (256-byte aligned) for the
 *       stored-dS backward; NULL selects the recompute backward of
 *       jgdpa_bwd.  With scratch the dK/dV pass writes every bf16 dS tile it
 *       forms to the scratch and the dQ pass is one streaming matmul
 *       dQ = s * dS K over the stored tiles, instead of recomputing S, dP and
 *       the activation derivative.  jgdpa_ds_scratch_bytes(...) bytes hold
 *       every segment's tiles; a smaller scratch is used as far as it goes:
 *       the tiles are laid out segment by segment, the segments whose tiles
 *       end within the scratch get the stored-dS dQ and the others (a suffix
 *       of the batch) get their dQ by recomputation, so the results are the
 *       same up to rounding whatever the scratch size.  A scratch smaller
 *       than one tile (32 KB) is not used.  The scratch contents need no
 *       initialisation and are clobbered.
 *   pass_events
 *       optional three CUDA events (cudaEvent_t, created by the caller on the
 *       current device; any entry, or pass_events itself, may be NULL),
 *       recorded on `stream` right before the dK/dV pass kernel, between the
 *       dK/dV and dQ pass kernels, and right after the dQ pass kernel, so
 *       that cudaEventElapsedTime gives each pass's duration.
 */
JGDPA_API jgdpa_status jgdpa_bwd_ex(const void* q, const void* k, const void* v,
                       const void* out, const float* lse, const void* dout,
                       const int32_t* q_offsets, const int32_t* kv_offsets,
                       int32_t batch, int64_t total_q, int64_t total_kv,
                       int32_t heads, int32_t head_dim, jgdpa_act act, float scale,
                       const float* bias_table, int32_t bias_len, int32_t causal, int32_t window,
                       void* dq, void* dk, void* dv, float* dbias,
                       void* workspace, size_t workspace_bytes,
                       void* ds_scratch, size_t ds_scratch_bytes, jgdpa_stream_t stream,
                       void* const* pass_events);

/*
 * Shared query rows (PMA-style pooling): every segment attends with the same
 * n_shared = S query rows, e.g. learned seed queries shared across the batch
 * ("GEM Training: How Meta Doubled the Efficiency of Its ..."
 * (globalainews.in), section "What to watch": PMA is one of the modules GDPA
 * serves).  Segment b's query row i (0 <= i < S) is row i of q; its output,
 * upstream gradient and LSE rows are b S + i.  The computation is otherwise
 * that of jgdpa_fwd_ex / jgdpa_bwd_ex with Lq_b = S for every segment, and
 * the gradient of the shared rows is the sum over segments of each
 * segment's dQ.
 *   q          bf16 [S][heads][head_dim], read by every segment (not expanded)
 *   out, dout  bf16 [batch S][heads][head_dim]
 *   lse        fp32 [heads][batch S] (SOFTMAX mode only, else NULL)
 *   dq         bf16 [S][heads][head_dim], written: sum over b of dQ_b,
 *              accumulated in fp32 in a fixed order (the same bits on every
 *              run) and rounded once
 *   kv_offsets, k, v, dk, dv, bias_table, dbias, causal, window, ds_scratch,
 *   pass_events
 *              as in jgdpa_bwd_ex (there are no query offsets: they are S b,
 *              formed in the workspace; the stored-dS scratch size is
 *              jgdpa_ds_scratch_bytes with query offsets S b)
 * The workspace must hold jgdpa_shared_q_workspace_bytes(...) bytes; what
 * the backward keeps there depends on S:
 *   S <= 64 with GELU / SiLU: the short-query kernels (the keys take the
 *     MMA's 128 rows, the S queries are its N).  The backward writes one
 *     fp32 [S][head_dim] dQ contribution per (segment, head, chunk of up to
 *     16 key tiles) and sums them in a fixed order; ds_scratch is not used.
 *   S <= 128 and head_dim <= 64 otherwise: the key-major pass writes one such
 *     contribution per (segment, head, key tile); ds_scratch is not used.
 *   otherwise: each segment's dQ rows in fp32 ([batch S][heads][head_dim]),
 *     summed in segment order; ds_scratch as in jgdpa_bwd_ex.
 * Errors as in
 * jgdpa_fwd / jgdpa_bwd; n_shared < 1 is INVALID_ARGUMENT, batch S beyond
 * int32 is UNSUPPORTED.
 */
JGDPA_API size_t jgdpa_shared_q_workspace_bytes(int32_t batch, int32_t n_shared, int64_t total_kv,
                                                int32_t heads, int32_t head_dim, jgdpa_act act,
                                                int32_t bias_len, int32_t for_backward);
JGDPA_API jgdpa_status jgdpa_fwd_shared_q(const void* q, int32_t n_shared, const void* k, const void* v,
                                          const int32_t* kv_offsets, int32_t batch, int64_t total_kv,
                                          int32_t heads, int32_t head_dim, jgdpa_act act, float scale,
                                          const float* bias_table, int32_t bias_len, int32_t causal,
                                          int32_t window, void* out, float* lse,
                                          void* workspace, size_t workspace_bytes, jgdpa_stream_t stream);
JGDPA_API jgdpa_status jgdpa_bwd_shared_q(const void* q, int32_t n_shared, const void* k, const void* v,
                                          const void* out, const float* lse, const void* dout,
                                          const int32_t* kv_offsets, int32_t batch, int64_t total_kv,
                                          int32_t heads, int32_t head_dim, jgdpa_act act, float scale,
                                          const float* bias_table, int32_t bias_len, int32_t causal,
                                          int32_t window, void* dq, void* dk, void* dv, float* dbias,
                                          void* workspace, size_t workspace_bytes,
                                          void* ds_scratch, size_t ds_scratch_bytes, jgdpa_stream_t stream,
                                          void* const* pass_events);

/*
 * Paged key/value cache: attention from a few new tokens per request over the
 * keys and values that earlier calls left in GPU memory (serving, without
 * gradients).  The computation is that of jgdpa_fwd_ex -- the same act, scale,
 * bias table, window and softmax mode -- with these segments:
 *
 *  - A page holds page_size (a power of two, 16 to 1024) consecutive tokens of
 *    one request, bf16 [page_size][kv_heads][head_dim]; the cache is num_pages
 *    of them, page_stride elements apart (at least a page, a multiple of 8:
 *    the cache may be one layer's or one half's slice of a larger pool).
 *    Token j of request b lies in page block_table[b][j / page_size], place
 *    j % page_size; slot = page * page_size + place.
 *  - Request b has kv_lens[b] tokens.  The last T_b = q_offsets[b + 1] -
 *    q_offsets[b] of them are this step's new tokens (their keys and values
 *    already in the cache), the C_b = kv_lens[b] - T_b before them its context.
 *  - Requests per call: at most 16384.  Rows of q, slots and outputs behind
 *    q_offsets[batch] (a padded batch) are allowed and left as they were.
 */

/*
 * Hands out pages and slots for a step's tokens, on the GPU.  For request b:
 *   ctx_lens[b]    tokens it keeps (what earlier steps left, or fewer: drafted
 *                  tokens that were not accepted; 0 for a new or ended request)
 *   new_lens[b]    tokens it adds
 *   held_pages[b]  pages it holds, the first entries of its table row
 * It comes to want_b = ceil((ctx + new) / page_size) pages: the pages
 * block_table[b][want .. held) go back to the pool, or block_table[b][held ..
 * want) are taken from it.  free_pages[0 .. free_count[0]) is the stack of free
 * pages (capacity num_pages).  All returned pages go onto it first, in (request,
 * page) order, then pages are taken off its top in the same order; the result
 * is the same on every run.
 *   block_table    int32 [batch][table_width], updated in place (the entries
 *                  taken; the others are left as they were)
 *   free_pages     int32 [num_pages], updated in place (the entries above the
 *                  old count that hold returned pages)
 *   free_count     int32 [1]; the new count goes to free_count_out [1]
 *   held_out       int32 [batch], the new page counts want_b
 *   q_offsets      int32 [batch + 1], kv_lens int32 [batch]: for
 *                  jgdpa_cache_fwd
 *   slots          int32 [total_new], the slot of each new token in request
 *                  order; -1 in rows behind the last
 * The outputs that are not updated in place must not overlap the inputs or one
 * another, and a page must stand at most once in the stack and the rows' held
 * entries.  The same call on the same inputs may be repeated: it writes the same
 * values.
 * Device-detected errors: BAD_OFFSETS (negative lengths, more tokens than
 * table_width pages or total_new rows hold, counts beyond num_pages),
 * OUT_OF_PAGES.  Such a call hands out nothing: table and stack are not
 * touched, held_out, free_count_out and kv_lens are the old counts and
 * ctx_lens, q_offsets is all 0 and slots all -1, so that an append and an
 * attention call that follow on the stream do nothing.  A page id outside
 * [0, num_pages) gives slot -1.
 * The workspace (jgdpa_cache_plan_workspace_bytes()) holds the status word;
 * NULL if it will not be read.
 */
JGDPA_API size_t jgdpa_cache_plan_workspace_bytes(void);
JGDPA_API jgdpa_status jgdpa_cache_plan(const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* held_pages,
                                        int32_t batch, int32_t page_size, int32_t* block_table, int32_t table_width,
                                        int32_t* free_pages, int32_t num_pages, const int32_t* free_count,
                                        int32_t total_new, int32_t* held_out, int32_t* free_count_out,
                                        int32_t* q_offsets, int32_t* kv_lens, int32_t* slots,
                                        void* workspace, size_t workspace_bytes, jgdpa_stream_t stream);

/*
 * Writes new keys and values into the cache: row r of k_new and v_new (bf16,
 * [kv_heads][head_dim], rows k_stride / v_stride elements apart, multiples of
 * 8) to slot slots[r]; rows whose slot is negative or beyond the cache are
 * skipped.  Rows of one call must have different slots, and k_new / v_new must
 * not overlap the cache.  After a tree of drafted tokens was checked, the same
 * call moves the accepted ones to their places: k_new and v_new once more, with
 * the accepted rows' new slots and -1 for the others.
 */
JGDPA_API jgdpa_status jgdpa_cache_append(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                                          const int32_t* slots, int32_t total_new, void* k_cache, void* v_cache,
                                          int64_t k_page_stride, int64_t v_page_stride, int32_t num_pages,
                                          int32_t page_size, int32_t kv_heads, int32_t head_dim,
                                          jgdpa_stream_t stream);

/*
 * Attention from the new tokens over each request's pages.
 *   q            bf16 rows [heads][head_dim], q_stride elements apart (a
 *                multiple of 8); row q_offsets[b] + t is new token t of request
 *                b.  heads is a multiple of kv_heads; query head h reads
 *                key/value head h / (heads / kv_heads)
 *   max_q        an upper bound of every T_b, known to the host
 *   tree_mask    NULL: new token t sees new tokens u <= t.  Otherwise int32
 *                [total_q][mask_words]: bit u % 32 of word u / 32 of its row
 *                says whether it sees new token u of its request (itself
 *                included); T_b must be at most 32 mask_words
 *   depths       NULL or int32 [total_q], >= 0: new token t is at position (an int32)
 *                C + depths (C + t without), and context token j at j; the bias
 *                index is clamp(pos_i - pos_j, -R, R) + R and a window w > 0
 *                keeps pairs with |pos_i - pos_j| < w
 *   act, scale, bias_table, bias_len   as in jgdpa_fwd, bias_table [heads]
 *                [bias_len]; a softmax bias of -inf hides a key
 *   out          bf16 [total_q][heads][head_dim]
 *   lse          fp32 [heads][total_q] in SOFTMAX mode, or NULL; NULL otherwise
 * out and lse must not overlap the inputs.  Every token sees the whole context (within the window).  A token that sees
 * nothing gets O = 0 (LSE = -inf).  Infinities and NaN in the cache reach only
 * the rows that see their token; places of a page behind kv_lens[b] may hold
 * anything.  Same bits on every run, whatever else runs beside it.  Weights are
 * rounded to bf16 before the product with V; GELU and SiLU are right to bf16's
 * last place relative to themselves, far below zero, too.
 * Device-detected errors: BAD_OFFSETS (offsets not monotone from 0, beyond
 * total_q, T_b > max_q or more than the tree mask's columns, kv_lens[b] < T_b or
 * beyond the table), in which case nothing is written; BAD_OFFSETS also for a
 * depth that is negative or leads beyond position 2^31 - 1, and BAD_PAGE (a table
 * entry of a live token outside [0, num_pages)): no such page is read.  After
 * these two the outputs of the request concerned are unspecified, the others as
 * without it.
 */
JGDPA_API size_t jgdpa_cache_fwd_workspace_bytes(int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t max_q);
JGDPA_API jgdpa_status jgdpa_cache_fwd(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                                       int64_t k_page_stride, int64_t v_page_stride, int32_t num_pages,
                                       int32_t page_size, const int32_t* block_table, int32_t table_width,
                                       const int32_t* q_offsets, const int32_t* kv_lens, int32_t batch,
                                       int64_t total_q, int32_t max_q, int32_t heads, int32_t kv_heads,
                                       int32_t head_dim, jgdpa_act act, float scale, const float* bias_table,
                                       int32_t bias_len, int32_t window, const int32_t* tree_mask, int32_t mask_words,
                                       const int32_t* depths, void* out, float* lse,
                                       void* workspace, size_t workspace_bytes, jgdpa_stream_t stream);

/*
 * Norms of queries and keys for each head with the rotation by position, in one
 * pass: what stands in front of jgdpa_fwd (and, backward, behind jgdpa_bwd) where
 * a model has them.  Of every head's vector x of every row,
 *
 *     h = x w / sqrt(mean(x^2) + eps)         (norm = 1; norm = 0: h = x)
 *     (y_a, y_b) = (h_a cos t - h_b sin t, h_b cos t + h_a sin t),  t = pos * inv_freq[i]
 *
 * over the pairs (a, b) = (i, i + pairs), i < pairs (interleaved = 0), or (2 i,
 * 2 i + 1) (interleaved = 1); columns from 2 pairs on are not rotated.
 *   q, k       bf16 rows [heads][head_dim] ([kv_heads][head_dim]), q_stride /
 *              k_stride elements apart (multiples of 8, at least a row: they may be slices of a
 *              fused projection's output)
 *   q_out, k_out  the same with strides of their own; an output may be its
 *              input itself, and must not overlap anything else.  k (with k_out
 *              and its other arguments) may be NULL with total_kv = 0: queries alone
 *   q_offsets, kv_offsets  int32 [batch + 1] as in jgdpa_fwd: a row's position is its
 *              place in its segment.  Rows behind the last segment (a padded
 *              batch) are left as they were.  Not read, and may be NULL, where
 *   q_positions, k_positions  int32 [total_q], [total_kv] are given instead of NULL: a row's
 *              position, any int32
 *   q_weight, k_weight  fp32 [head_dim], the w of the norms, or NULL for 1 (norm = 0: NULL)
 *   inv_freq   fp32 [pairs], finite; 1 <= pairs <= head_dim / 2, and a multiple of 8
 *              unless interleaved.  The angle of any position is right to some 2^-22 of a turn
 *   eps        finite, >= 0; not used with norm = 0
 *   workspace  where a device-detected error is to be read from
 *              (jgdpa_norm_rotate_workspace_bytes(head_dim, 0) bytes), or NULL
 * Device-detected errors: BAD_OFFSETS (offsets not in order from 0, or beyond the rows); the
 * outputs are then unspecified.  fp32 throughout, one rounding at the end.  (So a head's sum of squares has to be
 * an fp32 number: heads with values of some 2^60 and more, or with eps = 0 of nothing but values below 2^-60, are
 * unspecified, gradients included.)
 *
 * Backward, from dq_out and dk_out (rows as q and k; strides of their own):
 *   dq, dk     the gradients of q and k; either may be its dq_out / dk_out, or its q / k
 *   dq_weight, dk_weight  fp32 [head_dim], sums over all rows and heads, in a fixed order
 *              (the same bits on every run); NULL where not wanted (norm = 0: NULL)
 * With norm = 0 q and k are not read and may be NULL (their strides are not looked at).  The workspace
 * (jgdpa_norm_rotate_workspace_bytes(head_dim, 1) bytes) holds the CTAs' sums
 * and is required where a weight's gradient is wanted.
 */
JGDPA_API size_t jgdpa_norm_rotate_workspace_bytes(int32_t head_dim, int32_t for_backward);
JGDPA_API jgdpa_status jgdpa_norm_rotate(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                                         int64_t total_q, int32_t heads, const int32_t* q_offsets,
                                         const int32_t* q_positions, const float* q_weight, const void* k,
                                         int64_t k_stride, void* k_out, int64_t k_out_stride, int64_t total_kv,
                                         int32_t kv_heads, const int32_t* kv_offsets, const int32_t* k_positions,
                                         const float* k_weight, int32_t batch, int32_t head_dim, const float* inv_freq,
                                         int32_t pairs, int32_t interleaved, int32_t norm, float eps, void* workspace,
                                         size_t workspace_bytes, jgdpa_stream_t stream);
JGDPA_API jgdpa_status jgdpa_norm_rotate_bwd(const void* dq_out, int64_t dq_out_stride, const void* q,
                                             int64_t q_stride, void* dq, int64_t dq_stride, int64_t total_q,
                                             int32_t heads, const int32_t* q_offsets, const int32_t* q_positions,
                                             const float* q_weight, float* dq_weight, const void* dk_out,
                                             int64_t dk_out_stride, const void* k, int64_t k_stride, void* dk,
                                             int64_t dk_stride, int64_t total_kv, int32_t kv_heads,
                                             const int32_t* kv_offsets, const int32_t* k_positions,
                                             const float* k_weight, float* dk_weight, int32_t batch, int32_t head_dim,
                                             const float* inv_freq, int32_t pairs, int32_t interleaved, int32_t norm,
                                             float eps, void* workspace, size_t workspace_bytes, jgdpa_stream_t stream);

/*
 * jgdpa_cache_append with the norms and the rotation of jgdpa_norm_rotate on the
 * way, and the new tokens' queries in the same launch: stands between
 * jgdpa_cache_plan and jgdpa_cache_fwd.
 *   q, q_out   bf16 rows [heads][head_dim] of the new tokens (q_out may be q); q
 *              may be NULL with heads = 0: the cache alone
 *   k_new, v_new, slots, k_cache, v_cache, ...  as in jgdpa_cache_append, the keys with norm
 *              and rotation, the values as they are (of rows with the same slot, parts of either may stay)
 *   q_offsets, kv_lens, depths  as in jgdpa_cache_fwd: new token t of request b is at
 *              position kv_lens[b] - T_b + t, or + depths[its row] where depths are given
 * Rows behind q_offsets[batch] are left out.  When an accepted row moves to another slot
 * (jgdpa_verify's keep_slots), the same call with the same q_offsets, kv_lens and depths writes it
 * there: a token's position does not depend on its slot.
 * Device-detected errors (workspace of jgdpa_norm_rotate_workspace_bytes(head_dim, 0) bytes, or NULL):
 * BAD_OFFSETS (offsets not in order from 0 or beyond total_new, kv_lens[b] < T_b, a depth
 * that is negative or leads beyond 2^31 - 1; the rows concerned are then unspecified).
 */
JGDPA_API jgdpa_status jgdpa_cache_append_rotated(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                                                  int32_t heads, const void* k_new, const void* v_new,
                                                  int64_t k_stride, int64_t v_stride, const int32_t* slots,
                                                  int32_t total_new, void* k_cache, void* v_cache,
                                                  int64_t k_page_stride, int64_t v_page_stride, int32_t num_pages,
                                                  int32_t page_size, int32_t kv_heads, int32_t head_dim,
                                                  const int32_t* q_offsets, const int32_t* kv_lens,
                                                  const int32_t* depths, int32_t batch, const float* q_weight,
                                                  const float* k_weight, const float* inv_freq, int32_t pairs,
                                                  int32_t interleaved, int32_t norm, float eps, void* workspace,
                                                  size_t workspace_bytes, jgdpa_stream_t stream);

/*
 * Verification of drafted tokens against the target's probabilities, from given
 * random numbers, and the next token.  Row 0 of a request is the token it ended with, every other
 * row a drafted one that continues an earlier row of the request, its parent.
 *   target       probabilities [total_q][vocab], fp32 or (target_bf16 = 1) bf16, rows target_stride
 *                elements apart: row r's are those of the token after row r
 *   draft        the probabilities that the drafted tokens were drawn from, row r's
 *                those of row r's own token (a request's row 0 is not read); NULL: drafts without
 *                probabilities.  With them parents must be NULL
 *   tokens       int32 [total_q]
 *   parents      int32 [total_q], the parent's row within the request (row 0's is not
 *                looked at); NULL: chains, each row continues the one before
 *   uniforms     fp32 [total_q] in [0, 1): row r's decides on its token, a
 *                request's row 0's draws the next token
 *   q_offsets    int32 [batch + 1]; at most 1024 rows per request
 * From the root (row 0) on the children of a row are tried in order: child c with token
 * x stays if u_c draft_c(x) < target_parent(x), or without draft probabilities if u_c (1 - g) <
 * target_parent(x), g the target_parent of the tokens refused there before (a token that
 * was refused there before does not stay).  The first that stays is gone on from.  Where none
 * does, the next token is drawn from max(target - draft, 0) of the row and its refused child (each difference in fp32), or
 * from target without the refused tokens, or from target where no row was refused (or nothing
 * is left): the least i whose sum of entries 0 .. i exceeds u times the sum of all.  Sums
 * are kept to some 2^-46.  Entries of target that are negative, infinite or NaN count as 0, in what stays and
 * in what is drawn, and so do such differences.  A token whose draft entry is NaN or +infinity does not stay.
 *   accepted     int32 [batch]: rows that stay, row 0 among them (0 of a request without rows)
 *   next_tokens  int32 [batch], -1 of a request without rows and where the whole row holds nothing
 *   places       int32 [total_q]: a row's place among those that stay (0: the
 *                root), or -1
 *   keep_lens    int32 [batch], or NULL: kv_lens[b] - T_b + accepted, the next plan's ctx_lens;
 *                needs kv_lens [batch]
 *   keep_slots   int32 [total_q], or NULL: where a row that stays has to move in the cache so that those
 *                that stay lie side by side, slots[q_offsets[b] + place]; -1 for rows that go or
 *                lie there already.  For jgdpa_cache_append, jgdpa_cache_append_rotated and
 *                jgdpa_cache4_append; needs slots [total_q], the plan's
 * Rows behind q_offsets[batch] get -1.  Outputs must not overlap inputs.  The same bits on every run.
 * Device-detected errors (workspace of jgdpa_verify_workspace_bytes() bytes, or NULL): BAD_OFFSETS (offsets not in order
 * from 0 or beyond total_q, more than 1024 rows: such a request counts as one without rows; a row that several
 * requests then claim holds -1 or what one of them makes of it;
 * parents that are no earlier row, tokens outside the vocabulary: such a row does not stay).
 */
JGDPA_API size_t jgdpa_verify_workspace_bytes(void);
JGDPA_API jgdpa_status jgdpa_verify(const void* target, int64_t target_stride, int32_t target_bf16, const void* draft,
                                    int64_t draft_stride, int32_t draft_bf16, const int32_t* tokens,
                                    const int32_t* parents, const float* uniforms, const int32_t* q_offsets,
                                    int32_t batch, int32_t total_q, int32_t vocab, const int32_t* kv_lens,
                                    const int32_t* slots, int32_t* accepted, int32_t* next_tokens, int32_t* places,
                                    int32_t* keep_lens, int32_t* keep_slots, void* workspace, size_t workspace_bytes,
                                    jgdpa_stream_t stream);

/*
 * The paged cache held in 4 bits: 0.27 of the bf16 cache's bytes at head_dim 128.  Pages, slots and
 * block tables are jgdpa_cache_plan's.  Of keys, and of values:
 *   codes        uint8 [kv_heads][page_size][head_dim / 2] a page, code_stride bytes apart (a multiple
 *                of 16, at least a page): columns 2 j and 2 j + 1 in the low and high bits of byte j
 *   scales       bf16 [kv_heads][page_size][2] a page, scale_stride elements apart (a multiple of 8,
 *                at least a page): step s and middle z of each token's head
 * A code c stands for z + s (c - 8).
 *
 * jgdpa_cache4_append writes rows as jgdpa_cache_append does (rows with slots outside the cache are
 * skipped; of rows with the same slot, parts of either may stay).  With lo and hi the least and largest of a head's values, each operation rounded to fp32,
 * halves to even:
 *     s = bf16((hi - lo) / 15), z = bf16(lo + 8 s), c = clamp(rint((x - z) / s), -8, 7) + 8 (8 where s is 0).
 * A head with a NaN or an infinity (or whose hi - lo leaves fp32) stands for NaN or infinities as a whole.
 *
 * jgdpa_cache4_read is the way back: rows slots[r] of the cache as bf16 rows (k_out and v_out, strides as
 * k_new's), for the packed calls (the cached part of a long prompt) or another cache.  Zeros for slots
 * outside the cache.
 */
JGDPA_API jgdpa_status jgdpa_cache4_append(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                                           const int32_t* slots, int32_t total_new, void* k_codes, void* k_scales,
                                           void* v_codes, void* v_scales, int64_t k_code_stride, int64_t k_scale_stride,
                                           int64_t v_code_stride, int64_t v_scale_stride, int32_t num_pages,
                                           int32_t page_size, int32_t kv_heads, int32_t head_dim,
                                           jgdpa_stream_t stream);
JGDPA_API jgdpa_status jgdpa_cache4_read(const void* k_codes, const void* k_scales, const void* v_codes,
                                         const void* v_scales, int64_t k_code_stride, int64_t k_scale_stride,
                                         int64_t v_code_stride, int64_t v_scale_stride, int32_t num_pages,
                                         int32_t page_size, int32_t kv_heads, int32_t head_dim, const int32_t* slots,
                                         int32_t rows, void* k_out, void* v_out, int64_t k_stride, int64_t v_stride,
                                         jgdpa_stream_t stream);

/*
 * jgdpa_cache_fwd over a cache held in 4 bits: its arguments, its computation from the values that the
 * codes stand for, which are not rounded again, and its errors.  Made for few rows (max_q heads / kv_heads up to
 * some 16: the keys are read again for every 16).  NaN and infinities of steps and middles reach
 * only the rows that see their token; a row of q with an infinity or a NaN is NaN or infinite itself.
 */
JGDPA_API size_t jgdpa_cache4_fwd_workspace_bytes(int32_t head_dim);
JGDPA_API jgdpa_status jgdpa_cache4_fwd(const void* q, int64_t q_stride, const void* k_codes, const void* k_scales,
                                        const void* v_codes, const void* v_scales, int64_t k_code_stride,
                                        int64_t k_scale_stride, int64_t v_code_stride, int64_t v_scale_stride,
                                        int32_t num_pages, int32_t page_size, const int32_t* block_table,
                                        int32_t table_width, const int32_t* q_offsets, const int32_t* kv_lens,
                                        int32_t batch, int64_t total_q, int32_t max_q, int32_t heads, int32_t kv_heads,
                                        int32_t head_dim, jgdpa_act act, float scale, const float* bias_table,
                                        int32_t bias_len, int32_t window, const int32_t* tree_mask, int32_t mask_words,
                                        const int32_t* depths, void* out, float* lse, void* workspace,
                                        size_t workspace_bytes, jgdpa_stream_t stream);

/*
 * Forward pass without a caller-provided workspace: the same computation and
 * arguments as jgdpa_fwd minus (workspace, workspace_bytes).  There is no
 * counterpart on the pages; this entry point exists for callers that cannot
 * allocate device memory at call time -- for example a plugin interface that
 * hands over only input and output buffers, or a process whose device memory
 * is already fully reserved by another allocator, so that a cudaMalloc would
 * fail or force a synchronising reclaim.  The caller still owns and passes
 * every input and output.
 *
 * Scratch comes from a fixed array of JGDPA_NOALLOC_SCRATCH_BYTES (4 MiB)
 * compiled into the library; every GPU that loads the library holds that
 * array until the process exits.  Sizes whose scratch would not fit (about
 * 87,000 to 130,000 units of (segment, head, pair of 128-row query tiles),
 * depending on the segment lengths) are rejected with
 * JGDPA_ERR_WORKSPACE_TOO_SMALL before anything is launched.
 *
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture.  The address is kept for the life of the
 * process, so a device reset (cudaDeviceReset) after the first call on that
 * device is not supported: later calls would launch on the old address.  No call allocates or frees memory.  All calls
 * on a device share the one array and it keeps the previous call's contents
 * (the parts that must start at zero are cleared on the stream by each call):
 * calls that overlap in time on the GPU -- on different streams, or from
 * different host threads -- race on it and must be serialised by the caller.
 * Device-detected errors (bad offsets) leave the outputs unwritten and are not
 * reported by this entry point; use jgdpa_fwd to read them back.
 */
#define JGDPA_NOALLOC_SCRATCH_BYTES (4u << 20)
JGDPA_API jgdpa_status jgdpa_fwd_noalloc(const void* q, const void* k, const void* v,
                       const int32_t* q_offsets, const int32_t* kv_offsets,
                       int32_t batch, int64_t total_q, int64_t total_kv,
                       int32_t heads, int32_t head_dim, jgdpa_act act, float scale,
                       const float* bias_table, int32_t bias_len, int32_t causal,
                       void* out, float* lse, jgdpa_stream_t stream);

/*
 * Reads the device status word of `workspace` (synchronises `stream`) and
 * returns JGDPA_OK, a device-detected error, or JGDPA_ERR_CUDA.
 */
JGDPA_API jgdpa_status jgdpa_read_device_status(const void* workspace, jgdpa_stream_t stream);

/* Static, human-readable name of a status code. */
JGDPA_API const char* jgdpa_status_string(jgdpa_status s);

/*
 * Test hook: evaluates the device's own activation functions, exactly as the
 * forward and backward kernels use them, on n fp32 inputs.  act is GELU or
 * SiLU; y[i] = act(x[i]) and dy[i] = act'(x[i]) (dy may be NULL).  `path`
 * selects the evaluation route: 0 = the special-function-unit route (hardware
 * tanh), 1 = the ALU-only polynomial route, 2 = the exponential route
 * (hardware ex2, reciprocal on the FMA pipe; forward only, so its dy is the
 * route-0 derivative).  x, y, dy are device pointers.
 */
JGDPA_API jgdpa_status jgdpa_eval_activation(jgdpa_act act, int32_t path, const float* x, int64_t n,
                                   float* y, float* dy, jgdpa_stream_t stream);

/*
 * Test hook: sets how long one internal device wait of the kernels may take
 * before it gives up, for every kernel launched after this call in this
 * process (any device, any stream); 0 restores the default of 2 s.  A wait
 * that gives up records JGDPA_ERR_DEVICE_TIMEOUT in the workspace status word;
 * the CTA then waits (at most 200 ms each) for its copies and tensor-core
 * operations in flight, releases its Tensor Memory and exits, and the later
 * kernels of the call do nothing.  A limit of a few nanoseconds makes the
 * waits of any multi-tile call run out, which is how the timeout path is
 * tested without faulting or hanging a GPU.  Not thread-safe with respect to
 * calls in flight on other host threads (they may see either value).
 */
JGDPA_API void jgdpa_set_wait_limit_ns(uint64_t limit_ns);

#ifdef __cplusplus
}
#endif

#endif /* JGDPA_H */

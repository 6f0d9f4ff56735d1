/*
 * misa.h -- C ABI of the MISA indexer library (libmisa.so, CUDA, sm_100a).
 *
 * The method is the one on "MISA: Mixture of Indexer Sparse Attention for Long-Context LLM
 * Inference" (gist.science/paper/2605.07363), "Technical Summary":
 *   - "Methodology: MISA", "Lightweight Block-Pooled Router": the prefix is cut into
 *     M = ceil(L/B) blocks of B keys, every block is summarised by the mean of its index keys,
 *     every indexer head gets one affinity aggregated over those pooled keys, and the h best of
 *     the H_I heads are routed;
 *   - "Methodology: MISA", "Sparse Token Scoring": only the routed heads score every prefix
 *     token and the top-k tokens by that reduced score are kept;
 *   - "Hierarchical Variant (MISA-dagger)": the routed pass keeps k' > k candidates that the
 *     dense indexer with all H_I heads re-scores, keeping the top-k;
 *   - "Problem Statement": the dense DSA indexer scores every prefix token with all H_I heads.
 * The pages do not write the formulas.  This library computes, for query t with prefix n_t:
 *   kbar_b  = mean of keys [bB, min((b+1)B, n_t))             (b < M_t = ceil(n_t/B))
 *   r_{t,j} = w_{t,j} * sum_{b < M_t} max(0, q_{t,j} . kbar_b)     (router score of head j)
 *   R_t     = the h heads with the largest r_{t,j}                 (ties to the lower head)
 *   I_{t,s} = sum_{j in R_t} w_{t,j} * max(0, q_{t,j} . k_s)       (s < n_t)
 *   F_{t,s} = sum_{j < H_I}  w_{t,j} * max(0, q_{t,j} . k_s)       (dense score)
 * No scale factor is applied.  Selections order by score descending; exact ties go to the lower
 * token index.  Scores are accumulated in fp32 (bf16 products are exact in fp32).
 *
 * Common conventions
 *   - Every pointer argument is device memory owned by the caller unless stated otherwise.
 *     Nothing is allocated inside the library; scratch comes from the caller's workspace
 *     (size from misa_workspace_bytes), which must be 256-byte aligned.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL is the legacy default stream).
 *     Arguments are validated on the host before any launch; on error nothing is launched.
 *   - Layouts are dense row-major.  q is [T, H_I, d], w is [T, H_I] (fp32), n is [T] (int32).
 *     The key cache of query t starts at k + t * k_seq_stride elements: k_seq_stride = 0 makes
 *     all queries share one cache (prefill), k_seq_stride = L*d gives one cache per query
 *     (batched decode).  Each cache holds L keys of d elements.
 *   - dtype is the element type of q and k (MISA_BF16 or MISA_F32).  d must be 128.
 *     H_I must be a multiple of 8 in [8, 128]; 1 <= h <= H_I.
 *   - Prefix lengths n_t are read on the device: values above L count as L, values below 1 give
 *     an empty prefix (no tokens selected; all router scores 0).
 *   - Index outputs hold min(topk, n_t) token indices followed by -1 padding.  The selected set
 *     is what the method defines (and identical from run to run); the order of the indices
 *     inside a row is not specified.
 *   - Errors: MISA_ERR_INVALID_ARG (null pointer, size out of range), MISA_ERR_UNSUPPORTED
 *     (d != 128, H_I not a multiple of 8, dtype, k' too large), MISA_ERR_WORKSPACE (workspace
 *     too small or misaligned), MISA_ERR_CUDA (a launch failed; cudaGetLastError's code is
 *     consumed).  Errors that arise on the device after a launch are reported by
 *     misa_device_check.
 */
#ifndef MISA_H_
#define MISA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MISA_OK = 0,
  MISA_ERR_INVALID_ARG = 1,
  MISA_ERR_UNSUPPORTED = 2,
  MISA_ERR_WORKSPACE = 3,
  MISA_ERR_CUDA = 4,
  MISA_ERR_DEVICE_TIMEOUT = 5,
  MISA_ERR_BAD_INDEX = 6
} misa_status;

typedef enum { MISA_BF16 = 0, MISA_F32 = 1 } misa_dtype;

/* Operation codes for misa_workspace_bytes. */
typedef enum {
  MISA_OP_ROUTE = 0,
  MISA_OP_SCORE_TOPK = 1,
  MISA_OP_RERANK = 2,
  MISA_OP_DENSE_TOPK = 3,
  MISA_OP_TOPK_SELECT = 4,
  MISA_OP_BLOCK_FILTER = 5,
  MISA_OP_ROUTE_PAGED = 6,
  MISA_OP_SCORE_TOPK_PAGED = 7,
  MISA_OP_RERANK_PAGED = 8,
  MISA_OP_SCORE_TOPK_FUSED = 9,
  MISA_OP_HIER_FUSED = 10,
  MISA_OP_KV4_ATTENTION = 11,
  MISA_OP_KV4_COMPACT = 12,
  MISA_OP_KEYS_COMPACT_PAGED = 13,
  MISA_OP_PROMPT_ATTENTION = 14
} misa_op;

/* Largest k' accepted by misa_hier_rerank (its candidates are ranked in shared memory). */
#define MISA_MAX_KP 16384

/* Library version, major*10000 + minor*100 + patch. */
int misa_version(void);

/* Static text for a status code. */
const char* misa_status_str(int status);

/*
 * Workspace bytes needed by one call of `op` with these sizes (0 if it needs none).
 * Arguments an op does not use are ignored.  Sizes <= 0 give 0.  For MISA_OP_BLOCK_FILTER the
 * last argument carries m, the number of kept blocks (0 when m * B exceeds MISA_MAX_KP).  The calls
 * on 4-bit caches, compactions and prompt attention name what they put into these arguments themselves;
 * sizes that they refuse give 0.
 */
size_t misa_workspace_bytes(int op, int T, int L, int H_I, int B, int h, int topk, int kp);

/*
 * Block mean-pool of key caches ("Lightweight Block-Pooled Router": mean-pooled indexing keys
 * over M = ceil(L/B) blocks).
 *   k      : n_seq caches of L keys [L, d] at stride k_seq_stride elements (dtype)
 *   kbar   : out, fp32, n_seq x [ceil(L/B), d] at stride kbar_seq_stride floats
 *   blocks [block_begin, block_end) of every cache are written (clamped to [0, ceil(L/B)));
 *   block b averages keys [bB, min((b+1)B, L)) (a partial last block over its valid keys).
 * The router and the block filter average the last block of every prefix from the keys
 * themselves, so a decode loop calls this with [b, b+1) once its prefix has moved past block b
 * (once every B steps), not for the block that holds the newest key.
 */
misa_status misa_pool_keys(const void* k, int64_t k_seq_stride, int n_seq, int L, int d, int B,
                           int dtype, float* kbar, int64_t kbar_seq_stride, int block_begin,
                           int block_end, void* stream);

/*
 * Block-pooled router and top-h head selection ("Lightweight Block-Pooled Router").
 *   kbar   : fp32 block means from misa_pool_keys; query t reads kbar + t*kbar_seq_stride
 *            (0 = shared).  Only blocks b < M_t - 1 are read from it; the last block of a prefix,
 *            keys [(M_t - 1) B, n_t) (full or partial), is averaged from k directly, so it may
 *            hold the newest keys without being pooled.
 *   heads  : out [T, h] int32, routed heads in descending router score (ties: lower head)
 *   r_opt  : out [T, H_I] fp32 router scores, or NULL
 *   ws     : workspace of misa_workspace_bytes(MISA_OP_ROUTE, T, L, H_I, B, h, 0, 0) bytes
 */
misa_status misa_route(const void* q, const float* w, const void* k, int64_t k_seq_stride,
                       const float* kbar, int64_t kbar_seq_stride, const int32_t* n, int T, int L,
                       int H_I, int d, int B, int h, int dtype, int32_t* heads, float* r_opt,
                       void* ws, size_t ws_bytes, void* stream);

/*
 * Routed-head token scores ("Sparse Token Scoring"): scores[t, s] = I_{t,s} for s < n_t.
 *   heads    : [T, h] routed heads (any order; NULL = all H_I heads, i.e. the dense score F)
 *   scores   : out fp32 [T, ld_scores], ld_scores >= L; entries s >= n_t are not written.
 *   select_ws, select_ws_bytes, select_topk : optional (NULL, 0, 0).  A workspace of
 *              misa_workspace_bytes(MISA_OP_TOPK_SELECT, T, L, ...) bytes in which the call also
 *              prepares a top-select_topk selection of these scores; pass the same workspace to
 *              misa_topk_select with ws_prepared = 1.  For fewer than 256 rows longer than
 *              16384 entries it builds a candidate list per query right after the scores: one
 *              CTA per row places the row's cut from a sample of its scores (256 evenly spaced
 *              runs of 8; the rank of the expected count above the select_topk-th score plus
 *              three standard deviations), then CTAs over chunks of 8192 scores append every
 *              score at or above it.  The selection ranks those entries and takes an exact pass
 *              over the score row whenever they cannot hold the answer (fewer than select_topk,
 *              or the list overflowed), so the result never depends on where the cut fell.
 *              Shorter rows, many rows and rows whose lists would not fit get no list and are
 *              selected from the scores.
 */
misa_status misa_token_scores(const void* q, const float* w, const void* k, int64_t k_seq_stride,
                              const int32_t* n, const int32_t* heads, int T, int L, int H_I, int d,
                              int h, int dtype, float* scores, int64_t ld_scores, int select_topk,
                              void* select_ws, size_t select_ws_bytes, void* stream);

/*
 * Top-k selection over per-query score rows ("Sparse Token Scoring": the final top-k tokens
 * are selected on the reduced scores).  scores [T, ld_scores] fp32, entries s < n_t are read.
 *   idx         : out [T, topk] int32, -1 padded
 *   score_opt   : out [T, topk] fp32 score of each selected token (0 for padding), or NULL
 *   ws          : misa_workspace_bytes(MISA_OP_TOPK_SELECT, T, L, ...) bytes
 *   ws_prepared : 1 if misa_token_scores already prepared ws for these scores and this topk
 * Scores must be finite.  Without ws_prepared the call first builds the candidate lists of long
 * rows itself (as misa_token_scores does); then one CTA per row selects, from its list or, for rows
 * without one, from a sampled cut and a pass over the row.  Both give the same set.
 */
misa_status misa_topk_select(const float* scores, int64_t ld_scores, const int32_t* n, int T,
                             int L, int topk, int32_t* idx, float* score_opt, void* ws,
                             size_t ws_bytes, int ws_prepared, void* stream);

/*
 * Routed scoring followed by top-k: misa_token_scores (preparing the selection) then
 * misa_topk_select.  With topk = k' this is the coarse stage of MISA-dagger ("Hierarchical
 * Variant": enlarged candidate set).
 *   scores_full_opt : [T, L] fp32 buffer that receives every score, or NULL (scores then live in
 *                     the workspace)
 *   ws : misa_workspace_bytes(MISA_OP_SCORE_TOPK, T, L, ...) bytes (with scores_full_opt given,
 *        misa_workspace_bytes(MISA_OP_TOPK_SELECT, T, L, ...) bytes suffice)
 */
misa_status misa_score_topk(const void* q, const float* w, const void* k, int64_t k_seq_stride,
                            const int32_t* n, const int32_t* heads, int T, int L, int H_I, int d,
                            int h, int topk, int dtype, int32_t* idx, float* score_opt,
                            float* scores_full_opt, void* ws, size_t ws_bytes, void* stream);

/*
 * MISA-dagger fine stage ("Hierarchical Variant (MISA-dagger)": the dense indexer with all H_I
 * heads re-scores only the k' candidates and keeps the final top-k).
 *   cand      : [T, kp] candidate token indices; entries < 0 or >= n_t are empty slots
 *   idx       : out [T, topk] the kept candidates, -1 padded
 *   score_opt : out [T, topk] their dense scores, or NULL
 *   ws        : misa_workspace_bytes(MISA_OP_RERANK, T, 0, H_I, 0, 0, topk, kp) bytes
 * Requires topk <= kp <= MISA_MAX_KP; duplicate candidates are the caller's error.
 */
misa_status misa_hier_rerank(const void* q, const float* w, const void* k, int64_t k_seq_stride,
                             const int32_t* n, const int32_t* cand, int T, int L, int H_I, int d,
                             int kp, int topk, int dtype, int32_t* idx, float* score_opt, void* ws,
                             size_t ws_bytes, void* stream);

/*
 * Dense DSA indexer ("Problem Statement": every prefix token scored with all H_I heads, top-k
 * kept): top-k of F_{t,s} over s < n_t.  Outputs as misa_score_topk.
 *   ws : misa_workspace_bytes(MISA_OP_DENSE_TOPK, T, L, ...) bytes
 */
misa_status dsa_dense_topk(const void* q, const float* w, const void* k, int64_t k_seq_stride,
                           const int32_t* n, int T, int L, int H_I, int d, int topk, int dtype,
                           int32_t* idx, float* score_opt, void* ws, size_t ws_bytes,
                           void* stream);

/*
 * Token-axis block filter composed with MISA ("HISA: Efficient Hierarchical Indexing for
 * Fine-Grained Sparse Attention", arXiv 2603.28458, abstract: a coarse stage scores pooled block
 * representatives and keeps candidate blocks, then the indexer scores only their tokens; "MISA",
 * "Problem Statement" and "Significance and Claims": token-axis and head-axis savings combine).
 * For query t with routed heads R_t (heads[t], from misa_route):
 *   S_{t,b} = sum_{j in R_t} w_{t,j} * max(0, q_{t,j} . kbar_b)     (b < M_t = ceil(n_t/B))
 * with kbar_b the router's block means (the last block, full or partial, averaged from k); the m
 * blocks with the largest S_{t,b} are kept (ties: lower block); their prefix tokens are scored
 * with I_{t,s} and the top-k of those is selected (ties: lower token).  m >= M_t gives exactly
 * misa_score_topk's selection; h = H_I gives the block filter on the dense indexer.
 *   kbar             : fp32 block means from misa_pool_keys, 16-byte aligned; query t reads
 *                      kbar + t*kbar_seq_stride (0 = shared; else a multiple of 4, >= M*d);
 *                      blocks b < M_t - 1 only, as misa_route
 *   heads            : [T, h] routed heads in [0, H_I) (other ids are never dereferenced, but
 *                      the results are then unspecified)
 *   m                : blocks kept per query, 1 <= m with m * B <= MISA_MAX_KP
 *   block_scores_opt : out [T, ld_block_scores] fp32 S_{t,b} for b < M_t (ld >= ceil(L/B)), or NULL
 *   blocks           : out [T, m] kept blocks, -1 padded (order unspecified)
 *   idx, score_opt   : out [T, topk] selected tokens (-1 padded when the kept blocks hold fewer
 *                      than topk prefix tokens) and their scores I, or NULL for score_opt
 *   ws               : misa_workspace_bytes(MISA_OP_BLOCK_FILTER, T, L, H_I, B, h, topk, m) bytes
 * Errors as above; m * B > MISA_MAX_KP gives MISA_ERR_UNSUPPORTED.
 */
misa_status misa_block_filter_topk(const void* q, const float* w, const void* k,
                                   int64_t k_seq_stride, const float* kbar,
                                   int64_t kbar_seq_stride, const int32_t* n,
                                   const int32_t* heads, int T, int L, int H_I, int d, int B, int h,
                                   int m, int topk, int dtype, float* block_scores_opt,
                                   int64_t ld_block_scores, int32_t* blocks, int32_t* idx,
                                   float* score_opt, void* ws, size_t ws_bytes, void* stream);

/*
 * Paged key caches.  Serving stores each sequence's keys in fixed-size pages of one pool shared by
 * all sequences (the pages call MISA a drop-in replacement for the DSA indexer, "Key
 * Contributions"; this is the layout such a replacement reads).  The *_paged calls compute exactly
 * what their contiguous counterparts compute on each sequence's logical cache:
 *   pool       : [num_pages, page_size, d] keys (dtype); num_pages * page_size < 2^31
 *   page_table : [T, max_pages] int32; logical key s of query t's sequence is row s % page_size of
 *                physical page page_table[t][s / page_size].  Entries for pages past a prefix are
 *                never read.  max_pages * page_size >= L (L: the longest prefix, as elsewhere).
 *   n          : [T] prefix lengths, as elsewhere.
 * A page id outside [0, num_pages) inside a prefix is never dereferenced: its keys read as zero
 * (pooling, router) or the token is left out of scoring; results are then unspecified.
 * kbar is one pooled cache per query ([T, ceil(L/B), d] at kbar_seq_stride >= ceil(L/B) * d), as
 * written by misa_pool_keys_paged.  Queries that share a sequence repeat its table row.
 */
/* misa_pool_keys through page tables (page_table rows are the n_seq sequences). */
misa_status misa_pool_keys_paged(const void* pool, int64_t num_pages, int page_size,
                                 const int32_t* page_table, int64_t max_pages, int n_seq, int L,
                                 int d, int B, int dtype, float* kbar, int64_t kbar_seq_stride,
                                 int block_begin, int block_end, void* stream);

/* misa_route on paged caches.
 *   ws : misa_workspace_bytes(MISA_OP_ROUTE_PAGED, T, L, H_I, B, h, 0, 0) bytes */
misa_status misa_route_paged(const void* q, const float* w, const void* pool, int64_t num_pages,
                             int page_size, const int32_t* page_table, int64_t max_pages,
                             const float* kbar, int64_t kbar_seq_stride, const int32_t* n, int T,
                             int L, int H_I, int d, int B, int h, int dtype, int32_t* heads,
                             float* r_opt, void* ws, size_t ws_bytes, void* stream);

/* misa_score_topk on paged caches (with topk = k', the MISA-dagger coarse stage).
 *   ws : misa_workspace_bytes(MISA_OP_SCORE_TOPK_PAGED, T, L, H_I, 0, h, topk, 0) bytes */
misa_status misa_score_topk_paged(const void* q, const float* w, const void* pool, int64_t num_pages,
                                  int page_size, const int32_t* page_table, int64_t max_pages,
                                  const int32_t* n, const int32_t* heads, int T, int L, int H_I,
                                  int d, int h, int topk, int dtype, int32_t* idx, float* score_opt,
                                  void* ws, size_t ws_bytes, void* stream);

/* misa_hier_rerank on paged caches.
 *   ws : misa_workspace_bytes(MISA_OP_RERANK_PAGED, T, 0, H_I, 0, 0, topk, kp) bytes */
misa_status misa_hier_rerank_paged(const void* q, const float* w, const void* pool, int64_t num_pages,
                                   int page_size, const int32_t* page_table, int64_t max_pages,
                                   const int32_t* n, const int32_t* cand, int T, int L, int H_I,
                                   int d, int kp, int topk, int dtype, int32_t* idx,
                                   float* score_opt, void* ws, size_t ws_bytes, void* stream);

/*
 * misa_score_topk for queries that share one bf16 key cache (chunked prefill), without writing
 * score rows ("Sparse Token Scoring": the top-k tokens by the routed score).  The tensor-core
 * scorer first scores every 32nd tile of 128 keys of each prefix; each query's cut is placed on that
 * sample (the expected number of sampled scores above the k-th, plus three standard deviations and
 * a margin); a second pass over every key appends only the scores at or above the cut to a list of
 * 4k entries per query, from which the top-k is selected.  A query whose list holds fewer than
 * min(k, n_t) entries or overflowed is redone exactly on the device by the unfused scorer and
 * selection, so the selected set is always misa_score_topk's.
 *   k  : one shared cache [L, d] (k_seq_stride 0), bf16 like q
 *   ws : misa_workspace_bytes(MISA_OP_SCORE_TOPK_FUSED, T, L, H_I, 0, h, topk, 0) bytes (it also
 *        holds score rows for the queries that are redone)
 * Requires 4 * topk <= 16384 (else MISA_ERR_UNSUPPORTED); other arguments and outputs as
 * misa_score_topk.
 */
misa_status misa_score_topk_fused(const void* q, const float* w, const void* k, const int32_t* n,
                                  const int32_t* heads, int T, int L, int H_I, int d, int h,
                                  int topk, int dtype, int32_t* idx, float* score_opt, void* ws,
                                  size_t ws_bytes, void* stream);

/*
 * MISA-dagger for decode batches with one key cache per query, without gathering the candidates
 * ("Hierarchical Variant (MISA-dagger)": the top-k' tokens by the routed score are re-scored with
 * all H_I heads and the top-k of that dense score is kept).  The result is misa_score_topk with
 * topk = k' followed by misa_hier_rerank on its candidates, up to the rounding of the dense scores
 * (a different summation on the tensor cores: near-ties at the k-th dense score may be ordered
 * differently).  For fewer than 256 queries longer than 16384 keys and h <= 8, the list cut's sample
 * of each prefix (256 evenly spaced runs of 8 keys) is scored first, each query's cut is placed on
 * it (the expected number of sampled scores above the k'-th, plus three standard deviations and a
 * margin), and one pass over the keys writes every routed score and keeps each token at or above
 * the cut with its dense score, computed from the key row the pass already holds; the top-k' of
 * those by the routed score and the top-k of them by the dense score are then selected.  A query
 * whose kept tokens are fewer than k' or overflow 16384 is answered exactly from its score row on
 * the device (the dense scores of its k' candidates computed there), so the selected set never
 * depends on the sample.  Other shapes take that exact way for every query.
 *   k         : per-query caches [T, L, d] (k_seq_stride >= L * d), bf16 like q
 *   heads     : [T, h] routed heads (misa_route)
 *   idx       : out [T, topk] the kept tokens (order not specified), -1 padded when n_t < topk
 *   score_opt : out [T, topk] their dense scores, or NULL
 *   ws        : misa_workspace_bytes(MISA_OP_HIER_FUSED, T, L, H_I, 0, h, topk, kp) bytes
 * Requires topk <= kp <= MISA_MAX_KP (else MISA_ERR_INVALID_ARG / MISA_ERR_UNSUPPORTED); a shared
 * cache (k_seq_stride 0) or fp32 inputs give MISA_ERR_UNSUPPORTED.
 */
misa_status misa_hier_topk_fused(const void* q, const float* w, const void* k, int64_t k_seq_stride,
                                 const int32_t* n, const int32_t* heads, int T, int L, int H_I, int d,
                                 int h, int kp, int topk, int dtype, int32_t* idx, float* score_opt,
                                 void* ws, size_t ws_bytes, void* stream);

/*
 * Attention beside the indexer.
 *
 * The indexer selects tokens; these calls fill the caches its tokens live in, attend over them, and
 * thin them out.  They serve d = 64 or 128 with H_q query heads over H_kv key and value heads (H_q a
 * multiple of H_kv; query head h reads kv head h / (H_q / H_kv)).  Softmax is taken in fp32;
 * lse is its natural log-sum, minus infinity for a row that attends to nothing, whose output is zero.
 *
 * Packed rows.  cu [S + 1] and, where a cache is involved, start [S] (int32, on the device) say which
 * rows of a packed tensor belong to which sequence: row r of sequence b, cu[b] <= r < cu[b + 1], is
 * its logical position start[b] + r - cu[b].  cu must not decrease and cu[0] >= 0; a sequence may be
 * empty.  Rows outside [cu[0], cu[S]) are not written, and nothing depends on what they hold.
 *
 * Caches in 4 bits.  Every 16 elements of a row share a scale; an element is one of the 16 e2m1 values
 * (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign) times it:
 *   s_b = e4m3(max |x_i| / (6 g)),  code_i = e2m1(x_i / (s_b g)),  and x_i reads as code_i s_b g
 * over the 16 elements i of block b, both conversions to nearest with ties to even, the divisions and
 * 6 g in fp32; g is k_scale or v_scale, one fp32 number in [2^-60, 2^60] per tensor (1 suits blocks whose
 * largest element lies between about 0.1 and 2688; larger elements saturate, NaN stores as 0, infinite
 * elements as the largest value).  A block whose scale rounds to 0 stores zeros.
 *   pool       : uint8 [num_pages][H_kv][2][page_size * 9 d / 16], 16-byte aligned; the slab of one
 *                page, kv head and side (0 keys, 1 values) holds page_size code rows of d/2 bytes and
 *                behind them page_size scale rows of d/16 e4m3 bytes, 0 to 0x7e (other scale bytes are none of
 *                the format's; what attended rows with them give is not said).  Byte (d/8) c + 2 j + i of a
 *                code row holds elements 16 j + 4 c + 2 i (low nibble) and the next (c < 4, j < d/16, i < 2).
 *   page_size  : a multiple of 16, at most 1024 (else MISA_ERR_UNSUPPORTED)
 *   page_table : [S or T][max_pages] int32, as for the paged key caches; the same tables can serve
 *                both.  Ids outside [0, num_pages) are never dereferenced: rows are not written, read
 *                as zero, and left out of the attention.
 */

/*
 * Writes rows of k and v [rows][H_kv][d] (dtype; row strides ldk, ldv elements, multiples of 16 bytes;
 * 16-byte aligned) into the cache at their logical positions.  Two rows of one call must not have the
 * same place.  Positions that the page table does not reach are skipped.
 */
misa_status misa_kv4_append(const void* k, const void* v, int64_t ldk, int64_t ldv, int dtype, float k_scale,
                            float v_scale, void* pool, int64_t num_pages, int page_size, const int32_t* page_table,
                            int64_t max_pages, const int32_t* cu, const int32_t* start, int S, int rows, int H_kv,
                            int d, void* stream);

/*
 * Reads rows of the cache back into k and v [rows][H_kv][d] (dtype, 16-byte aligned; for a chunk of a
 * prompt that attends to what the cache already holds).  bf16 holds code_i s_b exactly.
 */
misa_status misa_kv4_read(const void* pool, int64_t num_pages, int page_size, const int32_t* page_table,
                          int64_t max_pages, const int32_t* cu, const int32_t* start, int S, int rows, int H_kv, int d,
                          int dtype, float k_scale, float v_scale, void* k, void* v, void* stream);

/*
 * Attention of one query token per sequence over its 4-bit cache:
 *   out[t, h] = sum_i softmax_i(scale q[t, h] . k_i) v_i   over i < n_t, or over i in idx[t].
 *   q, out     : [T][H_q][d], dtype; 16-byte aligned.  bf16 queries enter the products as they are; fp32 ones, and
 *                their softmax weights, as two fp16 parts (22 bits); sums are fp32
 *   idx        : [T][P] tokens to attend to, in any order (misa_score_topk and the other selections
 *                write such lists), or NULL for the whole prefix.  Entries < 0 or >= n_t are empty slots;
 *                a token named twice counts twice.
 *   lse_opt    : out [T][H_q] fp32, or NULL
 *   acc_opt    : [T][ld_acc] fp32, or NULL: acc[t][i] += sum over the H_q heads of token i's softmax
 *                weight (ld_acc >= L; other entries are not touched)
 *   ws         : misa_workspace_bytes(MISA_OP_KV4_ATTENTION, T, L, H_q, H_kv, d, P or 0, 1 with acc_opt
 *                else 0) bytes; with acc_opt it holds the logits, 4 H_q bytes per query and token, of as many
 *                queries at a time as 1 GiB holds (one at least)
 */
misa_status misa_kv4_attention(const void* q, const void* pool, int64_t num_pages, int page_size,
                               const int32_t* page_table, int64_t max_pages, const int32_t* n, const int32_t* idx,
                               int T, int L, int P, int H_q, int H_kv, int d, int dtype, float scale, float k_scale,
                               float v_scale, void* out, float* lse_opt, float* acc_opt, int64_t ld_acc, void* ws,
                               size_t ws_bytes, void* stream);

/*
 * misa_kv4_attention with an acc that has columns for the first acc_cols tokens only (1 <= acc_cols <= ld_acc;
 * acc_cols need not reach L).  Later tokens are attended to alike; their weights are not kept.
 */
misa_status misa_kv4_attention_cols(const void* q, const void* pool, int64_t num_pages, int page_size,
                                    const int32_t* page_table, int64_t max_pages, const int32_t* n, const int32_t* idx,
                                    int T, int L, int P, int H_q, int H_kv, int d, int dtype, float scale,
                                    float k_scale, float v_scale, void* out, float* lse_opt, float* acc_opt,
                                    int acc_cols, int64_t ld_acc, void* ws, size_t ws_bytes, void* stream);

/*
 * Which tokens stay when caches are thinned to `keep` tokens by the attention weight they have gathered
 * (acc of misa_kv4_attention).  Prefixes of at most keep tokens stay whole; of a longer one stay the
 * first `sink`, the last `recent` (sink + recent <= keep), and of those between the ones with the
 * largest acc (ties: lower token; NaN counts as the smallest).
 *   acc         : [T][ld_acc] fp32, entries i < n_t are read (ld_acc >= L)
 *   idx         : out [T][keep] the tokens that stay, ascending, -1 behind the last
 *   n_out       : out [T] min(n_t, keep); may be n itself (lengths updated in place), not overlap it otherwise
 *   acc_out_opt : out [T][ld_out] (ld_out >= keep): acc of the tokens that stay, in the order of idx,
 *                 then zeros to the end of the row; must not overlap acc.  Or NULL.
 */
misa_status misa_evict_select(const float* acc, int64_t ld_acc, const int32_t* n, int T, int L, int keep, int sink,
                              int recent, int32_t* idx, int32_t* n_out, float* acc_out_opt, int64_t ld_out,
                              void* stream);

/*
 * Closes up caches after misa_evict_select, in place: row idx[t][j] of sequence t moves to row j, for
 * the 4-bit cache or the indexer's paged keys (pool [num_pages][page_size][128] of dtype).  idx ascends
 * strictly, with -1 behind the last, as misa_evict_select writes it; keep is at most what the tables reach
 * (max_pages * page_size).  Rows from the number kept on keep their contents; block means of the keys are
 * pooled again with misa_pool_keys_paged.  The pages of the T sequences must be theirs alone.
 *   ws : misa_workspace_bytes(MISA_OP_KV4_COMPACT, T, 0, H_kv, 0, d, keep, 0), and
 *        misa_workspace_bytes(MISA_OP_KEYS_COMPACT_PAGED, T, 0, 0, 0, bytes of a key row, keep, 0) bytes
 *        (marks of which rows have been read, and counters of who reads which; cleared by the call)
 */
misa_status misa_kv4_compact(void* pool, int64_t num_pages, int page_size, const int32_t* page_table,
                             int64_t max_pages, const int32_t* idx, int T, int keep, int H_kv, int d, void* ws,
                             size_t ws_bytes, void* stream);
misa_status misa_keys_compact_paged(void* pool, int64_t num_pages, int page_size, const int32_t* page_table,
                                    int64_t max_pages, const int32_t* idx, int T, int keep, int d, int dtype, void* ws,
                                    size_t ws_bytes, void* stream);

/*
 * Causal attention of packed prompts.  Sequence b has queries cu_q[b] .. cu_q[b + 1] of q and keys
 * cu_k[b] .. cu_k[b + 1] of k and v, its queries being its last tokens: query i of it sees its keys
 * j <= i + (keys - queries).  With cu_k = cu_q that is a whole prompt; with more keys it is a chunk that
 * ends a longer one; queries before the first key see nothing.
 *   q      : [Tq][H_q][d] at row stride ldq elements; k, v : [Tk][H_kv][d] at ldk, ldv (multiples of 8
 *            elements, so the views of one fused projection serve; 16-byte aligned); bf16 only
 *   out    : [Tq][H_q][d] bf16;  lse_opt : [Tq][H_q] fp32, or NULL
 * Rows of other sequences never reach a sequence's outputs, whatever they hold, nor do keys and values
 * behind a query reach its own.
 *   ws     : misa_workspace_bytes(MISA_OP_PROMPT_ATTENTION, Tq, Tk, H_q, S, d, 0, 0) bytes (0 for a call of
 *            few short or many long prompts; otherwise mostly the pieces of what is cut between CTAs, 40 MB
 *            at d = 128)
 */
misa_status misa_prompt_attention(const void* q, const void* k, const void* v, int64_t ldq, int64_t ldk, int64_t ldv,
                                  const int32_t* cu_q, const int32_t* cu_k, int S, int Tq, int Tk, int H_q, int H_kv,
                                  int d, int dtype, float scale, void* out, float* lse_opt, void* ws, size_t ws_bytes,
                                  void* stream);

/*
 * Device-side status of the calls made so far on the current device.  The tensor-core kernels
 * (scoring and routing queries that share one bf16 cache, the re-rank of gathered candidates, and
 * prompt attention) pipeline their copies and MMAs through shared-memory barriers, and the calls that
 * close up caches wait for rows to be read before they write over them; every such wait is bounded
 * (about one second).  A wait that runs
 * out makes the kernel stop early, leaving its outputs incomplete, and records the event in a
 * per-device status word.  This call waits for all work on the device to finish
 * (cudaDeviceSynchronize), then reads and clears that word (and, in the bounds-checked build,
 * the counts of skipped out-of-range ids described below).
 *   returns MISA_OK, MISA_ERR_DEVICE_TIMEOUT (some call since the last check stopped early),
 *   MISA_ERR_BAD_INDEX (bounds-checked build: out-of-range ids were seen and skipped), or
 *   MISA_ERR_CUDA (the synchronisation or the read failed).
 */
misa_status misa_device_check(void);

/*
 * Bounds-checked build.  libmisa_checked.so (python -m long_context_sparse_mean_b200.build
 * --checked) is the same library compiled with MISA_CHECKED: every id that a kernel skips because
 * it lies outside its range is also counted on the device, by kind:
 *   out[0] routed head ids outside [0, H_I)            (scoring and block-filter calls)
 *   out[1] candidate token ids outside [0, n_t), other than the empty marker -1 (re-rank calls,
 *          paged or not, and attention over selected tokens; the header's "empty slot" rule still
 *          applies: they are skipped)
 *   out[2] page-table entries inside a prefix outside [0, num_pages) (paged calls; per key row
 *          read through the entry, in attention over a whole prefix per 16 of them)
 * The counts are occurrences seen, not distinct ids.  In both builds such ids are never
 * dereferenced.  misa_device_check returns MISA_ERR_BAD_INDEX (after MISA_ERR_DEVICE_TIMEOUT,
 * which takes precedence) when any count is nonzero, and clears them.
 */
/* 1 for the bounds-checked build, 0 otherwise. */
int misa_checked_build(void);

/*
 * Waits for the device (cudaDeviceSynchronize), then writes the counts of skipped out-of-range
 * ids since the last read into out[3] (kinds as above; zeros in the normal build) and clears them.
 * Returns MISA_OK, MISA_ERR_INVALID_ARG (out is NULL) or MISA_ERR_CUDA.
 */
misa_status misa_bad_index_counts(unsigned int* out);

/*
 * Capacity, in floats, of the fixed scratch array used by misa_hier_rerank_static
 * (4 MiB per GPU that loads the library, held until the process exits).
 */
#define MISA_STATIC_RERANK_SCRATCH_FLOATS (1 << 20)

/*
 * misa_hier_rerank without a workspace argument, for callers that cannot allocate device
 * memory.  The pages have no counterpart to this call; it exists for the deployment side only.
 * Who needs it: a plugin that its host framework hands only input and output buffers (the
 * framework owns the device memory and offers the plugin no allocator), or a latency-critical
 * decode loop that must not risk an allocation failure, or the device synchronisation that
 * cudaMalloc / cudaFree can cause, in the middle of a step.
 * Same arguments, results and checks as misa_hier_rerank, minus ws and ws_bytes.  Its T * kp
 * floats of scratch live in one array compiled into the library (MISA_STATIC_RERANK_SCRATCH_FLOATS
 * floats per device); the call allocates nothing.
 *   - T * kp above MISA_STATIC_RERANK_SCRATCH_FLOATS: returns MISA_ERR_WORKSPACE, nothing launched.
 *   - All calls on a device share the array and it keeps the last call's contents; nothing in it
 *     needs to start at zero.  Calls that overlap on the GPU (unordered streams) race on it and
 *     give undefined results: order them on one stream or with events.
 *   - The first call on a device looks up the array's device address with that device current
 *     (cudaGetSymbolAddress); make that first call before any stream capture.
 */
misa_status misa_hier_rerank_static(const void* q, const float* w, const void* k,
                                    int64_t k_seq_stride, const int32_t* n, const int32_t* cand,
                                    int T, int L, int H_I, int d, int kp, int topk, int dtype,
                                    int32_t* idx, float* score_opt, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MISA_H_ */

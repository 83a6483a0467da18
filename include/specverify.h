/*
 * specverify.h -- C ABI of the GB300 (sm_103a) batched speculative-decoding
 * verification library (libspecverify.so).
 *
 * What one call computes.  A batch holds B requests.  Request b drafted k_b
 * tokens x_0..x_{k_b-1} (0 <= k_b <= 32).  The target model supplied logits at
 * k_b + 1 positions (after 0, 1, .., k_b drafted tokens: "Speculative decoding
 * and multi-token prediction", section "Draft and verify", step Two; "DFlash"
 * §4 step 4, p_1..p_{gamma+1}) and the drafter supplied logits at k_b
 * positions.  Each row is turned into a temperature-scaled softmax ("FlashMap:
 * Flow Map Speculative Decoding…" §5, draft_block step 5), optionally
 * filtered by top-k and top-p, applied identically to target and draft rows
 * ("Speculative decoding and multi-token prediction", "Why the output is
 * identical").  Then:
 *   - temperature 0 (greedy): the longest prefix of drafts equal to the target
 *     argmax (lowest index on ties) is accepted and the target's own argmax
 *     token is emitted at the first disagreement, or as the bonus token after
 *     a full acceptance ("DFlash" §4 step 5; "Speculative decoding…",
 *     "Draft and verify", step Three);
 *   - temperature > 0 (sampling): draft i is accepted iff u_i < p_i(x_i) /
 *     q_i(x_i) and verification stops at the first rejection ("FlashMap…" §4
 *     "The Rejection Sampling Invariant", steps 1-2).  After a rejection at
 *     position L one token is drawn from the normalised residual
 *     max(0, p_L - q_L) ("FlashMap…" §4 step 3; "DFlash" §4); after a full
 *     acceptance a bonus token is drawn from p_k.  Both draws use the
 *     uniform u_k by inverse CDF in vocabulary-index order:
 *     y* = min{ y : C_y > u_k * S }.
 *
 * Row layout.  Request b owns target rows t_off[b] .. t_off[b] + k_b with
 * t_off[b] = sum_{j<b} (k_j + 1), and draft rows d_off[b] .. d_off[b] + k_b - 1
 * with d_off[b] = t_off[b] - b (ragged batches are packed contiguously).
 * draft_tokens[d_off[b] + i] is x_i; uniforms[t_off[b] + i] is u_i for i < k_b
 * and uniforms[t_off[b] + k_b] drives the final draw; out_tokens uses the
 * target-row layout: out_tokens[t_off[b] + j] is the j-th emitted token of
 * request b, -1 after the last emitted one.  For a fixed k this is exactly a
 * [B, k+1] matrix.
 *
 * Ownership and synchronisation.  Every pointer handed to spec_verify is a
 * device pointer owned by the caller, including the workspace.  The library
 * allocates nothing, frees nothing and never synchronises inside spec_verify:
 * all work is enqueued on the caller's stream (a cudaStream_t passed as void*;
 * NULL is the legacy default stream) and results are visible in stream order.
 * Concurrent calls are safe when they use distinct workspaces.
 *
 * Errors.  Argument errors that the host can see (null pointers, bad sizes,
 * misalignment, unsupported dtype, workspace too small) return a nonzero
 * SV_ERR_* code before anything is enqueued.  Data errors live in device
 * memory and are found by the kernels: the first one is recorded in the
 * workspace (read it with spec_verify_get_error) and every affected request
 * gets out_accept_len = -1 and out_tokens = -1.  Kernels never trap.
 */
#ifndef SPECVERIFY_H
#define SPECVERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define SV_OK 0
#define SV_ERR_ARG 1          /* null pointer, negative or inconsistent size   */
#define SV_ERR_UNSUPPORTED 2  /* dtype, vocabulary size, alignment, stride    */
#define SV_ERR_CUDA 3         /* a CUDA runtime call or launch failed          */
#define SV_ERR_WORKSPACE 4    /* workspace missing, too small or misaligned    */
/* data errors, found on the device (one request each unless stated) */
#define SV_ERR_DATA_K 16            /* k_b outside [0, SV_MAX_K]                 */
#define SV_ERR_DATA_TEMPERATURE 17  /* temperature negative, NaN or infinite     */
#define SV_ERR_DATA_TOP_P 18        /* top_p outside (0, 1]                      */
#define SV_ERR_DATA_TOP_K 19        /* top_k < 0                                 */
#define SV_ERR_DATA_TOKEN 20        /* a draft token outside [0, V)              */
#define SV_ERR_DATA_ROWS 21         /* sum(k+1) != target rows or sum(k) !=      */
                                    /* draft rows (whole batch)                  */
#define SV_ERR_DATA_LOGIT 22        /* NaN or +inf logit, or (sampling) a row    */
                                    /* with no finite logit                      */
#define SV_ERR_DATA_NO_DRAFT 23     /* temperature > 0 but draft logits absent   */
#define SV_ERR_TIMEOUT 24           /* an internal bounded wait expired (each    */
                                    /* wait gives up after 100 ms of GPU time)   */
#define SV_ERR_INTERNAL 25          /* an internal capacity invariant failed     */
#define SV_ERR_DATA_ACCEPT 26       /* KV commit: accept length above k_b         */
#define SV_ERR_DATA_PAGE 27         /* KV commit: a destination page missing from */
                                    /* the block table, or a negative kv_len;     */
                                    /* attention, eviction: a page of the request */
                                    /* missing from its block table; reservation: */
                                    /* one that would be given back               */
#define SV_ERR_DATA_LENGTH 28       /* attention, eviction: kv_len negative or    */
                                    /* longer than the block table or the scores  */
#define SV_ERR_DATA_TREE 29         /* a node's parent that is not an earlier     */
                                    /* node; KV commit: a path with no such node  */
#define SV_ERR_DATA_POOL 30         /* reservation: too few free pages for the    */
                                    /* request; of the whole call: a free count   */
                                    /* below 0, or past its list with what is     */
                                    /* given back                                 */

/* ---- limits -------------------------------------------------------------- */
#define SV_MAX_K 32              /* drafts per request (one warp ballot)       */
#define SV_TOPK_MAX 256          /* largest top-k whose kept set is listed     */
                                 /* (spec_verify_dump_rows); larger top-k and   */
                                 /* top-p alone keep a threshold instead        */
#define SV_VOCAB_MAX (1 << 22)   /* largest vocabulary                         */
#define SV_LOGPROBS_TOP_MAX 32   /* most alternatives per row (spec_logprobs)  */
#define SV_HEAD_DIM_MAX 256      /* largest attention head (spec_attention)    */
#define SV_TREE_MAX_K 63         /* drafts per request where they are a tree   */
                                 /* (and then less than 2^25 requests)         */

typedef enum { SV_F32 = 0, SV_BF16 = 1, SV_F16 = 2 } sv_dtype; /* logits: the first two */

/* A [rows, vocab] logit matrix in device memory.  `data` must be 16-byte
 * aligned and row_stride * element_size must be a multiple of 16 bytes
 * (row_stride >= vocab, in elements).  Target and draft share one dtype. */
typedef struct {
  const void* data;
  int32_t dtype;      /* sv_dtype */
  int32_t vocab;      /* V, 1 <= V <= SV_VOCAB_MAX */
  int64_t rows;
  int64_t row_stride; /* elements */
} sv_logits;

/* Optional extras of spec_verify; pass NULL for none. */
typedef struct {
  /* [draft_rows, 2] device doubles: (p_i(x_i), q_i(x_i)) of sampled requests
   * at every position the decision examined (0 .. min(L, k-1)); positions
   * after the first rejection may be NaN (filtered requests never evaluate
   * them).  NaN for greedy and failed requests (parity / diagnostics). */
  double* out_pq;
  /* cudaEvent_t handles recorded on the stream right before and right after
   * the row-streaming kernel (profiling); NULL to skip. */
  void* event_rowpass_begin;
  void* event_rowpass_end;
  /* Test of the timeout path (0 in normal use): nonzero makes one bounded
   * wait of the row pass expire, as a stalled copy's would; the request of
   * the first listed row then fails with SV_ERR_TIMEOUT and every other
   * request is verified as usual.  spec_verify only. */
  int32_t test_expire_wait;
  int32_t reserved;
} sv_options;

/* Bytes of device workspace spec_verify needs for this shape; 0 on bad
 * arguments.  The workspace must be 256-byte aligned and must not be used by
 * two calls that can run concurrently. */
size_t spec_verify_workspace_size(int32_t batch, int64_t target_rows, int64_t draft_rows);

/* Batched verification (see the file comment for what it computes).
 *   target_logits  [R_t, V]  R_t = sum_b (k_b + 1)
 *   draft_logits   [R_d, V]  R_d = sum_b k_b; the descriptor is required, its
 *                  `data` may be NULL when every temperature is 0
 *   draft_tokens   [R_d] int32            k_per_req   [B] int32, 0..SV_MAX_K
 *   temperature    [B] float, 0 = greedy
 *   top_k          [B] int32 or NULL; 0 or >= V switches top-k off; any
 *                  value in [1, V) is supported
 *   top_p          [B] float or NULL; 1 switches top-p off; (0, 1]; top-k
 *                  and top-p switch on and off independently; with both
 *                  NULL no row is filtered and the call launches one
 *                  kernel fewer (the row pass over threshold-filtered rows)
 *   uniforms       [R_t] float in [0, 1)
 *   out_accept_len [B] int32 (L, or -1 on a data error)
 *   out_tokens     [R_t] int32
 *   stream         cudaStream_t
 *   batch          B >= 0
 *   workspace      >= spec_verify_workspace_size(B, R_t, R_d) bytes
 * Returns SV_OK once the work is enqueued, else an SV_ERR_* code. */
int spec_verify(const sv_logits* target_logits, const sv_logits* draft_logits,
                const int32_t* draft_tokens, const int32_t* k_per_req,
                const float* temperature, const int32_t* top_k, const float* top_p,
                const float* uniforms, int32_t* out_accept_len, int32_t* out_tokens,
                void* stream, int32_t batch, void* workspace, size_t workspace_bytes,
                const sv_options* options);

/* Synchronises `stream`, then reads the first data error recorded by the last
 * call that used `workspace`: *code (SV_OK if none), *request and *row (-1
 * when not applicable).  Test / debug use. */
int spec_verify_get_error(const void* workspace, void* stream, int32_t* code,
                          int32_t* request, int64_t* row);

/* Synchronises `stream` and copies the per-row intermediate results of the
 * last call into host buffers (test / debug use).  Rows are numbered target
 * rows first (0 .. R_t-1), then draft rows (R_t .. R_t+R_d-1).
 *   stats      [R, 5] doubles: row max logit, softmax normaliser (sampling rows:
 *              sum of exp((x - max)/T) for unfiltered rows; the kept set's
 *              sum for rows filtered by top-p alone or a top-k above
 *              SV_TOPK_MAX; the kept weight for other filtered rows), p(x) of
 *              the row's draft token (NaN if none), greedy argmax (-1 if not
 *              computed), and the last kept token (in logit-descending,
 *              index-ascending order) of a row filtered by top-p alone or a
 *              top-k above SV_TOPK_MAX (-1 otherwise)
 *   kept_count [R] int32: size of the kept set after top-k / top-p (0 if the
 *              row was not filtered)
 *   kept_idx   [R, SV_TOPK_MAX] int32 and kept_p [R, SV_TOPK_MAX] doubles:
 *              the kept tokens in (logit desc, index asc) order and their
 *              renormalised probabilities, for rows whose top-k is active and
 *              at most SV_TOPK_MAX.  Those requests evaluate only the rows up
 *              to their first rejection (and the bonus row after k
 *              acceptances); other rows' entries are unspecified.
 * Any output pointer may be NULL. */
int spec_verify_dump_rows(const void* workspace, size_t workspace_bytes, int32_t batch,
                          int64_t target_rows, int64_t draft_rows, void* stream,
                          double* stats, int32_t* kept_count, int32_t* kept_idx,
                          double* kept_p);

/* ---- allocation-free variant ----------------------------------------------
 * The pages describe no counterpart of this entry point: it is a convenience of
 * this library for callers that cannot allocate device memory where they
 * verify (a C host program that links only this library and owns no device
 * allocator; a serving loop whose device memory is planned once and which must
 * not allocate inside its decode step).
 *
 * spec_verify_noalloc computes exactly what spec_verify computes, with the
 * same arguments minus the workspace: the workspace is a fixed buffer of
 * SV_NOALLOC_SCRATCH_BYTES inside the library (one per device).
 *   - A batch whose spec_verify_workspace_size exceeds SV_NOALLOC_SCRATCH_BYTES
 *     returns SV_ERR_WORKSPACE before anything is enqueued (16 MiB holds about
 *     1,400 logit rows, e.g. 32 requests with k = 15).
 *   - The buffer is shared: calls that can overlap on one device race on it.
 *     Order them on one stream or with events.
 *   - The buffer's address is looked up once per device, with that device
 *     current, on the first call; make that first call before any stream
 *     capture begins.
 *   - Nothing in the buffer has to start at zero.
 * Returns SV_OK once the work is enqueued, else an SV_ERR_* code. */
#define SV_NOALLOC_SCRATCH_BYTES (16u << 20)

int spec_verify_noalloc(const sv_logits* target_logits, const sv_logits* draft_logits,
                        const int32_t* draft_tokens, const int32_t* k_per_req,
                        const float* temperature, const int32_t* top_k, const float* top_p,
                        const float* uniforms, int32_t* out_accept_len, int32_t* out_tokens,
                        void* stream, int32_t batch, const sv_options* options);

/* Device address and size of the current device's spec_verify_noalloc buffer,
 * so that spec_verify_get_error / spec_verify_dump_rows can read the last
 * allocation-free call. */
int spec_verify_noalloc_scratch(void** scratch, size_t* bytes);

/* ---- draft-side sampler ---------------------------------------------------
 * The drafter's token choice that produces the drafts verified above
 * ("FlashMap: Flow Map Speculative Decoding…", §5 draft_block step 5: logits
 * divided by the temperature, softmax, a multinomial draw; the argmax at
 * temperature 0), for a batch of drafter rows laid out like spec_verify's
 * draft rows: request b owns rows d_off[b] .. d_off[b] + k_b - 1 with
 * d_off[b] = sum_{j<b} k_j.
 *   Row i of request b draws x_i = min{ y : C_y > u_i * S } by inverse CDF in
 *   vocabulary-index order over the row's distribution at the request's
 *   temperature, filtered by its top-k / top-p exactly as spec_verify filters
 *   p and q (so the q that verification recomputes is the one drawn from);
 *   temperature 0 takes the argmax of the raw logits, lowest index on ties.
 *   draft_logits  [R, V], R = sum_b k_b; same alignment rules as spec_verify
 *   k_per_req     [B] int32, 0 .. SV_MAX_K
 *   temperature   [B] float, 0 = greedy
 *   top_k, top_p  [B] or NULL, as in spec_verify
 *   uniforms      [R] float in [0, 1): row d_off[b] + i draws with u_i
 *   out_tokens    [R] int32: x_i; -1 for every row of a request with a data
 *                 error (bad parameters, NaN / +inf logit)
 *   out_q         [R] float or NULL: q_i(x_i), the drawn token's probability
 *                 (NaN for greedy and failed rows)
 *   workspace     >= spec_draft_sample_workspace_size(B, R) bytes, 256-byte
 *                 aligned, owned by the caller
 *   options       NULL, or row-pass events as in spec_verify (out_pq ignored)
 * Same ownership, stream and error conventions as spec_verify (errors are read
 * back with spec_verify_get_error on this workspace).  Returns SV_OK once the
 * work is enqueued, else an SV_ERR_* code. */
size_t spec_draft_sample_workspace_size(int32_t batch, int64_t rows);

int spec_draft_sample(const sv_logits* draft_logits, const int32_t* k_per_req,
                      const float* temperature, const int32_t* top_k, const float* top_p,
                      const float* uniforms, int32_t* out_tokens, float* out_q, void* stream,
                      int32_t batch, void* workspace, size_t workspace_bytes,
                      const sv_options* options);

/* ---- KV-cache commit after verification ------------------------------------
 * The verification stage of the serving pipeline updates the paged KV cache
 * with the accepted tokens ("FlashMap: Flow Map Speculative Decoding…",
 * section "Architecture"), and the rollback truncates on rejection
 * ("Speculative decoding and multi-token prediction", "Practical guidance").
 * The pages define no layout; this one is chosen:
 *   cache  [num_pages, n_layers, 2, page_size, E]  (K, then V), E elements of
 *          elem_bytes each per token per layer
 *   spec   [B, spec_slots, n_layers, 2, E]: the K/V the verification pass
 *          wrote for its k_b + 1 inputs, entry 0 the last emitted token (not in
 *          the cache yet), entries 1..k_b the drafts
 *   position p of request b lives in page block_table[b * max_pages + p /
 *   page_size] at slot p % page_size.
 * With accept length L = accept_len[b] >= 0 (spec_verify's output), entries
 * 0..L are written to positions kv_len[b] .. kv_len[b] + L and kv_len[b]
 * grows by L + 1; the entries of rejected drafts are not written.  L = -1 (a
 * request that failed verification) leaves the request untouched.  A request
 * with L > k_b (or L + 1 > spec_slots) fails with SV_ERR_DATA_ACCEPT, one
 * whose destination page is missing (entry < 0 or >= num_pages, or a column
 * past max_pages) or whose kv_len is negative with SV_ERR_DATA_PAGE: nothing
 * of a failed request is written and its kv_len is unchanged.  The first data
 * error is read back with spec_verify_get_error on this workspace.
 * E * elem_bytes must be a multiple of 16 and both base pointers 16-byte
 * aligned (SV_ERR_UNSUPPORTED otherwise).  All pointers are device pointers
 * owned by the caller; the call is asynchronous on `stream`. */
typedef struct {
  void* data;
  int64_t num_pages;
  int32_t n_layers;
  int32_t page_size;    /* tokens per page */
  int32_t entry_elems;  /* E */
  int32_t elem_bytes;   /* 2 or 4 */
} sv_kv_cache;

size_t spec_kv_commit_workspace_size(int32_t batch);

int spec_kv_commit(const sv_kv_cache* cache, const void* spec, int32_t spec_slots,
                   const int32_t* accept_len, const int32_t* k_per_req, int32_t* kv_len,
                   const int32_t* block_table, int32_t max_pages, void* stream, int32_t batch,
                   void* workspace, size_t workspace_bytes);

/* The same for a tree of drafts (spec_verify_tree_greedy): of request b the
 * entries path[t_off[b]] .. path[t_off[b] + L] are written, in this order, to
 * positions kv_len[b] .. kv_len[b] + L, and k_b <= SV_TREE_MAX_K.
 *   path       [rows] int32, rows = sum (k_b + 1), the layout of target rows
 *   workspace  >= spec_kv_commit_path_workspace_size(batch) bytes
 * A k_b outside [0, SV_TREE_MAX_K] or sum (k_b + 1) != rows leaves the whole
 * batch untouched (SV_ERR_DATA_K / SV_ERR_DATA_ROWS); a request with a node
 * outside [0, k_b] or not below spec_slots on its path fails with
 * SV_ERR_DATA_TREE. */
size_t spec_kv_commit_path_workspace_size(int32_t batch);

int spec_kv_commit_path(const sv_kv_cache* cache, const void* spec, int32_t spec_slots,
                        const int32_t* accept_len, const int32_t* k_per_req, const int32_t* path,
                        int64_t rows, int32_t* kv_len, const int32_t* block_table,
                        int32_t max_pages, void* stream, int32_t batch, void* workspace,
                        size_t workspace_bytes);

/* ---- LM-head GEMM with fused verification statistics ----------------------
 * The target's logits are its final hidden states times the unembedding
 * matrix, z = H W^T ("FlashMap: Flow Map Speculative Decoding…", section 1),
 * and verification needs of each logit row only its softmax statistics at the
 * row's temperature, its argmax and the logit of its token (§5 draft_block
 * step 5; §4).  spec_lmhead_stats computes them in the GEMM's epilogue on the
 * tensor cores (bf16 inputs, f32 accumulation), so the logits never reach
 * memory.  Per row r, with T_r = temperature[r] (1 is used when it is 0) and
 * x_r = tokens[r] (or -1):
 *   out_max[r]    = max_y z[r][y]                         (float)
 *   out_sum[r]    = sum_y exp((z[r][y] - out_max[r]) / T_r)  (double)
 *   out_argmax[r] = the first y with z[r][y] = out_max[r]
 *   out_token[r]  = z[r][x_r], NaN when x_r < 0 or tokens is NULL
 * so that p_r(x_r) = exp((out_token[r] - out_max[r]) / T_r) / out_sum[r].
 *   hidden   [rows, d] bf16, row-major, 16-byte aligned, d a multiple of 8
 *   unembed  [vocab, d] bf16, row-major, 16-byte aligned
 *   workspace >= spec_lmhead_stats_workspace_size(rows, vocab) bytes
 * All pointers are device pointers owned by the caller; asynchronous on
 * `stream`.  A bounded internal wait that expires is recorded as
 * SV_ERR_TIMEOUT (spec_verify_get_error on this workspace). */
size_t spec_lmhead_stats_workspace_size(int32_t rows, int32_t vocab);

int spec_lmhead_stats(const void* hidden, const void* unembed, int32_t rows, int32_t vocab,
                      int32_t d, const float* temperature, const int32_t* tokens,
                      float* out_max, double* out_sum, int32_t* out_argmax, float* out_token,
                      void* stream, void* workspace, size_t workspace_bytes);

/* ---- greedy verification from the target rows' argmax ----------------------
 * At temperature 0 verification needs of each target row only its argmax
 * (lowest index on ties): the longest prefix of drafts equal to it is accepted
 * and the argmax at the first disagreement, or after a full acceptance, is
 * emitted ("DFlash" §4 step 5; "Speculative decoding and multi-token
 * prediction", "Draft and verify", step Three).  Fed by spec_lmhead_stats'
 * out_argmax, a greedy request never needs its logits in memory.  Same row
 * layout as spec_verify:
 *   target_argmax  [R_t] int32, the argmax of target row t_off[b] + i
 *   draft_tokens   [R_d] int32 (R_d = R_t - B)    k_per_req [B] int32
 *   out_accept_len [B] int32 (L, or -1)           out_tokens [R_t] int32
 *   vocab          V: tokens and argmax values must lie in [0, V)
 *   workspace      >= spec_verify_greedy_workspace_size() bytes, 256-byte
 *                  aligned; spec_verify_get_error reads its error record
 * A k outside [0, SV_MAX_K] or sum(k + 1) != R_t fails the whole batch (all
 * outputs -1, SV_ERR_DATA_K / SV_ERR_DATA_ROWS); a token or argmax outside
 * [0, V) fails its request (SV_ERR_DATA_TOKEN).  Device pointers owned by the
 * caller; asynchronous on `stream`.  Returns SV_OK once enqueued. */
size_t spec_verify_greedy_workspace_size(void);

int spec_verify_greedy_from_argmax(const int32_t* target_argmax, const int32_t* draft_tokens,
                                   const int32_t* k_per_req, int32_t* out_accept_len,
                                   int32_t* out_tokens, void* stream, int32_t batch,
                                   int64_t target_rows, int32_t vocab, void* workspace,
                                   size_t workspace_bytes);

/* ---- greedy verification of a tree of drafts --------------------------------
 * Node 0 of a request is its last emitted token, nodes 1 .. k_b are its drafts,
 * and draft j hangs from the earlier node parent[t_off[b] + j].  The walk begins
 * at node 0 and goes on to the child whose token is the target's argmax at the
 * node it is at (the lowest such child) until there is none: the rule of
 * spec_verify at temperature 0 on the branch that the target takes.
 *   target_argmax, parent [R_t] int32, rows t_off[b] + j of node j; node 0's
 *                  parent is not read
 *   draft_tokens   [R_t - B] int32, d_off[b] + j - 1 of node j
 *   out_accept_len [B] int32 (L drafts, or -1)
 *   out_tokens     [R_t] int32: the L accepted tokens and the argmax at the last
 *                  node, then -1
 *   out_path       [R_t] int32: the L + 1 nodes of the walk, then -1
 *   workspace      >= spec_verify_tree_greedy_workspace_size(batch) bytes
 * A k outside [0, SV_TREE_MAX_K] or sum(k + 1) != R_t fails the whole batch (all
 * outputs -1, SV_ERR_DATA_K / SV_ERR_DATA_ROWS); a parent that is not an earlier
 * node (SV_ERR_DATA_TREE), a token or argmax outside [0, V) (SV_ERR_DATA_TOKEN)
 * fails its request.  Same ownership, stream and error conventions as
 * spec_verify; with batch 0 nothing is launched or written. */
size_t spec_verify_tree_greedy_workspace_size(int32_t batch);

int spec_verify_tree_greedy(const int32_t* target_argmax, const int32_t* draft_tokens,
                            const int32_t* parent, const int32_t* k_per_req,
                            int32_t* out_accept_len, int32_t* out_tokens, int32_t* out_path,
                            void* stream, int32_t batch, int64_t target_rows, int32_t vocab,
                            void* workspace, size_t workspace_bytes);

/* ---- adaptive speculation length -------------------------------------------
 * "Speculative decoding and multi-token prediction", section "Acceptance rate
 * is the whole economics": a drafted position beyond k is worth alpha^k tokens
 * for a draft step's cost c (a fraction of a target step), so speculation
 * pays while alpha^k stays above c; alpha varies per request and within a
 * response.  spec_adapt_k updates, per request, decayed counts of accepted
 * and rejected positions from the last pass's accept length and picks the next
 * k, on the stream right after spec_verify:
 *   succ[b] = decay * succ[b] + L_b,  fail[b] = decay * fail[b] + (L_b < k_b)
 *   alpha_b = (succ[b] + 1) / (succ[b] + fail[b] + 2)
 *   k_next[b] = the largest k in [k_min, k_max] with alpha_b^k > c, else k_min
 * A request with L_b = -1 keeps its counts and k_next[b] = k_used[b].
 *   accept_len, k_used [B] int32; succ, fail [B] double, in / out (start at 0);
 *   k_next [B] int32 out; alpha [B] float out or NULL.
 * 0 <= k_min <= k_max <= SV_MAX_K, 0 <= decay <= 1, c >= 0 (SV_ERR_ARG
 * otherwise).  Device pointers; asynchronous on `stream`. */
int spec_adapt_k(const int32_t* accept_len, const int32_t* k_used, double* succ, double* fail,
                 double decay, double c, int32_t k_min, int32_t k_max, int32_t* k_next,
                 float* alpha, void* stream, int32_t batch);

/* ---- attention over the paged cache ----------------------------------------
 * The target's pass over the last emitted token and the k_b drafts of every
 * request (or over one new token: k_b = 0), against the cache and the
 * speculative entries that spec_kv_commit reads and writes.  For query token j
 * of request b and head hq, whose keys are those of KV head h = hq / G with
 * G = q_heads / kv_heads:
 *   s_p = scale * q . K[p]            lse = ln sum_p exp(s_p)
 *   out = sum_p exp(s_p - lse) V[p]
 * over the positions p the token sees.  With `spec`, positions 0 ..
 * kv_len[b] - 1 are the cache's and kv_len[b] + i is entry i of the request;
 * token j sits at position kv_len[b] + j.  Without (NULL), the tokens' own
 * entries are in the cache already and token j sits at kv_len[b] - 1 - k_b + j.
 * A token sees the positions up to its own and, with window W > 0, only the
 * last W of them.  A token that sees nothing gets out = 0 and lse = -inf.
 * Slots past a request's positions are not read into any result, whatever
 * they hold.
 *   cache      elem type `dtype` (sv_dtype); entry_elems = kv_heads * head
 *              size D, D <= SV_HEAD_DIM_MAX, D * element size a multiple of 16
 *   q          [rows, q_heads, D], element strides q_token_stride and
 *              q_head_stride, D contiguous, any alignment; rows = sum (k_b + 1)
 *   spec       [B, spec_slots, n_layers, 2, E] or NULL
 *   out        [rows, q_heads, D], contiguous
 *   lse        [rows, q_heads] float
 *   workspace  >= spec_attention_workspace_size(batch, D) bytes, 256-byte
 *              aligned (its size depends on the current device's SM count)
 * A k outside [0, SV_MAX_K] or sum (k + 1) != rows fails the whole batch
 * (SV_ERR_DATA_K / SV_ERR_DATA_ROWS, every output NaN).  A request whose
 * kv_len is negative or above max_pages * page_size, or of more than 2^31 - 256
 * positions with its tokens (SV_ERR_DATA_LENGTH), or with more than spec_slots tokens (SV_ERR_DATA_K) gets NaN rows; so does a
 * row of a request that needs a page missing from its block table
 * (SV_ERR_DATA_PAGE).  Results do not depend on the batch's order in time:
 * sums have a fixed order on a given device.  Same ownership, stream and
 * error conventions as spec_verify; a call of this and the following entries
 * with batch (rows) 0 launches nothing and leaves the workspace as it is, so
 * that there is no error of it to read. */
size_t spec_attention_workspace_size(int32_t batch, int32_t head_dim);

int spec_attention(const sv_kv_cache* cache, int32_t dtype, int32_t layer, int32_t kv_heads,
                   const void* q, int64_t q_token_stride, int64_t q_head_stride, int32_t q_heads,
                   int64_t rows, const void* spec, int32_t spec_slots, const int32_t* k_per_req,
                   const int32_t* kv_len, const int32_t* block_table, int32_t max_pages,
                   float scale, int32_t window, void* out, float* lse, void* stream,
                   int32_t batch, void* workspace, size_t workspace_bytes);

/* The same over a tree of drafts: node j of request b (node 0 the last emitted
 * token) hangs from the earlier node parent[t_off[b] + j], lies one position
 * behind it (node 0 at kv_len[b]), and sees the cached positions, its ancestors
 * and itself, with window W > 0 only the last W of them.  k_b <= SV_TREE_MAX_K,
 * and `spec`, entry j of node j, is needed.  A request whose tree has a parent
 * that is no earlier node gets NaN rows (SV_ERR_DATA_TREE); node 0's parent is
 * not read.  A row that sees an infinite value whose weight is 0 in the type may
 * be NaN there, where the formula's weight is tiny and its result infinite.  All
 * else as in spec_attention. */
size_t spec_tree_attention_workspace_size(int32_t batch, int32_t head_dim);

int spec_tree_attention(const sv_kv_cache* cache, int32_t dtype, int32_t layer, int32_t kv_heads,
                        const void* q, int64_t q_token_stride, int64_t q_head_stride,
                        int32_t q_heads, int64_t rows, const void* spec, int32_t spec_slots,
                        const int32_t* k_per_req, const int32_t* parent, const int32_t* kv_len,
                        const int32_t* block_table, int32_t max_pages, float scale, int32_t window,
                        void* out, float* lse, void* stream, int32_t batch, void* workspace,
                        size_t workspace_bytes);

/* ---- attention over packed prompts -----------------------------------------
 * Causal attention within each of B sequences that lie one behind another in the
 * rows of q, k and v; sequence b has rows offsets[b] .. offsets[b + 1] - 1.  For
 * its token i and head hq, whose keys are those of KV head h = hq / G with
 * G = q_heads / kv_heads:
 *   s_j = scale * q_i . k_j        lse = ln sum_j exp(s_j)
 *   out = sum_j exp(s_j - lse) v_j
 * over its tokens j <= i, with window W > 0 only the last W of them.
 *   q        [rows, q_heads, D], k, v [rows, kv_heads, D] of `dtype` (sv_dtype),
 *            element strides of row and head, D contiguous, any alignment
 *   offsets  [B + 1] int32
 *   out      [rows, q_heads, D], contiguous;  lse  [rows, q_heads] float
 *   workspace >= spec_prompt_attention_workspace_size(batch) bytes, 256-byte
 *            aligned (its size depends on the current device's SM count)
 * Rows of no sequence are neither read into a result nor written.  Infinite and
 * NaN keys and values reach the tokens that see them only; such a value where the
 * type holds no weight but 0 gives NaN.  A product of +inf makes its row NaN, a
 * position of -inf weighs nothing.  Offsets that descend or leave [0, rows]
 * fail the whole batch (SV_ERR_DATA_ROWS, every output NaN).  rows < 2^31 - 256,
 * batch * kv_heads < 2^31 - 1.
 * Results do not depend on the run.  Same ownership, stream and error
 * conventions as spec_verify; with rows or batch 0 nothing is launched. */
size_t spec_prompt_attention_workspace_size(int32_t batch);

int spec_prompt_attention(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                          const void* k, int64_t k_row_stride, int64_t k_head_stride,
                          const void* v, int64_t v_row_stride, int64_t v_head_stride,
                          int32_t dtype, int64_t rows, int32_t q_heads, int32_t kv_heads,
                          int32_t head_dim, const int32_t* offsets, float scale, int32_t window,
                          void* out, float* lse, void* stream, int32_t batch, void* workspace,
                          size_t workspace_bytes);

/* ---- block tables from the requests' lengths ---------------------------------
 * Gives every request the pages for length[b] positions: need[b] = ceil(length[b]
 * / page_size) entries of its table row instead of held[b].  The free pages are a
 * stack, free_pages[0 .. *free_count - 1].
 *   - Columns need[b] .. held[b] - 1 of requests that hold more become -1, and
 *     their pages go onto the stack in the order of the requests and columns.
 *   - Requests that need more take pages off its end, request by request and
 *     column by column, as long as what is wanted so far is there: a request from
 *     which on it is not, and those behind it that want any, keep what they hold
 *     (SV_ERR_DATA_POOL).
 *   - Entries of the list from the new count up to the old one become -1; those
 *     past both stay as they are.
 *   table, out_table      [B, max_pages] int32; held, out_held, length [B] int32
 *   free_pages, out_free  [capacity] int32; free_count, out_count [1] int32
 *   workspace             >= spec_kv_reserve_workspace_size(batch, capacity)
 * An output may be its input (in place) or a buffer of its own, which then gets
 * the whole contents.  A request with held or need outside [0, max_pages] or a
 * negative length is left as it is (SV_ERR_DATA_LENGTH), and so is one with an
 * entry below 0 among those it would give back (SV_ERR_DATA_PAGE).  A free count
 * below 0, or above the capacity with all that would be given back, changes nothing
 * for the whole batch (SV_ERR_DATA_POOL, request -1).  Same conventions as spec_verify; with
 * batch 0 the free list and its count are still copied to buffers of their own, and
 * nothing is launched where they are in place. */
size_t spec_kv_reserve_workspace_size(int32_t batch, int64_t capacity);

int spec_kv_reserve(const int32_t* table, int32_t* out_table, int32_t max_pages,
                    const int32_t* held, int32_t* out_held, const int32_t* length,
                    const int32_t* free_pages, int32_t* out_free, int64_t capacity,
                    const int32_t* free_count, int32_t* out_count, int32_t page_size,
                    void* stream, int32_t batch, void* workspace, size_t workspace_bytes);

/* ---- slots of a step's new tokens ---------------------------------------------
 * Row r of a step that appends count[b] tokens to request b, request by request
 * (offsets[b] = sum of the counts before it), is token start[b] + r - offsets[b]
 * of the request and lies in slot page * page_size + position % page_size.
 *   out_slots    [rows] int64, -1 for rows past the last token
 *   out_request, out_position  [rows] int32, -1 there
 *   out_offsets  [B + 1] int32, as spec_prompt_attention takes them
 *   workspace    >= spec_kv_slots_workspace_size(batch, rows)
 * A request with a negative start or count, or with positions past its table row,
 * has slots -1 (SV_ERR_DATA_LENGTH; a negative count is none); so has a row whose
 * page is missing (SV_ERR_DATA_PAGE).  More tokens than rows fail the batch (every
 * row -1, SV_ERR_DATA_ROWS).  Same conventions as spec_verify. */
size_t spec_kv_slots_workspace_size(int32_t batch, int64_t rows);

int spec_kv_slots(const int32_t* block_table, int32_t max_pages, const int32_t* start,
                  const int32_t* count, int64_t rows, int32_t page_size, int64_t* out_slots,
                  int32_t* out_request, int32_t* out_position, int32_t* out_offsets, void* stream,
                  int32_t batch, void* workspace, size_t workspace_bytes);

/* ---- keys and values into their slots -------------------------------------------
 * cache[slot / page_size, layer, 0 | 1, slot % page_size] = k | v of each row.
 *   k, v       [rows, kv_heads, D] of the cache's type, element strides of row and
 *              head, D contiguous, any alignment
 *   slots      [rows] int64, none twice; -1: the row is not written
 *   workspace  >= spec_kv_write_workspace_size(rows) bytes
 * A row with any other slot outside the pool is not written (SV_ERR_DATA_PAGE, and
 * its row).  Of two rows with one slot either may stay, in pieces.  Same conventions
 * as spec_verify; with rows 0 nothing is launched. */
size_t spec_kv_write_workspace_size(int64_t rows);

int spec_kv_write(const sv_kv_cache* cache, int32_t layer, int32_t kv_heads, const void* k,
                  int64_t k_row_stride, int64_t k_head_stride, const void* v,
                  int64_t v_row_stride, int64_t v_head_stride, const int64_t* slots, int64_t rows,
                  void* stream, void* workspace, size_t workspace_bytes);

/* ---- accumulated attention weights -----------------------------------------
 * How much each cached position is attended to, for spec_kv_evict:
 *   out_score[b][p] = score[b][p] + sum_j sum_hq exp(s_p - lse[j][hq])
 * over the heads and the query tokens j = 0 .. accept_len[b] (all k_b + 1 when
 * accept_len is NULL; none, and nothing written, when it is -1), with the q,
 * lse and lengths of spec_attention before spec_kv_commit.  Positions 0 ..
 * kv_len[b] - 1 are written, and with `spec` also kv_len[b] .. kv_len[b] +
 * accept_len[b], the positions that spec_kv_commit appends; positions past
 * them stay as they are, so scores that start at zero stay zero beyond the
 * cached length.
 *   score, out_score  [B, score_cols] float with row strides score_stride and
 *                     out_stride; they may be the same buffer
 *   workspace         >= spec_attention_weights_workspace_size(batch)
 * A request with an accept length above k_b (SV_ERR_DATA_ACCEPT), with
 * positions past score_cols or its block table (SV_ERR_DATA_LENGTH) or more
 * than spec_slots tokens (SV_ERR_DATA_K) is left untouched; positions on a
 * missing page are not written (SV_ERR_DATA_PAGE).  A batch error writes
 * nothing; positions that an expired wait left out (SV_ERR_TIMEOUT) stay as they
 * are.  Each score has one writer and a fixed order of its sum. */
size_t spec_attention_weights_workspace_size(int32_t batch);

int spec_attention_weights(const sv_kv_cache* cache, int32_t dtype, int32_t layer,
                           int32_t kv_heads, const void* q, int64_t q_token_stride,
                           int64_t q_head_stride, int32_t q_heads, int64_t rows, const void* spec,
                           int32_t spec_slots, const int32_t* k_per_req, const int32_t* kv_len,
                           const int32_t* block_table, int32_t max_pages, float scale,
                           int32_t window, const float* lse, const int32_t* accept_len,
                           const float* score, int64_t score_stride, float* out_score,
                           int64_t out_stride, int32_t score_cols, void* stream, int32_t batch,
                           void* workspace, size_t workspace_bytes);

/* ---- eviction from the paged cache -----------------------------------------
 * Keeps at most `budget` positions of every request: its first `sinks`, its
 * last `recent` and, of the others, those of the largest score (the lowest
 * position on ties, NaN below every number); sinks + recent <= budget.  A
 * request of n <= budget positions keeps all.  Kept positions keep their
 * order: kept position i moves to position i, K and V of every layer, its
 * score moves to out_score[b][i], scores from there to n become 0 and
 * out_len[b] the number kept.
 * In place (dst NULL, or this cache with block_table itself): entries move within
 * the request's own pages, which no other request may share; pages past the new
 * length are free.  Else the kept entries are written to dst at dst_table's pages
 * (another cache of the same geometry, or pages of this one that no request's
 * source lies in) and the source stays as it is.
 *   score       [B, score_cols] float, row stride score_stride
 *   out_score   [B, out_cols] float, row stride out_stride; may be score
 *   kv_len      [B] int32; out_len [B] int32, may be kv_len
 *   out_kept    [B, budget] int32 or NULL: the kept positions, then -1
 *   workspace   >= spec_kv_evict_workspace_size(batch, budget) bytes
 * A request with kv_len negative or past its block table, score_cols or (kept
 * part) out_cols or dst_table fails with SV_ERR_DATA_LENGTH, one with a
 * missing page with SV_ERR_DATA_PAGE: nothing of it moves, out_kept is -1,
 * out_len stays where it is kv_len and is -1 elsewhere.  batch <= 65535. */
size_t spec_kv_evict_workspace_size(int32_t batch, int32_t budget);

int spec_kv_evict(const sv_kv_cache* cache, const int32_t* block_table, int32_t max_pages,
                  const sv_kv_cache* dst, const int32_t* dst_table, int32_t dst_max_pages,
                  const float* score, int64_t score_stride, int32_t score_cols, float* out_score,
                  int64_t out_stride, int32_t out_cols, const int32_t* kv_len, int32_t* out_len,
                  int32_t budget, int32_t sinks, int32_t recent, int32_t* out_kept, void* stream,
                  int32_t batch, void* workspace, size_t workspace_bytes);

/* ---- log probabilities of given tokens -------------------------------------
 * Per row r of the logits, with z = x / T_r (T_r = temperature[r]; NULL or 0
 * stands for 1), m = max x and t = tokens[r]:
 *   out_logsum[r]  = ln sum_y exp((x_y - m) / T)     out_max[r] = m
 *   out_logprob[r] = (x_t - m) / T - out_logsum[r]
 *   out_entropy[r] = -sum_y p_y ln p_y
 *   out_top_tokens[r][i], out_top_logprobs[r][i]: the n_top most likely tokens,
 *     the largest logit first and the lowest index on ties; tokens of
 *     probability 0 (-inf) are none: -1 and -inf stand for what is missing
 * A row with token -1 (spec_verify's mark past the last emitted token) is not
 * read: NaN, and -1 for tokens.  tokens NULL: no log probability (NaN), the
 * rest as usual.  Rows may start at any element: `data` needs the alignment of
 * its element only and row_stride >= vocab is any.
 *   out_*       [rows] float, each may be NULL; out_top_* [rows, n_top] int32
 *               and float, needed when n_top > 0; n_top <= SV_LOGPROBS_TOP_MAX
 *   workspace   >= spec_logprobs_workspace_size(rows) bytes
 * A row with a temperature that is negative, not finite or below 1e-30
 * (SV_ERR_DATA_TEMPERATURE), a token below -1 or not below vocab
 * (SV_ERR_DATA_TOKEN), or a NaN, a +inf or no finite logit (SV_ERR_DATA_LOGIT)
 * gets NaN and -1. */
size_t spec_logprobs_workspace_size(int64_t rows);

int spec_logprobs(const sv_logits* logits, const int32_t* tokens, const float* temperature,
                  int32_t n_top, float* out_logprob, float* out_entropy, float* out_max,
                  float* out_logsum, int32_t* out_top_tokens, float* out_top_logprobs,
                  void* stream, void* workspace, size_t workspace_bytes);

/* The gradient of a loss with respect to the logits, given its gradients
 * g_logprob and g_entropy ([rows] float, either may be NULL for 0) and the
 * forward call's out_max, out_logsum and (with g_entropy) out_entropy:
 *   dx_y = (1/T) (g_logprob (1[y = t] - p_y) - g_entropy p_y (ln p_y + H))
 * out: [rows, vocab] of the logits' type, row stride out_stride, any
 * alignment; it may be the logits themselves.  A row with token -1 gets 0, one
 * whose forward results are NaN or whose token or temperature is bad NaN. */
int spec_logprobs_grad(const sv_logits* logits, const int32_t* tokens, const float* temperature,
                       const float* max, const float* logsum, const float* entropy,
                       const float* g_logprob, const float* g_entropy, void* out,
                       int64_t out_stride, void* stream);

/* Test of the timeout path of spec_logprobs, and of spec_attention and
 * spec_attention_weights on the tensor cores (process-wide, 0 in normal use): while
 * it is n > 0, block n - 1 of every call, if it has work, lets one bounded wait, on
 * a barrier nothing arrives on, run out after 1 ms.  The call then reports
 * SV_ERR_TIMEOUT. */
void spec_test_expire_wait(int32_t n);

/* Human-readable text of a status code. */
const char* spec_verify_strerror(int code);

/* Library version, major * 10000 + minor * 100 + patch. */
int spec_verify_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_H */

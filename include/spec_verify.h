/*
 * spec_verify.h -- C ABI of the speculative-decoding verify step on GB300.
 *
 * The verify step of speculative decoding (draft model proposes gamma tokens
 * or a tree of them; the target model checks them all in one forward) has
 * three data-parallel parts:
 *
 *   spec_verify_attn    append the new rows' K/V to a paged cache and run the
 *                       masked attention of the gamma+1 (or tree) queries;
 *   spec_reject_sample  temperature softmax of target and draft logits,
 *                       accept/reject of each draft token, and the
 *                       replacement or bonus draw;
 *   kv_commit           roll the cache back to the accepted prefix, or
 *                       compact the accepted tree path;
 *
 * and beside them what a serving step needs around the verify:
 *
 *   spec_block_tables   block tables, slot map and positions of the new rows
 *                       from the requests' lengths;
 *   spec_qk_norm_rope   per-head norm and position rotation of the queries and
 *                       keys that spec_verify_attn takes;
 *   spec_verify_attn_window  verify attention with a sliding window and sinks;
 *   spec_sample         the draft's own draws, and plain decoding.
 *
 * Conventions shared by every call
 *   - Every tensor pointer is caller-owned DEVICE memory, dense and
 *     row-major in the stated shape.  The library never allocates, never
 *     frees and never synchronises (except spec_get_device_status).  All work
 *     is enqueued on `stream` (a cudaStream_t passed as void*; NULL = the
 *     legacy default stream).  Calls are re-entrant; the state kept between
 *     calls is a per-thread count of launches (spec_last_launch_count),
 *     cached driver entry points, and the scratch array of
 *     spec_reject_sample_noalloc with its device address per CUDA context.
 *   - Every device-side wait is bounded (spec_dims.wait_limit_kcycles); one
 *     that gives up raises SPEC_ERR_TIMEOUT.  After that bit is seen, clear
 *     the status word and zero the workspace again (spec_workspace_init)
 *     before the next call: counters inside it may be left mid-way.
 *   - B requests, M query rows per request (row 0 = the pending root token
 *     whose K/V is not cached yet, rows 1.. = drafts or tree nodes), Hq query
 *     heads, Hkv KV heads (Hq % Hkv == 0), head size D, vocabulary V.
 *   - Tree topology: parent[B][M] int32 with parent[b][0] = -1 and
 *     0 <= parent[b][n] < n for n >= 1 (BFS or any topological numbering).
 *     parent == NULL means the chain parent[n] = n - 1.
 *   - Errors the host can see (bad sizes, NULL pointers, short workspace)
 *     return at once and launch nothing.  Errors only the device can see
 *     (a block id out of range, a context that does not fit the block table,
 *     a bad temperature, a row with no distribution) set a bit in the status
 *     word kept in the workspace and make the affected request a no-op with
 *     defined outputs; read them with spec_get_device_status.
 *
 * Sources: three practitioner pages on speculative decoding -- page 1
 * "投机推理..." (kwkr.cn) §2.1, §2.3, §4.1, §4.3, §5.1, §5.3; page 2
 * "推测解码..." (cf-1.com) §2.1-§2.3, §3.3, §4.3, §5.4; page 3
 * "推测解码的工程真相 2026" (blog.lonae.com), formal-definition and
 * tree-attention sections.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum spec_status {
  SPEC_OK = 0,
  SPEC_ERR_INVALID_ARG = 1,   /* bad size, NULL pointer, bad temperature/topology */
  SPEC_ERR_CAPACITY = 2,      /* ctx + M exceeds the request's block-table capacity */
  SPEC_ERR_UNSUPPORTED = 3,   /* shape or dtype this build has no kernel for */
  SPEC_ERR_CUDA = 4,          /* a CUDA runtime call failed */
  SPEC_ERR_NONFINITE = 5,     /* a logits row holds NaN/+inf or only -inf */
  SPEC_ERR_DEVICE_BOUNDS = 6, /* a block id or token id out of range */
  SPEC_ERR_TIMEOUT = 7        /* a device-side wait gave up (bounded, never hangs) */
} spec_status;

typedef enum spec_dtype { SPEC_BF16 = 0, SPEC_F32 = 1 } spec_dtype;

/* Attention kernel selection (spec_dims.attn_impl). */
typedef enum spec_attn_impl {
  SPEC_ATTN_AUTO = 0,          /* tensor cores when the shape allows, else CUDA cores */
  SPEC_ATTN_CUDA_CORES = 1,    /* split-KV on CUDA cores: group*M <= 128, D 64/128, bf16/f32 */
  SPEC_ATTN_TENSOR_CORES = 2   /* tcgen05 + TMA: bf16, D = 128, group*M <= 128 */
} spec_attn_impl;

/* Reject-sample kernel selection (spec_dims.reject_impl). */
typedef enum spec_reject_impl {
  SPEC_REJECT_AUTO = 0,        /* the staged kernels (the faster choice measured on
                                  GB300 at every shape tried) */
  SPEC_REJECT_STAGED = 1,      /* logit statistics, then for a chain with 16-byte
                                  aligned rows and no filter one tail kernel
                                  (decisions, residual masses and draw, several CTAs
                                  per request); for a tree with such rows and no
                                  filter the walk by a cluster of 8 CTAs per request
                                  beside the statistics (which still decide which
                                  requests fail); else three kernels (decisions,
                                  residual masses, residual draws); any alignment,
                                  V up to 2^20 */
  SPEC_REJECT_FUSED = 2        /* one kernel for a chain: every warp streams logit
                                  statistics and decides each request as soon as its
                                  rows are done; chains with 16-byte aligned rows
                                  (V * element size a multiple of 16, aligned row
                                  pointers), V up to 2^20, no filter;
                                  SPEC_ERR_UNSUPPORTED otherwise */
} spec_reject_impl;

typedef struct spec_dims {
  int32_t B;            /* requests in the batch */
  int32_t M;            /* query rows per request: gamma+1, or tree nodes incl. root;
                           1..128 (SPEC_ERR_UNSUPPORTED above) */
  int32_t Hq;           /* query heads */
  int32_t Hkv;          /* KV heads; query head h reads KV head h / (Hq/Hkv) */
  int32_t D;            /* head size (64 or 128) */
  int32_t block;        /* tokens per KV block; must be 16 */
  int32_t max_blocks;   /* entries per block-table row */
  int32_t num_blocks;   /* physical blocks in each cache */
  int32_t V;            /* vocabulary size */
  int32_t kv_dtype;     /* spec_dtype of q, k_new, v_new, caches and out */
  int32_t logits_dtype; /* spec_dtype of target and draft logits */
  float softmax_scale;  /* attention score scale; 0 selects 1/sqrt(D) */
  int32_t attn_impl;    /* spec_attn_impl; 0 = automatic choice */
  int32_t reject_impl;  /* spec_reject_impl; 0 = automatic choice */
  int32_t wait_limit_kcycles; /* every bounded device wait gives up after this
                                 many thousand SM clocks and raises
                                 SPEC_ERR_TIMEOUT; 0 = the default, 4e6
                                 (about 2 s at 2 GHz).  Work already issued
                                 (copies, MMAs) is always waited for before a
                                 CTA exits, whatever this limit. */
} spec_dims;

/* Bytes of caller-owned device workspace every call with these dims needs
 * (status word, split-KV partials, row statistics, per-request state).
 * Returns 0 if the dims are invalid. */
size_t spec_workspace_size(const spec_dims* dims);

/* Zero the workspace (status word included).  Call once after allocating it;
 * afterwards every call leaves it ready for the next.  An async memset on
 * `stream`.
 *
 * Calls of different dims may take turns on one workspace (of the largest
 * one's size) if they are spec_verify_attn, spec_verify_attn_window,
 * spec_block_tables, spec_qk_norm_rope, spec_sample, spec_lm_head and
 * kv_commit.  spec_reject_sample, its filtered form and
 * spec_reject_sample_lm_head keep counters at places that depend on dims: a
 * workspace that they use serves one spec_dims, or is zeroed again before a
 * call of theirs that follows one of other dims.  Calls that may run at the same
 * time (on two streams, in two graphs) have a workspace each; only
 * spec_qk_norm_rope, spec_sample, spec_lm_head and kv_commit, which keep nothing
 * in it but the status word and a count, may share one. */
spec_status spec_workspace_init(void* ws, size_t ws_bytes, void* stream);

/* Synchronise `stream` and read the device status word: bit (1 << code) is
 * set for every spec_status code a device-side check raised since the last
 * clear.  clear != 0 resets the word afterwards. */
spec_status spec_get_device_status(void* ws, void* stream, int32_t* flags,
                                   int32_t clear);

/*
 * spec_verify_attn -- KV append and verify attention (one layer).
 *
 * Page 1 §2.1: feed all candidate positions at once; under the causal mask
 * each position sees only what precedes it, so the parallel pass equals
 * token-by-token decoding, provided the KV cache is extended in the right
 * order.  Page 2 §3.3: reuse the cached prefix and compute K/V only for the
 * new positions.  Page 3 (tree-attention section) and page 2 §5.4: a draft
 * tree is verified in one pass under a mask that follows the tree.
 *
 *   q        [B, M, Hq, D]   kv_dtype   queries (position encoding applied)
 *   k_new    [B, M, Hkv, D]  kv_dtype   K of the M new rows
 *   v_new    [B, M, Hkv, D]  kv_dtype   V of the M new rows
 *   k_cache  [num_blocks, Hkv, 16, D]   paged K cache (in/out)
 *   v_cache  [num_blocks, Hkv, 16, D]   paged V cache (in/out)
 *   block_table [B, max_blocks] int32   position t of request b lives in
 *                                       block block_table[b][t/16], slot t%16
 *   ctx_lens [B] int32      cached tokens of request b before this step
 *   parent   [B, M] int32 or NULL (chain)
 *   out      [B, M, Hq, D]   kv_dtype   attention output
 *   lse      [B, M, Hq] float or NULL   natural-log log-sum-exp of the
 *                                       scaled scores of each row
 *
 * Effect: rows i = 0..M-1 of k_new/v_new are written to positions
 * ctx+i; the remaining slots of the last block touched are set to zero.
 * Then row i attends to positions 0..ctx-1 and to the new positions
 * ctx+k for every k that is i or an ancestor of i (k <= i for a chain),
 * with scores scaled by softmax_scale.
 * A request whose ctx + M exceeds max_blocks*16 (SPEC_ERR_CAPACITY, the
 * pages' cue to fall back to plain decoding) or whose needed block ids are
 * out of range (SPEC_ERR_DEVICE_BOUNDS) leaves the caches untouched and
 * gets out = 0, lse = -inf.
 */
spec_status spec_verify_attn(const void* q, const void* k_new,
                             const void* v_new, void* k_cache, void* v_cache,
                             const int32_t* block_table,
                             const int32_t* ctx_lens, const int32_t* parent,
                             void* out, float* lse, const spec_dims* dims,
                             void* ws, size_t ws_bytes, void* stream);

/*
 * spec_verify_attn_window -- spec_verify_attn with a sliding window and sinks.
 *
 * Page 3 (tree-attention section) and page 2 §3.3 leave the cache's growth to
 * the engine; a model with a sliding window reads only the last `window`
 * positions and the first `sinks` ones.  Row i stands at position
 * ctx + depth(i) (ctx + i in a chain); of the keys that spec_verify_attn shows
 * it, it sees those at positions below `sinks` or greater than its own less
 * `window` (itself included; a new key stands at ctx plus its node's depth).
 *
 *   window >= 1, sinks >= 0
 * Other arguments as in spec_verify_attn.  Keys and values at positions that
 * are neither among the first `sinks` nor from ctx - window + 1 on are not
 * read and may be anything, and so may the table entries of pages that hold
 * only such positions (spec_block_tables returns those pages).  Keys and
 * values that some row of a request sees have to be finite.  A window of the whole context
 * gives spec_verify_attn's results, up to the order of the sums and the bf16
 * rounding of the probabilities, which the tensor cores take relative to the
 * running maximum (as without a window: an output is off by up to 2^-8 of
 * sum p |v| before it is rounded; the CUDA cores hold probabilities in fp32).
 */
spec_status spec_verify_attn_window(const void* q, const void* k_new, const void* v_new,
                                    void* k_cache, void* v_cache, const int32_t* block_table,
                                    const int32_t* ctx_lens, const int32_t* parent, int32_t window,
                                    int32_t sinks, void* out, float* lse, const spec_dims* dims,
                                    void* ws, size_t ws_bytes, void* stream);

/*
 * spec_reject_sample -- accept / reject / resample of the drafts.
 *
 * p = softmax(target/T), q = softmax(draft/T) with the request's temperature
 * (page 1 §3.3).  Draft token x of node c is accepted iff
 * u_acc(c) * q(x) < p(x), i.e. with probability min(1, p/q) (page 1 §2.3,
 * §4.1; page 2 §2.1); the walk stops at the first rejection (page 1 §4.3).
 * After a rejection the token is drawn from normalize(max(0, p - q)); if the
 * walk reaches a node without children the bonus token is drawn from p
 * (page 3, formal definition).  In a tree the children of a node are tried
 * in ascending order and each rejection replaces the working target P by
 * normalize(max(0, P - q)); the first accepted child is entered.  Draws use
 * the inverse CDF in vocabulary order: the smallest k with C_k > u*Z.
 *
 * Uniforms: Philox4x64-10 (Salmon et al., SC'11), key (seed, 0), counter
 * (n+1, b_base+b, offset, 0) for node n of request b; u_acc = (w0>>40)*2^-24,
 * u_smp = (w1>>40)*2^-24.
 *
 *   target_logits [B, M, V] logits_dtype   row n: law of n's children
 *   draft_logits  [B, M, V] logits_dtype   row n: q that drafted n's children
 *                                          (rows of leaves are not read)
 *   tokens        [B, M] int32   drafted token of node n (tokens[b][0] unused)
 *   parent        [B, M] int32 or NULL (chain)
 *   temperature   [B] float      a positive normal finite value, or 0:
 *                                greedy (page 1 §4.3, first point) -- each
 *                                row's law is the point mass on its largest
 *                                logit (smallest index among equal ones), so
 *                                a draft is accepted iff it is that token
 *                                and every draw returns it
 *   out_tokens    [B, M] int32   emitted tokens: the a accepted drafts, then
 *                                the drawn token; -1 after that
 *   path          [B, M] int32   accepted node indices, starting with 0; -1 after
 *   accepted_len  [B] int32      a (number of accepted drafts), -1 if failed
 *   probe         [B, M, 4] float or NULL: for every tested node n, p(x_n)
 *                 and q(x_n) as used in its test (cols 0, 1); at the node
 *                 where the draw happened, the mass Z of the residual that
 *                 was drawn from (1 for a bonus draw) and the probability of
 *                 the drawn token (cols 2, 3); -1 elsewhere.
 * A failed request (bad temperature, token, topology, or a needed row with
 * no distribution) gets accepted_len = -1 and -1 rows.  If a wait gave up
 * (SPEC_ERR_TIMEOUT in the status word, from this call or an earlier one not
 * yet cleared), every request of the call gets accepted_len = -1: no
 * decision is made on statistics that may be incomplete.
 */
spec_status spec_reject_sample(const void* target_logits,
                               const void* draft_logits,
                               const int32_t* tokens, const int32_t* parent,
                               const float* temperature, uint64_t seed,
                               uint64_t offset, uint64_t b_base,
                               int32_t* out_tokens, int32_t* path,
                               int32_t* accepted_len, float* probe,
                               const spec_dims* dims, void* ws,
                               size_t ws_bytes, void* stream);

/*
 * spec_reject_sample_filtered -- spec_reject_sample with top-k / top-p
 * restricted laws.
 *
 * Page 2 §5.1: target and draft must sample by one rule (its example: a
 * nucleus-sampling target against a differently sampling draft).  For a
 * request with top_k[b] = k and top_p[b] = t, the law of every row it uses,
 * target and draft alike, is restricted to a prefix of the row's tokens in
 * the order of their logits, largest first, the smaller index first among
 * equal logits: the first k tokens (k = 0: all), then the shortest prefix of
 * those whose mass reaches t times their mass (t = 1: all of them); the
 * restricted law is renormalised and the walk above runs on it, so the
 * emitted tokens follow the restricted target law.  At temperature 0 the
 * filters change nothing.
 *
 *   top_k  [B] int32 or NULL   >= 0 (0: no top-k)
 *   top_p  [B] float or NULL   in (0, 1] (1: no top-p)
 * Other arguments as in spec_reject_sample.  A request with k < 0 or t
 * outside (0, 1] fails (SPEC_ERR_INVALID_ARG, accepted_len = -1).  The probe
 * reports the restricted laws.  Filters run on the staged kernels: with
 * dims->reject_impl = SPEC_REJECT_FUSED and a filter given the call returns
 * SPEC_ERR_UNSUPPORTED and launches nothing.  Each needed row of a filtered
 * request costs a few extra passes over the row (its kept prefix is found by
 * a radix select over the logits' order keys).
 */
spec_status spec_reject_sample_filtered(const void* target_logits,
                                        const void* draft_logits,
                                        const int32_t* tokens, const int32_t* parent,
                                        const float* temperature,
                                        const int32_t* top_k, const float* top_p,
                                        uint64_t seed, uint64_t offset, uint64_t b_base,
                                        int32_t* out_tokens, int32_t* path,
                                        int32_t* accepted_len, float* probe,
                                        const spec_dims* dims, void* ws,
                                        size_t ws_bytes, void* stream);

/*
 * spec_lm_head -- logits of an LM head: logits[r, v] = sum_k hidden[r, k] *
 * weight[v, k] (bf16 inputs, fp32 accumulation on the tensor cores, bf16
 * output rounded to nearest even).
 *
 * Page 2 §1.2: decoding is bound by weight and logit reads; this is the
 * product the verify step's logits come from.
 *   hidden  [rows, H] bf16   row-major, 16-byte aligned
 *   weight  [V, H]    bf16   row-major (one vocabulary row of H weights)
 *   logits  [rows, V] bf16   output
 *   ws, ws_bytes             at least 16 bytes (its first word is the status
 *                            word of spec_get_device_status)
 * H must be a multiple of 64 and V of 256 (else SPEC_ERR_UNSUPPORTED).
 */
spec_status spec_lm_head(const void* hidden, const void* weight, int32_t rows, int32_t H,
                         int32_t V, void* logits, void* ws, size_t ws_bytes, void* stream);

/*
 * spec_reject_sample_lm_head -- the LM heads and the verify decisions in one
 * call, without a second pass over the logit rows.
 *
 * The target and draft logits of the B*M new rows are computed as in
 * spec_lm_head (target: hidden_target [B, M, Ht] x weight_target [V, Ht];
 * draft: hidden_draft [B, M, Hd] x weight_draft [V, Hd]) into target_logits
 * and draft_logits ([B, M, V] bf16, written); their epilogue also forms the
 * per-chunk statistics the decisions need (page 2 §1.2: the logit rows are
 * read once less), and spec_reject_sample's decisions and draws follow on
 * them.  Arguments after draft_logits and the outputs are those of
 * spec_reject_sample; dims->logits_dtype must be bf16, Ht and Hd multiples
 * of 64, dims->V a multiple of 256; SPEC_REJECT_FUSED is refused.
 */
spec_status spec_reject_sample_lm_head(const void* hidden_target, const void* weight_target,
                                       int32_t Ht, const void* hidden_draft,
                                       const void* weight_draft, int32_t Hd,
                                       void* target_logits, void* draft_logits,
                                       const int32_t* tokens, const int32_t* parent,
                                       const float* temperature, uint64_t seed, uint64_t offset,
                                       uint64_t b_base, int32_t* out_tokens, int32_t* path,
                                       int32_t* accepted_len, float* probe,
                                       const spec_dims* dims, void* ws, size_t ws_bytes,
                                       void* stream);

/*
 * kv_commit -- roll back / compact the cache to the accepted path.
 *
 * Page 2 §3.3: after a partial acceptance the cache past the accepted
 * position is dropped; page 2 §5.4 and page 3 (tree section): a tree verify
 * rolls back along the accepted path.  The K/V of the root and of the a
 * accepted nodes are kept; for j = 1..a (increasing), the slot ctx+path[j]
 * is moved to slot ctx+j.  new_ctx_lens[b] = ctx_lens[b] + a + 1 (the drawn
 * token's K/V comes with the next step).  For a chain nothing moves.
 *
 *   k_cache, v_cache, block_table, ctx_lens  as in spec_verify_attn
 *   new_ctx_lens [B] int32   output; may alias ctx_lens
 *   path [B, M], accepted_len [B]  as produced by spec_reject_sample
 * Requests with accepted_len < 0, a bad path, or out-of-range block ids are
 * left unchanged (new length = old length) and flagged in the status word.
 */
spec_status kv_commit(void* k_cache, void* v_cache, const int32_t* block_table,
                      const int32_t* ctx_lens, int32_t* new_ctx_lens,
                      const int32_t* path, const int32_t* accepted_len,
                      const spec_dims* dims, void* ws, size_t ws_bytes,
                      void* stream);

/*
 * spec_reject_sample_noalloc -- spec_reject_sample for callers that cannot
 * allocate device memory.
 *
 * The pages have no counterpart to this call; it exists for callers that
 * cannot provide a workspace: cudaMalloc may synchronise the whole device,
 * is not allowed while a stream is being captured, and engines that hand all
 * of HBM to a fixed KV-cache pool at start-up often have no allocator to call.
 * Arguments, outputs and semantics are those of spec_reject_sample without
 * ws / ws_bytes.  The scratch (a status word; 16 bytes of row statistics per
 * request, row and 2048-logit chunk -- 1024 for fp32 logits; 8 bytes of
 * residual mass per request and chunk; an 816-byte draw state per
 * request) lives in a 1 MiB array inside the library that every GPU loading
 * the library holds until exit.
 *   - Sizes whose scratch exceeds that array (for bf16 logits, roughly
 *     B * ((32 * M + 8) * ceil(V / 2048) + 816) > 1 MiB)
 *     return SPEC_ERR_UNSUPPORTED and launch nothing; use
 *     spec_reject_sample there.
 *   - The first call in a CUDA context looks up the array's device address
 *     in that context (cudaGetSymbolAddress, once per context, with the
 *     context current) and keeps it; make that first call before any stream
 *     capture.  A new context on the same device (after cudaDeviceReset, or
 *     another context made current) gets its own lookup.
 *   - No memory is allocated or freed, by the library or any routine it
 *     calls.  The status word is cleared at the start of each call with an
 *     async memset on `stream`; device-side failures show as
 *     accepted_len = -1 for the request, and the status word is not readable
 *     through this call.
 *   - Every call shares the one array: calls whose work overlaps on the GPU
 *     (different streams, or different host threads on one device) race and
 *     must be serialised by the caller.
 *   - It does not update spec_last_launch_count.
 */
spec_status spec_reject_sample_noalloc(const void* target_logits,
                                       const void* draft_logits,
                                       const int32_t* tokens,
                                       const int32_t* parent,
                                       const float* temperature, uint64_t seed,
                                       uint64_t offset, uint64_t b_base,
                                       int32_t* out_tokens, int32_t* path,
                                       int32_t* accepted_len, float* probe,
                                       const spec_dims* dims, void* stream);

/*
 * spec_block_tables -- block tables, slot map and positions of a step's new
 * rows, from the requests' lengths.
 *
 * Page 2 §4.3 and page 3: the cache is paged and a block table maps a
 * request's positions to blocks; page 2 §3.3: what lies past the accepted
 * prefix is dropped.  One call before a step makes each request hold exactly
 * the pages that the step reads or writes: it takes pages for the new rows
 * from a ring of free block ids and returns the pages that a rollback
 * (kv_commit), a window that moved on, or the request's end left over.
 *
 *   ctx_lens  [B] int32   cached tokens; -1: the request has ended (or its
 *                         place is empty) and returns every page
 *   row_start [B+1] int32 or NULL   rows row_start[b] .. row_start[b+1]-1 are
 *                         request b's new rows (ascending, within [0, rows]);
 *                         NULL: M rows each, b*M .. b*M+M-1
 *   parent    [B, M] int32 or NULL   trees (only without row_start): positions
 *                         follow the nodes' depths; slots stay ctx + i
 *   rows                  rows of slots and positions (>= B*M without row_start)
 *   window, sinks         0, or the window and sinks of
 *                         spec_verify_attn_window, the same in every call:
 *                         only pages of the first `sinks` positions and of
 *                         positions from ctx - window + 1 on are held
 *   block_table [B, max_blocks] int32 (in/out)   entries of pages not held: -1
 *   span      [B, 2] int32 (in/out)   pages (lo, hi) held: p < hi
 *                         with p >= lo or among the sinks' pages; 0, 0 at first
 *   pool      [num_blocks] int32 (in/out)   ring of free ids
 *   pool_state [2] int32 (in/out)   head, count: entries (head + i) %
 *                         num_blocks, i < count, are free
 *   slots     [rows] int64    block * 16 + offset of each row, -1 without one
 *                         (NULL, like positions, if rows is 0)
 *   positions [rows] int32    position of each row, -1 without one
 *   ok        [B] int32 or NULL   1: the request may run this step
 *
 * Pages are taken from the ring's head and returned to its tail, both in
 * (request, page) order; returned pages are free from the next call on.  A
 * request gets its pages if the ring holds those that it and all requests
 * before it ask for; else it takes none (it still returns what it no longer
 * needs), its rows get -1, ok is 0 and SPEC_ERR_CAPACITY is raised.  Rows
 * behind the last request's are left as they are.  A request with a bad length
 * or topology (SPEC_ERR_INVALID_ARG), one that needs pages again that its
 * window has returned (SPEC_ERR_INVALID_ARG), one whose rows pass max_blocks
 * (SPEC_ERR_CAPACITY) or a bad span (SPEC_ERR_DEVICE_BOUNDS) is left
 * unchanged, with rows of -1 and ok 0.  A bad pool_state (SPEC_ERR_DEVICE_BOUNDS)
 * leaves every request unchanged, and so does a row_start that does not ascend
 * within [0, rows] (SPEC_ERR_INVALID_ARG; all of slots and positions are -1
 * then).  An entry of the table or the ring that is no block id raises
 * SPEC_ERR_DEVICE_BOUNDS when it is met and spreads to no other request: one that
 * takes it (the table then holds -1), or whose rows would be written to it, does
 * not run (rows of -1, ok 0; it keeps its pages), and returned to the ring are
 * block ids alone.
 * rows and B * max_blocks are at most 2^30.  Calls that share a page
 * state or a workspace must not overlap.
 */
spec_status spec_block_tables(const int32_t* ctx_lens, const int32_t* row_start,
                              const int32_t* parent, int32_t rows, int32_t window, int32_t sinks,
                              int32_t* block_table, int32_t* span, int32_t* pool,
                              int32_t* pool_state, int64_t* slots, int32_t* positions, int32_t* ok,
                              const spec_dims* dims, void* ws, size_t ws_bytes, void* stream);

/*
 * spec_qk_norm_rope -- RMS norm of every query and key head and the position
 * rotation in one pass; keys and values to the paged cache by slot.
 *
 * The queries and keys that spec_verify_attn takes, with their position
 * encoding applied.  A verify step passes no slots: spec_verify_attn appends the
 * new rows itself.  The cache is written here for rows that other attention
 * reads, a prompt's prefill for instance, as are the ragged rows of
 * spec_block_tables (the verify calls take M rows of every request, at most 128
 * per KV head).  For a head x at position t:
 *   y = x * rsqrt(mean(x^2) + eps) * weight       (no norm without a weight)
 *   (a, b) -> (a cos - b sin, b cos + a sin), angle t * inv_freq[j], for the
 *   pairs (j, j + rot_dim/2), or (2j, 2j + 1) if interleaved, j < rot_dim/2
 * in fp32 (angles reduced exactly), rounded once; elements past rot_dim do not
 * turn, and without a weight keep their bits.  Values of q and k that turn, or
 * that a norm is taken of, have to be finite.  rows = 0 does nothing.
 *
 *   q [rows, Hq, D], k, v [rows, Hkv, D]  kv_dtype   rows q_stride, k_stride,
 *                 v_stride elements apart (multiples of 16 bytes), heads dense:
 *                 views of one projection's output will do
 *   q_weight, k_weight [D] kv_dtype or NULL
 *   positions [rows] int32   -1: the row's outputs are zero and the caches
 *                 stay as they are
 *   inv_freq [rot_dim/2] double   rot_dim: a multiple of 16 up to D (0: no
 *                 rotation)
 *   q_out [rows, Hq, D], k_out [rows, Hkv, D]   dense; q_out may be q itself
 *                 and k_out k itself where those are dense
 *   slots [rows] int64 or NULL   with slots, the rotated key and the value of
 *                 each row also go to k_cache / v_cache ([num_blocks, Hkv, 16,
 *                 D]) at that slot; slots < 0 write nothing, slots past the
 *                 cache raise SPEC_ERR_DEVICE_BOUNDS and write nothing.  Slots
 *                 must differ from one another.  v, k_cache and v_cache are
 *                 needed with slots (k_out may then be NULL) and not read
 *                 without
 */
spec_status spec_qk_norm_rope(const void* q, const void* k, const void* v, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, const void* q_weight,
                              const void* k_weight, float eps, const int32_t* positions,
                              const double* inv_freq, int32_t rot_dim, int32_t interleaved,
                              int32_t rows, void* q_out, void* k_out, const int64_t* slots,
                              void* k_cache, void* v_cache, const spec_dims* dims, void* ws,
                              size_t ws_bytes, void* stream);

/*
 * spec_sample -- one token per logits row from given uniforms, with
 * temperature, top-k, top-p and min-p.
 *
 * The draft's own draws, and plain decoding (gamma 0, the fallback of
 * spec_ctrl_update).  Drafts have to be drawn by the law that the verify tests
 * them against: with the temperature alone for spec_reject_sample, with its
 * top_k and top_p for spec_reject_sample_filtered, and without min_p, which the
 * verify does not know (its outputs would not follow the target's law).  min_p
 * is for plain decoding.  The law of a row is softmax(x / T) (page 1 §3.3)
 * restricted as in spec_reject_sample_filtered (the first top_k tokens by
 * logit, the smaller index first among equal ones; of those the shortest
 * prefix whose mass reaches top_p times theirs) and then to the tokens of at
 * least min_p times the largest probability, renormalised; the token is the
 * smallest i with C_i > u * Z in vocabulary order.  T = 0 is greedy: the first
 * largest logit.
 *
 *   logits [rows, V] logits_dtype, rows row_stride elements apart (any
 *                 stride >= V, any alignment of the elements); -inf: never drawn
 *   temperature [rows] float   as in spec_reject_sample
 *   top_k [rows] int32 or NULL   >= 0 (0: off)
 *   top_p [rows] float or NULL   in (0, 1] (1: off)
 *   min_p [rows] float or NULL   in [0, 1] (0: off)
 *   uniform [rows] float         in [0, 1)
 *   out_tokens [rows] int32; out_prob [rows] float or NULL   the token and its
 *                 probability under the restricted law (1 when greedy)
 *   ws, ws_bytes  at least 16 bytes (its first word is the status word)
 * V up to 2^20.  A bad parameter (SPEC_ERR_INVALID_ARG) or a row with NaN,
 * +inf or only -inf (SPEC_ERR_NONFINITE) gives token -1 and probability 0.
 * Accuracy (T up to 2^100): a weight is held to 2^-28.9 of its value at worst and
 * 2^-31.5 on average; where the draw is among a row's few largest tokens also to
 * 2^-41 of the largest weight, the masses that top_p compares to 2^-41 or 2^-43
 * of it a token; sums add 2^-40.  So the token is the definition's unless u * Z
 * lies within 2^-28 * Z of a step, or a filter's cut that close to its target.
 * Without filters the Z of out_prob is off by up to 2^-20 of its value (about 2^-24
 * in practice), with them as above.
 * rows = 0 does nothing.  Of the workspace the
 * second word counts rows that needed a second look, modulo 2^32; its value
 * does not matter, and calls that overlap may share it.
 */
spec_status spec_sample(const void* logits, int64_t row_stride, int32_t rows, int32_t V,
                        int32_t logits_dtype, const float* temperature, const int32_t* top_k,
                        const float* top_p, const float* min_p, const float* uniform,
                        int32_t* out_tokens, float* out_prob, void* ws, size_t ws_bytes,
                        void* stream);

/*
 * Host-side controller and metrics (no GPU work; plain host memory).
 *
 * Page 3 ("推测解码的工程真相 2026"), dynamic scheduling and observability:
 * the acceptance rate of a request's last `window` verify steps sets its
 * next draft length (above high_acceptance: gamma_high; from
 * low_acceptance to high_acceptance: gamma_mid; below: gamma_low); a
 * temperature above hot_temperature sets gamma_hot at once; a request whose
 * speculation does not pay over a full window falls back to plain decoding
 * (gamma 0) and stays there.  Page 2 §5.1: log drafted and accepted counts
 * and where the rejections fall.
 *
 * Speculative efficiency is read as page 2 §2.3's speedup of a verify step:
 * emitted tokens per step (accepted + 1) / (1 + gamma * draft_cost); a
 * request below min_efficiency falls back.  Requests the device failed
 * (accepted_len = -1, e.g. SPEC_ERR_CAPACITY, the pages' fallback trigger)
 * fall back too.
 */
#define SPEC_CTRL_MAX_WINDOW 64
#define SPEC_CTRL_HIST_BINS 10
#define SPEC_STEP_MAX_POS 129

typedef struct spec_ctrl_config {
  int32_t window;          /* steps the acceptance rate is taken over (<= 64); 16 */
  float high_acceptance;   /* 0.6 */
  float low_acceptance;    /* 0.3 */
  int32_t gamma_high;      /* 8 */
  int32_t gamma_mid;       /* 4 */
  int32_t gamma_low;       /* 2 */
  float hot_temperature;   /* 0.8 */
  int32_t gamma_hot;       /* 1 */
  float draft_cost;        /* draft forward / target forward, 0.02 */
  float min_efficiency;    /* 1.0 */
  int32_t max_gamma;       /* cap on any draft length (<= 63) */
} spec_ctrl_config;

/* Per-request state, caller-owned (zeroed by spec_ctrl_init). */
typedef struct spec_ctrl_request {
  int16_t drafted[SPEC_CTRL_MAX_WINDOW];  /* ring of the last steps */
  int16_t accepted[SPEC_CTRL_MAX_WINDOW];
  int32_t head, steps;
  int32_t gamma;           /* draft length of the next step; 0 = plain decoding */
  int32_t fallback;        /* 1 once the request fell back */
  int32_t failed_steps;
} spec_ctrl_request;

typedef struct spec_ctrl_metrics_out {
  int32_t requests;
  int32_t acceptance_hist[SPEC_CTRL_HIST_BINS]; /* per-request window rates, 0.1-wide bins */
  float acceptance_mean, acceptance_p50, acceptance_p95, acceptance_p99;
  float emitted_per_step;
  float speculative_efficiency;
  float fallback_rate;
} spec_ctrl_metrics_out;

typedef struct spec_step_stats_out {
  int32_t requests, failed;
  int64_t accepted, emitted;
  int32_t rejection_pos[SPEC_STEP_MAX_POS];  /* 1-based draft position of the first
                                                rejection; index M: none rejected */
  float tree_width_effective;  /* mean share of the tree's root-to-leaf paths through
                                  the first accepted node (-1 for chains) */
} spec_step_stats_out;

void spec_ctrl_default_config(spec_ctrl_config* cfg);
spec_status spec_ctrl_init(spec_ctrl_request* reqs, int32_t n, int32_t gamma0);
/* Feed one verify step's accepted lengths (host copy of spec_reject_sample's
 * output; temperature may be NULL) and get each request's next draft length. */
spec_status spec_ctrl_update(const spec_ctrl_config* cfg, spec_ctrl_request* reqs, int32_t n,
                             const int32_t* accepted_len, const float* temperature,
                             int32_t* next_gamma);
spec_status spec_ctrl_metrics(const spec_ctrl_config* cfg, const spec_ctrl_request* reqs,
                              int32_t n, spec_ctrl_metrics_out* out);
/* Statistics of one verify step from host copies of its outputs: accepted
 * and emitted counts, the rejection-position histogram, and, for a tree
 * (parent != NULL), the tree width effective. */
spec_status spec_step_stats(const int32_t* accepted_len, const int32_t* path,
                            const int32_t* parent, int32_t B, int32_t M,
                            spec_step_stats_out* out);

/* Host-side Philox4x64-10 block (the generator the kernels use), for
 * known-answer tests: out = Philox4x64-10(counter, key). */
void spec_philox_block(const uint64_t key[2], const uint64_t counter[4],
                       uint64_t out[4]);

/* Human-readable name of a status code. */
const char* spec_status_string(int32_t status);

/* Number of kernel launches the last call on this thread enqueued. */
int32_t spec_last_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */

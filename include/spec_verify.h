/*
 * spec_verify.h — C ABI of the speculative-decoding verification library
 * (libspecverify.so, sm_103a).
 *
 * One call verifies the draft tokens of B requests against the target model's
 * logits on the caller's CUDA stream.  Sources of each operation:
 *
 *   chain verify   vLLM anatomy page ("Inside vLLM", part 3), section
 *                  "Speculative Decoding": accept/reject left to right, stop
 *                  at the first rejection, sample the rebalanced distribution
 *                  max(0, p_large - p_draft) normalised, or the bonus token
 *                  from the extra row when all k drafts are accepted.  The
 *                  vLLM learning book, section 2 (Leviathan 2023 flowchart),
 *                  gives the test r < min(1, p(x_i)/q(x_i)).  The TensorRT-LLM
 *                  walkthrough (part 10), rejection-sampling section, fixes the
 *                  shapes draft [batch, D, vocab], target [batch, D+1, vocab]
 *                  and the output accepted_tokens [batch, D+1] padded with -1.
 *   greedy verify  Kestrel article 32, section 3.3: accept while the target's
 *                  argmax equals the draft; the emitted stream is the target's
 *                  own argmax chain.  TensorRT-LLM walkthrough, rejection-
 *                  sampling section: an all-greedy batch takes the base path.
 *   tree verify    TensorRT-LLM deployment page ("05-TensorRT-LLM 推测解码"),
 *                  section "Eagle-2 多层级树状草稿生成": paths tensor
 *                  [batch, max_decoding_tokens, max_path_len].
 *   rollback       TensorRT-LLM walkthrough, update_requests section
 *                  (py_rewind_len = verified_len - accepted) and the paged
 *                  rewind_cache section (only the logical length moves; rows
 *                  are not cleared).  Kestrel article 32, section 3.1
 *                  (truncate = move the cursor, copy nothing).
 *
 * Conventions for every call
 *   - All array pointers are DEVICE pointers owned by the caller; the library
 *     never allocates or frees memory.  It keeps no global state apart from
 *     the fixed scratch array of spec_verify_chain_noalloc.  Arrays are
 *     dense, row-major, with the shapes given below.
 *   - Calls are asynchronous on `stream` (NULL = the legacy default stream).
 *     A host-detectable error (bad size, null pointer, small workspace)
 *     returns before any launch and writes nothing.  A failed launch returns
 *     SPEC_ECUDA.
 *   - Data-dependent errors (a token or node id out of range) do not stop the
 *     call: the affected request fails closed (its num_accepted is -1, its
 *     token row is all -1, its seq_len is left unchanged) and the status word
 *     in the workspace records SPEC_EBADINDEX; read it with spec_last_error().
 *   - Logits must be finite or -inf (masked), with at least one finite value
 *     per row; NaN and +inf are outside the contract and are not checked.
 *   - One workspace serves one stream at a time: calls that overlap on the GPU
 *     must not share a workspace.
 *   - The second phase of a verify waits (bounded, about one second) for
 *     words the first phase publishes.  A wait that runs out records
 *     SPEC_ETIMEOUT in the status word and fails the requests that depended
 *     on it closed, as above; it cannot happen unless the GPU is broken or
 *     another kernel starves the call.
 *   - Every call leaves its workspace ready for the next.  After a call that
 *     returned SPEC_ECUDA, or whose status word reads SPEC_ETIMEOUT, zero the
 *     workspace again with spec_workspace_init before reusing it.
 *   - Calls run on the device that is current for the calling thread; the
 *     arrays and the stream must belong to it.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
struct CUstream_st;
typedef struct CUstream_st *spec_stream_t;

typedef enum {
    SPEC_OK = 0,
    SPEC_EINVAL = -1,      /* bad size, dtype, temperature or null pointer; arrays that
                              overlap where a call checks them */
    SPEC_EBADINDEX = -2,   /* a token or node id was out of range (device status) */
    SPEC_ECUDA = -3,       /* a CUDA launch or copy failed */
    SPEC_EWORKSPACE = -4,  /* workspace missing or smaller than spec_workspace_size() */
    SPEC_ETIMEOUT = -5,    /* a bounded device wait ran out (device status) */
    SPEC_ELIMIT = -6       /* a filtered row's cut search found its bins inconsistent
                              (an internal check, not expected; device status) */
} spec_status_t;

/* SPEC_F16: the KV cache calls only (logits are fp32 or bf16). */
typedef enum { SPEC_F32 = 0, SPEC_BF16 = 1, SPEC_F16 = 2 } spec_dtype_t;

/* Largest supported draft length k of a chain call, and the largest tree
 * (N nodes, L path length) of a tree call. */
#define SPEC_MAX_DRAFT 64
/* Largest batch B of any call. */
#define SPEC_MAX_BATCH 8192
/* Largest top_k the filtered chain verify serves with explicit kept lists;
 * a larger top_k (and top-p or min_p without top-k) takes per-row cuts. */
#define SPEC_MAX_TOPK 256
#define SPEC_MAX_TREE_NODES 1024
#define SPEC_MAX_PATH_LEN 64

/* Bytes of scratch one call needs for B requests of `rows_per_request` logit
 * rows of width V (chain: 2k+1, greedy: k+1, tree: N).  Returns 0 for invalid
 * sizes.  The same workspace may be reused by any call whose own size is not
 * larger.  Every workspace starts with a fixed 512 KB block of per-request
 * sync lines (SPEC_MAX_BATCH of them). */
size_t spec_workspace_size(int B, int rows_per_request, int V);

/* Bytes of scratch of a filtered chain verify (spec_chain_params with
 * top_k > 0, or top_k = 0 with top_p < 1 or min_p > 0) of B requests, k
 * drafts, width V: the chain's, plus for 1 <= top_k <= SPEC_MAX_TOPK each
 * row's kept list (top_k words), 2k probabilities per request and two bytes
 * per 2048 logits of each row; for top_k = 0 or top_k > SPEC_MAX_TOPK
 * (per-row cuts) each row's 2048-bin mass histogram and counts (24 KB), a
 * 64-byte record and a 4096-entry candidate list (16 KB).  Returns 0 for
 * invalid sizes (top_k < 0 included). */
size_t spec_workspace_size_filtered(int B, int k, int V, int top_k);

/* Zero a workspace (asynchronously, on `stream`).  Call once after allocating
 * it; every verify call leaves it ready for the next. */
int spec_workspace_init(void *workspace, size_t workspace_bytes, spec_stream_t stream);

/* Chain rejection-sampling verify.
 *   target_logits  [B, k+1, V] of `dtype`: row i (i < k) is the target
 *                  distribution of draft position i, row k the bonus row.
 *   draft_logits   [B, k, V] of `dtype`: row i is the draft distribution
 *                  that draft token i was sampled from.
 *   draft_tokens   [B, k] int32 in [0, V).
 *   uniforms       [B, k+1] float32 in [0, 1): column i < k is the accept
 *                  test of position i, column k drives the final sample.
 *   temperature    > 0 and finite; both rows are softmax(logits / T).
 * Accepts x_i while uniforms[b,i] < p_i(x_i) / q_i(x_i) (q == 0 accepts).
 * At the first rejection j the last token is drawn from max(0, p_j - q_j)
 * normalised; when all k are accepted it is drawn from p_k.  The draw takes
 * the smallest t whose cumulative weight exceeds uniforms[b,k] times the
 * total.
 *   out_tokens       [B, k+1] int32: x_0..x_{n-1}, the final token, -1 pad.
 *   out_num_accepted [B] int32: n in [0, k] (-1 for a failed request).
 *   out_probs        [B, k, 2] float32 or NULL: p_i(x_i), q_i(x_i) for every i.
 *   seq_lens         [B] int32 or NULL: KV cursor, updated in place to
 *                    seq_len + n + 1 (see spec_rollback_lengths).
 * Probabilities are accumulated in fp32. */
int spec_verify_chain(const void *target_logits, const void *draft_logits, int dtype,
                      const int32_t *draft_tokens, const float *uniforms, float temperature,
                      int B, int k, int V,
                      int32_t *out_tokens, int32_t *out_num_accepted, float *out_probs,
                      int32_t *seq_lens,
                      void *workspace, size_t workspace_bytes, spec_stream_t stream);

/* Chain verify with each request's uniforms drawn inside the kernel from a
 * per-request Philox state (TensorRT-LLM walkthrough, rejection-sampling
 * section: chain_speculative_sampling takes a seed and an offset per request,
 * the offset keeping each request's stream apart so that the seed can stay
 * constant).  Arguments and results are those of spec_verify_chain, with
 *   seeds    [B] uint64: Philox4x32-10 key (low word first);
 *   offsets  [B] uint64: counter, advanced by the caller between steps;
 * in place of uniforms.  Uniform i of request b (i = 0..k; i < k are the
 * accept tests, i = k drives the final draw) is word i % 4 of
 * Philox4x32-10(counter = (low word of offset, high word of offset, i / 4, 0),
 * key = seed) (Salmon et al., SC'11), shifted right by 8 and scaled by 2^-24.
 * The pages fix the state, not this mapping: it is this library's reading. */
int spec_verify_chain_philox(const void *target_logits, const void *draft_logits, int dtype,
                             const int32_t *draft_tokens, const uint64_t *seeds,
                             const uint64_t *offsets, float temperature, int B, int k, int V,
                             int32_t *out_tokens, int32_t *out_num_accepted, float *out_probs,
                             int32_t *seq_lens, void *workspace, size_t workspace_bytes,
                             spec_stream_t stream);

/* Parameters of spec_verify_chain_ex: those of spec_verify_chain and
 * spec_verify_chain_philox in one struct, plus ragged draft lengths and
 * top-k / top-p filtering.  Set size = sizeof(spec_chain_params); fields a
 * later version adds go at the end, and a smaller size (an earlier version
 * of the struct, ending at seq_lens) leaves the added fields at their
 * defaults (no filtering).
 *   draft_lens [B] int32 or NULL: request b has k_b <= k real drafts in the
 *     buffers padded to k (TensorRT-LLM walkthrough: the real draft count is
 *     kept apart from the padded buffer, pad_draft_tokens_for_cuda_graph; the
 *     verified window is per request, verify_lens).  It is verified as a chain
 *     of k_b: accept tests on positions 0..k_b-1, the final draw uses uniform
 *     column (or Philox index) k_b and target row k_b is its bonus row.  Rows
 *     past k_b are not read (pass 1 skips them) and their draft tokens are not
 *     checked; out_probs there is NaN.  A length outside [0, k] fails the
 *     request closed (SPEC_EBADINDEX in the status word).
 *   uniforms or (seeds, offsets): exactly as in the two calls above; when
 *     uniforms is NULL both seeds and offsets are required. */
typedef struct spec_chain_params {
    size_t size;
    const void *target_logits;  /* [B, k+1, V] */
    const void *draft_logits;   /* [B, k, V] */
    int dtype;
    const int32_t *draft_tokens; /* [B, k] */
    const int32_t *draft_lens;   /* [B] or NULL */
    const float *uniforms;       /* [B, k+1] or NULL */
    const uint64_t *seeds;       /* [B] when uniforms is NULL */
    const uint64_t *offsets;     /* [B] when uniforms is NULL */
    float temperature;
    int B, k, V;
    int32_t *out_tokens;         /* [B, k+1] */
    int32_t *out_num_accepted;   /* [B] */
    float *out_probs;            /* [B, k, 2] or NULL */
    int32_t *seq_lens;           /* [B] or NULL */
    /* Symmetric filtering (TensorRT-LLM walkthrough, rejection-sampling
     * section: target and draft are filtered by the same backend and
     * parameters, or the accept test is silently wrong).  top_k = 0: none.
     * top_k >= 1: every target and draft row keeps its top_k tokens by
     * (logit descending, token ascending) (top_k >= V: all), then the
     * shortest prefix of them whose softmax mass (over those top_k, at
     * temperature T) reaches top_p (top_p = 1: all top_k); p and q are the
     * softmax over the kept set, and the chain verify above runs on them
     * (the final draw takes u * Z over the kept tokens in token order).
     * out_probs holds the filtered p and q.  Logits of -inf carry weight 0
     * (they change no probability, no top-p prefix and no draw); logits must
     * not be NaN or +inf.  top_p in (0, 1].  top_k = 0 with top_p < 1 keeps
     * the shortest prefix of the whole row whose mass reaches top_p.  Kept
     * sets of any size are exact: 1 <= top_k <= SPEC_MAX_TOPK uses explicit
     * kept lists, top_k = 0 (with top_p < 1 or min_p > 0) and top_k >
     * SPEC_MAX_TOPK a per-row cut found from a mass histogram and a radix
     * selection over the tokens of the bins the cut can fall in.  The
     * workspace must hold spec_workspace_size_filtered(B, k, V, top_k)
     * bytes. */
    int top_k;
    float top_p;
    /* min_p in [0, 1] (0: off), applied after top-p (the walkthrough names
     * temperature, top-k, top-p and min_p in that order): a token of the
     * kept set stays when its probability is at least min_p times the
     * largest, 2^((x - x_max) log2(e) / T) >= min_p.  A struct ending at
     * top_p leaves it at 0. */
    float min_p;
} spec_chain_params;
int spec_verify_chain_ex(const spec_chain_params *params, void *workspace,
                         size_t workspace_bytes, spec_stream_t stream);

/* Parameters of spec_verify_greedy_ex: spec_verify_greedy's plus ragged
 * draft lengths (as in spec_chain_params: a request with k_b drafts is
 * greedy-verified over positions 0..k_b-1 and its bonus token is the argmax
 * of target row k_b; rows past k_b are not read). */
typedef struct spec_greedy_params {
    size_t size;
    const void *target_logits;   /* [B, k+1, V] */
    int dtype;
    const int32_t *draft_tokens; /* [B, k] */
    const int32_t *draft_lens;   /* [B] or NULL */
    int B, k, V;
    int32_t *out_tokens;         /* [B, k+1] */
    int32_t *out_num_accepted;   /* [B] */
    int32_t *seq_lens;           /* [B] or NULL */
} spec_greedy_params;
int spec_verify_greedy_ex(const spec_greedy_params *params, void *workspace,
                          size_t workspace_bytes, spec_stream_t stream);

/* Rollback with ragged draft lengths and paged block accounting
 * (TensorRT-LLM walkthrough: update_requests sets rewind = verified_len -
 * accepted; rewind_cache recomputes the blocks needed from tokens_per_block
 * and returns only whole surplus blocks, clearing nothing).
 *   k_b = draft_lens[b] (or k when NULL); new_lens = old_lens + n + 1;
 *   rewind_lens (nullable) = k_b - n; free_blocks (nullable) = max(0,
 *   blocks_held[b] - ceil(new_len / tokens_per_block)), 0 when blocks_held is
 *   NULL.  new_lens may alias old_lens.  An entry with k_b outside [0, k] or
 *   n outside [0, k_b] (a failed request reads n = -1) keeps its length; its
 *   rewind reads -1 and its free count 0. */
int spec_rollback_paged(const int32_t *old_lens, const int32_t *num_accepted,
                        const int32_t *draft_lens, int k, const int32_t *blocks_held,
                        int tokens_per_block, int B, int32_t *new_lens, int32_t *rewind_lens,
                        int32_t *free_blocks, spec_stream_t stream);

/* The uniforms spec_verify_chain_philox draws: out[b, i] for i = 0..n-1
 * (n <= SPEC_MAX_DRAFT + 1), from the same per-request Philox streams, so a
 * caller can log or replay a step's randomness. */
int spec_philox_uniforms(const uint64_t *seeds, const uint64_t *offsets, int B, int n,
                         float *out, spec_stream_t stream);

/* Greedy chain verify.
 *   target_logits [B, k+1, V], draft_tokens [B, k] in [0, V).
 * g_i = argmax_t target[b,i,t] on the stored values, lowest id on ties;
 * n = the longest prefix with g_i == d_i; out_tokens [B, k+1] =
 * d_0..d_{n-1}, g_n, -1 pad; out_num_accepted [B]; seq_lens as above. */
int spec_verify_greedy(const void *target_logits, int dtype, const int32_t *draft_tokens,
                       int B, int k, int V,
                       int32_t *out_tokens, int32_t *out_num_accepted, int32_t *seq_lens,
                       void *workspace, size_t workspace_bytes, spec_stream_t stream);

/* Greedy tree verify over EAGLE-style paths.
 *   target_logits [B, N, V]: row n is the target distribution after node n;
 *                 node 0 is the root (the last committed token).
 *   tree_tokens   [B, N] int32 in [0, V): node n's token.
 *   paths         [B, P, L] int32 in [-1, N): root-to-leaf node lists padded
 *                 with -1; a used path starts with 0, an unused one with -1.
 * For every used path, step j = 1..L-1 is accepted while its node is >= 0 and
 * its token equals argmax of its parent's row; the path with the most
 * accepted steps wins (lowest path index on ties).
 *   out_tokens         [B, L] int32: accepted tokens, then argmax of the last
 *                      accepted node's row, -1 pad.
 *   out_num_accepted   [B] int32 (-1 for a failed request).
 *   out_best_path      [B] int32 or NULL (-1 when no path is used).
 *   out_accepted_nodes [B, L] int32 or NULL: the root and the accepted node
 *                      ids (the KV rows to keep), -1 pad.
 *   seq_lens           [B] int32 or NULL, updated to seq_len + n + 1. */
int spec_verify_tree(const void *target_logits, int dtype, const int32_t *tree_tokens,
                     const int32_t *paths, int B, int N, int P, int L, int V,
                     int32_t *out_tokens, int32_t *out_num_accepted, int32_t *out_best_path,
                     int32_t *out_accepted_nodes, int32_t *seq_lens,
                     void *workspace, size_t workspace_bytes, spec_stream_t stream);

/* Stochastic tree verify (TensorRT-LLM deployment page, "目标模型验证：树注意力
 * 与批量并行": the tree's tokens are judged against the target logits by
 * rejection sampling; children are chosen by top-K per level, "Eagle-2
 * 多层级树状草稿生成").  A chosen child is a point-mass proposal on its token,
 * so the rejection-sampling rule becomes: at each node, try its children in
 * increasing node id; accept child c iff uniforms[b, c] < p'(token of c), the
 * current residual of the node's softmax(row / T); on a rejection remove that
 * token from the residual and renormalise; when no child is accepted (or the
 * node has none, or L - 1 steps were taken) draw the final token from the
 * residual by inverse CDF at uniforms[b, 0] (from the node's own row if the
 * residual's mass vanished).  The emitted tokens follow the target rows.
 *   target_logits [B, N, V], tree_tokens [B, N], paths [B, P, L]: as for
 *                 spec_verify_tree; a node's children are the entries d + 1
 *                 of the used paths whose first d + 1 entries are the
 *                 accepted prefix.  P * L <= 4096.
 *   uniforms      [B, N] float32 in [0, 1): column n >= 1 is node n's accept
 *                 test, column 0 drives the final draw.
 *   temperature   > 0 and finite.
 *   Outputs as for spec_verify_tree: tokens [B, L] (accepted tokens, the
 *   final token, -1 pad), num_accepted [B], best_path [B] (the lowest used
 *   path holding the accepted nodes, -1 when none), accepted_nodes [B, L];
 *   seq_lens advanced by n + 1.  Workspace: spec_workspace_size(B, N, V). */
int spec_verify_tree_sampled(const void *target_logits, int dtype, const int32_t *tree_tokens,
                             const int32_t *paths, const float *uniforms, float temperature,
                             int B, int N, int P, int L, int V,
                             int32_t *out_tokens, int32_t *out_num_accepted,
                             int32_t *out_best_path, int32_t *out_accepted_nodes,
                             int32_t *seq_lens, void *workspace, size_t workspace_bytes,
                             spec_stream_t stream);

/* KV cursor rollback as length arithmetic only (no KV row is copied or
 * cleared; rows past the new length become invisible and are overwritten
 * later).
 *   old_lens [B]: cursor before the verify window was written.
 *   num_accepted [B]: n per request; k = draft rows in the verify window
 *   (chain: k; tree: N - 1).
 *   new_lens [B] = old_lens + n + 1 (may alias old_lens);
 *   rewind_lens [B] or NULL = k - n (rows written but not kept).
 * An entry with n outside [0, k] (a failed request reads n = -1) keeps its
 * length and its rewind reads -1, so a caller can tell it from a valid
 * rewind (>= 0); the call itself returns SPEC_OK. */
int spec_rollback_lengths(const int32_t *old_lens, const int32_t *num_accepted, int k, int B,
                          int32_t *new_lens, int32_t *rewind_lens, spec_stream_t stream);

/* Accepted-KV relocation after a tree verify (TensorRT-LLM walkthrough, the
 * "moving to the right place" step before update_resources,
 * _update_kv_cache_draft_token_location): the KV rows of the accepted nodes,
 * written in tree order during the draft step, are gathered into consecutive
 * logical positions right after the committed prefix.  As on that page the
 * cache is paged.
 *   kv_pool        [num_blocks * tokens_per_block, row_bytes] device memory,
 *                  16-byte aligned; one row per token (one layer's K and V
 *                  of every KV head, or however the caller lays a token out).
 *                  row_bytes must be a multiple of 16.
 *   block_tables   [B, max_blocks] int32: request b's logical position t is
 *                  pool row block_tables[b][t / tokens_per_block] *
 *                  tokens_per_block + t % tokens_per_block.  Blocks holding
 *                  the window must not be shared between requests.
 *   base_lens      [B] int32: logical position of tree node 0 (the committed
 *                  length before the verify window).
 *   accepted_nodes [B, L] int32 and num_accepted [B]: spec_verify_tree's
 *                  outputs (root, then the n accepted nodes; -1 padded).
 * For j = 1..n, row base + accepted_nodes[b][j] moves to row base + j; rows
 * past base + n are left as they are (the rollback makes them invisible).
 * A request is left untouched when n <= 0 or n >= L (failed closed), or when
 * its path does not start at node 0 with strictly increasing nodes, or a row
 * it would read or write is unmapped (a block id outside [0, num_blocks) or
 * a position past max_blocks * tokens_per_block); no status is recorded.
 * Returns SPEC_EINVAL for null pointers, sizes outside the limits or a
 * misaligned pool. */
int spec_relocate_accepted_kv(void *kv_pool, size_t row_bytes, int tokens_per_block,
                              int num_blocks, const int32_t *block_tables, int max_blocks,
                              const int32_t *base_lens, const int32_t *accepted_nodes,
                              const int32_t *num_accepted, int B, int L, spec_stream_t stream);

/* Chain verify without a caller-provided workspace, for callers that cannot
 * allocate device memory (code whose allocator forbids allocations while a
 * step runs, or host code that owns no CUDA allocator).  The pages have no
 * counterpart: it is an addition of this library.
 *   Arguments and results are those of spec_verify_chain; inputs and outputs
 *   are still the caller's device arrays.
 *   Scratch: a file-scope device array of SPEC_NOALLOC_SCRATCH_BYTES that
 *   every GPU loading the library holds until the process exits.  A problem
 *   whose spec_workspace_size(B, 2k+1, V) exceeds it returns SPEC_EWORKSPACE
 *   before any launch.
 *   Every call on a device shares the one array: calls that can overlap on the
 *   GPU (other streams, other threads) race and must be serialised by the
 *   caller.  Each call clears the array's counters and status word on
 *   `stream` before launching, so there is no status word to read: the only
 *   data-dependent signal is a request that fails closed (num_accepted ==
 *   -1, tokens -1, seq_len unchanged), whether for a bad draft token or for
 *   a device wait that ran out.
 *   The arrays must be device (or managed) memory of the current device:
 *   the array used as scratch is the current device's.  Every argument is
 *   checked before the array is written; a refused call (SPEC_EINVAL,
 *   SPEC_EWORKSPACE) leaves it untouched.  Each call looks up the array's
 *   device address (cudaGetSymbolAddress) with its device current, so no
 *   call needs a set-up step first.
 * Allocates nothing: no cudaMalloc, cudaFree or allocating library call. */
#define SPEC_NOALLOC_SCRATCH_BYTES (4u << 20)
int spec_verify_chain_noalloc(const void *target_logits, const void *draft_logits, int dtype,
                              const int32_t *draft_tokens, const float *uniforms,
                              float temperature, int B, int k, int V,
                              int32_t *out_tokens, int32_t *out_num_accepted, float *out_probs,
                              int32_t *seq_lens, spec_stream_t stream);

/* Fault injection for tests of the bounded device waits (no counterpart on
 * the pages).  Each runs its call with the first phase left out, so that the
 * words the second phase waits for are never written, and with every device
 * wait bounded by wait_cycles SM clock cycles (>= 1) instead of about one
 * second.  Arguments are those of spec_verify_chain_ex (plain or filtered
 * with kept lists; a filtered call whose rows are wider than one CTA's codes
 * has no wait and returns SPEC_ECUDA, and the per-row-cut filter (top_k = 0
 * with top_p < 1 or min_p > 0, or top_k > SPEC_MAX_TOPK) waits for nothing
 * and returns SPEC_EINVAL) / spec_verify_greedy_ex.  Expected outcome: every
 * request fails closed and the status word reads SPEC_ETIMEOUT.  The
 * workspace may hold stale words afterwards: zero it with
 * spec_workspace_init before its next use. */
int spec_test_timeout_chain(const spec_chain_params *params, long long wait_cycles,
                            void *workspace, size_t workspace_bytes, spec_stream_t stream);
int spec_test_timeout_greedy(const spec_greedy_params *params, long long wait_cycles,
                             void *workspace, size_t workspace_bytes, spec_stream_t stream);

/* ------------------------------------------------------------------------
 * The 8-bit paged KV cache a verify step runs on: blocks taken and given
 * back, the tree's ancestor masks, the quantising store, attention, and the
 * relocation of accepted rows.  None of these calls uses a workspace or
 * records a status; each says below how a request with bad lengths or block
 * ids shows.
 *
 * A window is the run of tokens a step puts behind a request's committed
 * prefix: seq_lens[b] is the prefix length (the cursor before the window is
 * written), and token i of the window sits at logical position
 * seq_lens[b] + i.  Arrays are padded to W tokens per request;
 * window_lens [B] (NULL: every request has W) gives the real count w_b in
 * [0, W].  Padded rows are neither read nor written.
 * ---------------------------------------------------------------------- */

/* Largest W of a call. */
#define SPEC_MAX_WINDOW 65536

/* Blocks for the windows of a step, block tables and slot maps.
 *   block_tables [B, max_blocks] and blocks_held [B], updated in place: the
 *     first blocks_held[b] entries of a row are the request's blocks.
 *   free_blocks [num_blocks] with free_count [1]: a stack of free block ids,
 *     free_blocks[free_count - 1] on top; free_count is updated in place,
 *     free_blocks is not written.
 * Request b needs max(0, ceil((seq_lens[b] + w_b) / tokens_per_block) -
 * blocks_held[b]) more blocks.  They come off the stack in request order
 * (request 0's first block is the top), up to the first request that the
 * stack cannot serve: it and every later request that needs a block get
 * none.
 *   granted [B]: w_b, or -1 for a request that got none of the blocks it
 *     needs or whose entries are out of range (seq_lens < 0, w_b outside
 *     [0, W], blocks_held outside [0, max_blocks], or more than max_blocks
 *     blocks in all): its row and count are left as they are.  free_count
 *     outside [0, num_blocks] grants no block.
 *   slots [B, W] or NULL: the pool row block * tokens_per_block + offset of
 *     each window token; -1 where padded, not granted, or in a block whose
 *     id lies outside [0, num_blocks).  num_blocks * tokens_per_block must
 *     then be below 2^31. */
int spec_reserve_blocks(const int32_t *seq_lens, const int32_t *window_lens, int W,
                        int tokens_per_block, int B, int32_t *block_tables, int max_blocks,
                        int32_t *blocks_held, const int32_t *free_blocks, int num_blocks,
                        int32_t *free_count, int32_t *slots, int32_t *granted,
                        spec_stream_t stream);

/* Gives back the last counts[b] blocks of every request (the counts of
 * spec_rollback_paged): they go on the free stack, their table entries read
 * -1 and blocks_held drops.  The order on the stack is the one they came off
 * in, so releasing what spec_reserve_blocks has just granted restores the
 * stack.  A request whose count lies outside [0, blocks_held[b]] or whose
 * blocks_held lies outside [0, max_blocks] gives back nothing; when the
 * stack cannot hold what is given back (or free_count is out of range) the
 * call changes nothing. */
int spec_release_blocks(const int32_t *counts, int B, int32_t *block_tables, int max_blocks,
                        int32_t *blocks_held, int32_t *free_blocks, int num_blocks,
                        int32_t *free_count, spec_stream_t stream);

/* Ancestor masks of a tree: bit m % 32 of masks[b, n, m / 32] is set when
 * node m is node n itself or precedes it on a used path (paths as in
 * spec_verify_tree; entries after a path's first -1 are ignored).  A node on
 * no used path has an empty row; a request with a node id >= N on a used
 * path has only empty rows (spec_verify_tree fails it closed).
 *   paths [B, P, L], masks [B, N, ceil(N / 32)] int32. */
int spec_tree_masks(const int32_t *paths, int B, int P, int L, int N, int32_t *masks,
                    spec_stream_t stream);

/* A paged KV cache in 8 bits (e4m3) with one scale per block of tokens, K or
 * V, and head.
 *   pool   [num_blocks, 2, kv_heads, tokens_per_block, head_dim] e4m3 bytes,
 *          32-byte aligned (index 0 of the second axis: K, 1: V);
 *   scales [num_blocks, 2, kv_heads] float32: an element is its e4m3 value
 *          times the scale.  Scales are finite and >= 0; spec_store_kv makes
 *          powers of two (0 for a block of zeros).
 *   block_tables [B, max_blocks]: as for spec_relocate_accepted_kv.
 * tokens_per_block is a multiple of 16 up to 1024, head_dim 64 or 128,
 * kv_heads at most 1024.  Set size = sizeof(spec_kv_cache). */
typedef struct spec_kv_cache {
    size_t size;
    void *pool;
    float *scales;
    const int32_t *block_tables;
    int num_blocks, max_blocks, tokens_per_block, kv_heads, head_dim;
} spec_kv_cache;

/* Writes a window's K and V rows into the cache.
 *   k, v  [B, W, kv_heads, head_dim] of `dtype` (SPEC_BF16 or SPEC_F16),
 *         element (b, i, h, d) at b * strides[0] + i * strides[1] +
 *         h * strides[2] + d (strides in elements, multiples of 8, bases
 *         16-byte aligned), so slices of a fused projection need no copy.
 * Storing appends: the rows of a block before the first one written stay
 * live, everything behind the window is dead.  For each block, kind and head
 * the scale becomes the least power of two s (at least 2^-126) with
 * |x| <= 448 s for every finite new element x, or the block's old scale if
 * it has live rows and its scale is larger; where a block with live rows
 * gets a larger scale, their codes are rounded again, q' = rne(q old / new).
 * A new element is stored as rne(x / s), rounded to the nearest e4m3 value,
 * ties to even; an element that is not finite is stored as NaN.
 * A request with seq_lens < 0, w_b outside [0, W], a window past max_blocks
 * blocks, or a window block id outside [0, num_blocks) stores nothing.
 * Blocks holding a window must not be shared between requests, nor stand
 * twice in a request's row. */
int spec_store_kv(const spec_kv_cache *cache, const void *k, const int64_t *k_strides,
                  const void *v, const int64_t *v_strides, int dtype, const int32_t *seq_lens,
                  const int32_t *window_lens, int B, int W, spec_stream_t stream);

/* Attention of each window token over its request's cached prefix and the
 * window (whose rows spec_store_kv has written).
 *   q     [B, W, q_heads, head_dim] of `dtype` (SPEC_BF16 or SPEC_F16),
 *         strided as in spec_store_kv; q_heads is a multiple of kv_heads and
 *         head h reads KV head h / (q_heads / kv_heads).
 *   masks [B, W, ceil(W / 32)] int32 or NULL (W <= SPEC_MAX_TREE_NODES):
 *         window token i sees window token j when bit j % 32 of word j / 32
 *         of its row is set (spec_tree_masks).  NULL: the chain, j <= i.
 *         Every prefix position is seen.
 *   out = sum_t p_t v_t with p = softmax over the seen positions t of
 *   scale * q . k_t; lse = log sum exp of those scores (natural log).  A
 *   token that sees nothing gets out = 0 and lse = -inf.  Positions that a
 *   token does not see have no influence on it, whatever they hold (NaN and
 *   scales of any size included).
 *   out     [B, W, q_heads, head_dim] of `dtype`, dense.
 *   out_lse [B, W, q_heads] float32 or NULL.
 * The rows of a request with seq_lens < 0, w_b outside [0, W] (all W rows),
 * a window past max_blocks blocks, or a block id outside [0, num_blocks)
 * among those it reads are NaN.  Scores and sums are held in fp32; scores
 * stay below 2^26 in magnitude.  The weights, times the V scales of their
 * blocks, are rounded to fp16 before they meet V's codes: to 11 bits, in steps
 * of at least 2^-32 of the largest such product among the positions that the
 * token sees.
 *   scratch: spec_attend_scratch_size(...) bytes, 256-byte aligned, used
 *   during the call only; it need not be initialised and may hold anything,
 *   but calls that overlap on the GPU must not share it, and it must not be
 *   the workspace of a verify call.  Results do not depend on timing: equal
 *   inputs give equal bits.
 * Limits: max_blocks * tokens_per_block and B * W * q_heads at most 2^30. */
typedef struct spec_attend_params {
    size_t size;
    const void *q;
    int64_t q_strides[3];
    int dtype;
    int B, W, q_heads;
    const int32_t *seq_lens;
    const int32_t *window_lens;  /* [B] or NULL */
    const int32_t *masks;        /* or NULL */
    float scale;                 /* finite, times log2(e) too */
    void *out;
    float *out_lse;              /* or NULL */
} spec_attend_params;
int spec_attend_kv(const spec_kv_cache *cache, const spec_attend_params *params, void *scratch,
                   size_t scratch_bytes, spec_stream_t stream);

/* Scratch of spec_attend_kv for B requests of W window tokens (0 for invalid
 * sizes). */
size_t spec_attend_scratch_size(int B, int W, int q_heads, int kv_heads, int head_dim);

/* spec_relocate_accepted_kv for the 8-bit cache: for j = 1..n the K and V
 * rows of node accepted_nodes[b][j] move to logical position base + j, with
 * the same rules for which requests are left untouched.  A block written to
 * gets, per kind and head, the largest scale among the rows that it
 * receives, and its own old scale if rows before the first one written stay
 * live (as in spec_store_kv); codes whose scale grows are rounded again.
 * Rows past base + n are dead. */
int spec_relocate_quantised_kv(const spec_kv_cache *cache, const int32_t *base_lens,
                               const int32_t *accepted_nodes, const int32_t *num_accepted, int B,
                               int L, spec_stream_t stream);

/* ------------------------------------------------------------------------
 * What a step needs around the verify and the cache: the target's logits
 * penalised, biased and masked before the verify, queries and keys rotated to
 * their positions before the store and the attention, and the positions of
 * least attention dropped from a cache that has grown to its budget.  None of
 * these calls uses a workspace or records a status.  Results do not depend on
 * timing: equal inputs give equal bits.
 * ---------------------------------------------------------------------- */

/* Most entries of a request's bias list. */
#define SPEC_MAX_BIAS 1024

/* Penalties for repeated tokens, biases and grammar masks on the logits of a
 * window's rows, for the verify calls to read.
 *   logits, out [B, R, V] of `dtype` (SPEC_F32 or SPEC_BF16); R at most
 *           SPEC_MAX_TREE_NODES.  `out` may be `logits`: then only the logits
 *           that change are written.  Otherwise the two must not overlap.
 *   tokens  [B, T] int32 or NULL: the request's tokens so far, the first
 *           prompt_lens[b] of them its prompt, the others its output;
 *           token_lens [B] (NULL: T) of them are real.  Lengths are taken into
 *           [0, T] and [0, token_lens[b]]; prompt_lens NULL: no prompt.  T is
 *           below 2^29.
 *   draft_tokens: the window's tokens, which count as output for the rows
 *           behind them.  Without masks [B, R - 1], a chain: row i follows
 *           drafts 0..i-1.  With masks [B, R] and masks [B, R, ceil(R / 32)]
 *           int32 (spec_tree_masks), a tree: row n follows the nodes m >= 1
 *           whose bits of its mask are set (node 0 is the last of `tokens`).
 *           NULL: none.
 *   draft_lens [B] int32 or NULL (a chain's): only rows 0..draft_lens[b] are
 *           read and written; none where it lies outside [0, R - 1].
 *   repetition, frequency, presence [B] float32, each or NULL (1, 0, 0).
 *           With c the times that token t stands in the output before the row,
 *           and x its logit: if t stands in the prompt or c > 0, x becomes
 *           x / repetition where x > 0 and x * repetition elsewhere; then, if
 *           c > 0, x - frequency c - presence.
 *   bias_ids, bias_values [B, num_bias]: then x + the sum of the values of t
 *           (in the list's order; -inf bans it).  Ids outside [0, V), like
 *           tokens outside it in the other lists, are ignored.
 *   allowed [num_allowed, ceil(V / 32)] int32 or NULL: last, x becomes -inf
 *           where bit t % 32 of word t / 32 of the row's mask is clear,
 *           whatever x is (NaN included).  allowed_rows [B, R] is each row's
 *           mask, below 0 for none (num_allowed or more: all of the row
 *           becomes -inf, which the verify calls do not take); NULL: mask
 *           b * R + i, and num_allowed is B * R.
 * Arithmetic in fp32, rounded once. */
typedef struct spec_adjust_params {
    size_t size;
    const void *logits;
    void *out;
    int dtype;
    int B, R, V;
    const int32_t *tokens;
    const int32_t *token_lens;
    const int32_t *prompt_lens;
    int T;
    const int32_t *draft_tokens;
    const int32_t *masks;
    const int32_t *draft_lens;
    const float *repetition;
    const float *frequency;
    const float *presence;
    const int32_t *bias_ids;
    const float *bias_values;
    int num_bias;
    const int32_t *allowed;
    const int32_t *allowed_rows;
    int num_allowed;
} spec_adjust_params;
int spec_adjust_logits(const spec_adjust_params *params, spec_stream_t stream);

/* Rotary positions of a window's queries and keys.
 *   q [B, W, q_heads, head_dim], k [B, W, k_heads, head_dim] of `dtype`
 *         (SPEC_BF16 or SPEC_F16), strided as in spec_store_kv, and out_q,
 *         out_k likewise; head_dim a multiple of 16 up to 512.  q or k is NULL
 *         with no heads.  An output may be its input (same strides).  One that
 *         shares a byte with another array, or has two elements in one place,
 *         is refused (rows between the other's rows are apart).
 *   starts [B] int32: the position of window token 0.  It may differ from the
 *         cache's cursor (spec_evict_kv drops positions of the cache, not of
 *         the text).  Token i has position starts[b] + i, or with masks
 *         [B, W, ceil(W / 32)] (spec_tree_masks; W <= SPEC_MAX_TREE_NODES)
 *         starts[b] + its depth, one less than the bits of its row (at least 0).
 *   inv_freq [pairs] float64, finite: radians per position; pairs a multiple of 8,
 *         2 * pairs at most head_dim.  Pair i is
 *         elements (i, i + pairs), or (2 i, 2 i + 1) where interleaved != 0;
 *         elements from 2 * pairs on are copied.
 *   (a, b) becomes gain * (a cos - b sin, b cos + a sin) of the angle position
 *         * inv_freq.  The angle is reduced before it is rounded: while it
 *         stays below 2^34 radians, sine and cosine are good to 2^-21 however
 *         far the position.  Rounded once.
 * Padded rows (window_lens) are neither read nor written; a length outside
 * [0, W] has none. */
typedef struct spec_rotate_params {
    size_t size;
    const void *q;
    const void *k;
    void *out_q;
    void *out_k;
    int64_t q_strides[3], k_strides[3], out_q_strides[3], out_k_strides[3];
    int dtype;
    int B, W, q_heads, k_heads, head_dim;
    const int32_t *starts;
    const int32_t *window_lens;  /* [B] or NULL */
    const int32_t *masks;        /* or NULL */
    const double *inv_freq;
    int pairs, interleaved;
    float gain;                  /* finite */
} spec_rotate_params;
int spec_rotate_qk(const spec_rotate_params *params, spec_stream_t stream);

/* spec_rotate_qk and spec_store_kv in one call: q rotated to out_q, the
 * rotated keys (rounded to their type, as spec_rotate_qk leaves them) and v
 * into the cache at seq_lens, with the results of the two calls, bit for bit.
 * out_k must be NULL, k_heads and head_dim are the cache's; v is strided like
 * k.  The rows of q are rotated for every request whose window length is in
 * [0, W], those that store nothing included.  Arrays that overlap are refused as
 * there; the pool, its scales and the scratch are written too.
 *   scratch: spec_rotate_store_scratch_size(...) bytes (room for the rotated
 *         keys of long windows), 256-byte aligned, with the rules of
 *         spec_attend_kv's. */
int spec_rotate_store_kv(const spec_kv_cache *cache, const spec_rotate_params *params,
                         const void *v, const int64_t *v_strides, const int32_t *seq_lens,
                         void *scratch, size_t scratch_bytes, spec_stream_t stream);

/* Scratch of spec_rotate_store_kv (0 for invalid sizes). */
size_t spec_rotate_store_scratch_size(int B, int W, int kv_heads, int head_dim, int tokens_per_block);

/* The attention that each cached position drew from a window's rows.
 *   q, q_strides, dtype, seq_lens, window_lens, scale: as for spec_attend_kv,
 *         the window a chain.  (Of a tree, the accepted path is one: its rows
 *         of q and lse, window length n + 1, after the relocation.)
 *   lse   [B, W, q_heads] float32: spec_attend_kv's, of the same rows.
 *   weights, out [B, kv_heads, T] float32: for the positions t of request b,
 *         t < min(seq_lens[b] + w_b, T),
 *         out[b, h, t] = decay * weights[b, h, t]   (t < seq_lens[b] only)
 *                        + sum of exp(scale * q . k_t - lse)
 *         over the window's tokens that see t and the query heads of KV head
 *         h.  weights NULL: 0.  `out` may be `weights`, and is left as it is
 *         at every other position; that it or the scratch overlaps another array
 *         is refused.  A row whose lse is -inf adds nothing.
 * Positions in a block whose id lies outside [0, num_blocks) read NaN; for a
 * request with seq_lens < 0, w_b outside [0, W] or a window past max_blocks
 * blocks nothing is written.  Scores and sums are held in fp32 (a score is off by
 * at most D * 2^-23 of the sum of its products' magnitudes; exp(x) by 2^-22 +
 * |x| 2^-23 of itself); q's elements count to at least 2^-28 of their row's largest.
 *   scratch: spec_weigh_scratch_size(...) bytes, 256-byte aligned, with the
 *         rules of spec_attend_kv's (which may serve where it is large enough).
 * Limits: as spec_attend_kv's. */
typedef struct spec_weigh_params {
    size_t size;
    const void *q;
    int64_t q_strides[3];
    int dtype;
    int B, W, q_heads;
    const int32_t *seq_lens;
    const int32_t *window_lens;  /* [B] or NULL */
    const float *lse;
    float scale;                 /* finite, times log2(e) too */
    const float *weights;        /* or NULL */
    float decay;                 /* finite */
    float *out;
    int T;
} spec_weigh_params;
int spec_weigh_kv(const spec_kv_cache *cache, const spec_weigh_params *params, void *scratch,
                  size_t scratch_bytes, spec_stream_t stream);

/* Scratch of spec_weigh_kv for B requests of W window tokens (0 for invalid
 * sizes). */
size_t spec_weigh_scratch_size(int B, int W, int q_heads, int kv_heads, int head_dim);

/* Drops cached positions, head by head, down to `keep` of them.
 *   weights [B, kv_heads, T] float32 (spec_weigh_kv).  Of a request with
 *         seq_lens[b] > keep, each KV head keeps the first `first` positions,
 *         the last `recent`, and of those between the ones of largest weight,
 *         the lowest position among equals (NaN counts as less than any
 *         number, -0 as 0).  first + recent <= keep.
 *   The kept rows of K and V move, in their order, to positions 0..keep-1.  A
 *         block that receives rows gets, per kind and head, the largest scale
 *         among them; codes whose scale grows are rounded again, as in
 *         spec_relocate_quantised_kv.  Rows from position keep on are dead.
 *   new_lens [B] = min(seq_lens[b], keep) (may alias seq_lens);
 *   kept [B, kv_heads, keep] int32: the positions that the rows came from, -1
 *         behind new_lens[b]; out_weights [B, kv_heads, T_out] float32, T_out
 *         >= keep: their weights, left as it is from new_lens[b] on (may be
 *         `weights` itself, with T_out = T).  Arrays that overlap in any other
 *         way are refused;
 *   free_blocks [B] or NULL = max(0, blocks_held[b] - ceil(new_len /
 *         tokens_per_block)), for spec_release_blocks.
 * A request of at most `keep` positions keeps all and moves nothing.  One with
 * seq_lens < 0, more than max_blocks blocks or T positions, or a block id
 * outside [0, num_blocks) among those it has is left untouched: new_lens =
 * seq_lens, its kept rows all -1, free_blocks 0.  Blocks must not be shared
 * between requests, nor stand twice in a request's row.  Layers that share
 * block tables are evicted one by one, each with the same seq_lens.
 *   scratch: spec_evict_scratch_size(...) bytes, 256-byte aligned, with the
 *         rules of spec_attend_kv's. */
typedef struct spec_evict_params {
    size_t size;
    const float *weights;
    int T;
    int B;
    const int32_t *seq_lens;
    int keep, first, recent;
    int32_t *new_lens;
    int32_t *kept;
    float *out_weights;
    int T_out;
    const int32_t *blocks_held;  /* [B] or NULL */
    int32_t *free_blocks;        /* [B] or NULL */
} spec_evict_params;
int spec_evict_kv(const spec_kv_cache *cache, const spec_evict_params *params, void *scratch,
                  size_t scratch_bytes, spec_stream_t stream);

/* Scratch of spec_evict_kv (0 for invalid sizes). */
size_t spec_evict_scratch_size(int B, int kv_heads, int keep, int tokens_per_block);

/* Synchronise `stream`, read the workspace status word into *status_out
 * (SPEC_OK, SPEC_EBADINDEX or SPEC_ETIMEOUT) and clear it.  Returns SPEC_OK, SPEC_EINVAL or
 * SPEC_ECUDA. */
int spec_last_error(void *workspace, size_t workspace_bytes, spec_stream_t stream,
                    int *status_out);

/* Static text for a status code. */
const char *spec_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */

/*
 * spec_verify.h - batched speculative-sampling verifier for AMD MI355X (gfx950).
 *
 * One call verifies B rows of K draft tokens against one target pass:
 *
 *   - The target scored the prefix extended by the drafts in a single pass,
 *     so it provides K+1 next-token distributions per row: position i is
 *     conditioned on drafts d_0..d_{i-1}, position K is the bonus position
 *     ("Speculative decoding: memverifikasi token draft sebelum diterima",
 *     subsection "Draft mengubah tebakan serial menjadi batch verifikasi").
 *   - Both logit sets are turned into probabilities by softmax(l / T), the
 *     temperature acting at the verification gate (RheoSampling 2026,
 *     section 7).  The draft may first be cut to its topk_draft largest
 *     logits, the rest set to -inf, ties at the cut to the lowest id
 *     (RheoSampling 2026, section 3).
 *   - Draft d_i is accepted when u_i < min(1, p_i(d_i) / q_i(d_i)), evaluated
 *     as u_i * q < p; the first rejection ends the committed prefix
 *     (RheoSampling 2026, section 4, step 1; "Speculative decoding: ...",
 *     subsection "Penolakan memendekkan pekerjaan speculative yang berguna").
 *   - After a rejection at position n the final token is drawn from
 *     norm(max(0, p_n - q_n)); if all K drafts are accepted it is drawn from
 *     the bonus position p_K (RheoSampling 2026, section 4, step 3).  The
 *     draw is an inverse CDF in ascending token id with uniform u_K: the
 *     smallest x whose cumulative weight exceeds u_K * (total weight).
 *   - A row with T <= 0 is verified greedily: drafts are accepted while they
 *     equal the target's argmax (lowest id among equal maxima), and the
 *     target's argmax at the first mismatch (or at the bonus position) is
 *     emitted ("Speculative decoding: ...", subsection "Semantik penerimaan
 *     bergantung pada algoritma decoding").  Uniforms and draft logits of
 *     such rows are not read.
 *
 * All pointers are device pointers owned by the caller.  Inputs are read
 * only; outputs are fully overwritten.  The library allocates nothing, keeps
 * no mutable global state other than spec_verify_noalloc's static scratch,
 * and never synchronises: every call only enqueues
 * at most four kernels on `stream` (no memory set or copy), so a call can
 * be captured in a HIP graph and replayed; outputs are valid once the caller
 * has synchronised that stream.  Calls on different workspaces are
 * reentrant.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Storage type of both logit tensors. */
typedef enum { SV_BF16 = 0, SV_F32 = 1 } sv_dtype;

/* Return codes.  No call prints, throws or aborts. */
typedef enum {
  SV_OK = 0,
  SV_ERR_ARG = 1,          /* bad scalar or a NULL pointer that is required      */
  SV_ERR_WORKSPACE = 2,    /* *workspace_bytes smaller than the size required    */
  SV_ERR_UNSUPPORTED = 3,  /* 0 < topk_draft < V with topk_draft > SV_MAX_TOPK, or */
                           /* K > SV_MAX_K                                        */
  SV_ERR_HIP = 4,          /* a kernel launch failed (hipGetLastError)           */
  SV_ERR_SCRATCH = 5       /* spec_verify_noalloc: the shape needs more scratch  */
                           /* than SV_SCRATCH_BYTES                              */
} sv_status;

#define SV_MAX_TOPK 1024
#define SV_MAX_K 64
#define SV_MAX_NODES 64
/* Size of spec_verify_noalloc's static device scratch (per GPU). */
#define SV_SCRATCH_BYTES (32u << 20)

/*
 * spec_verify - verify B rows; see the description at the top of this file.
 *
 * target_logits  [B, K+1, V] device, dtype, row-major contiguous.
 * draft_logits   [B, K, V]   device, dtype, row-major contiguous; may be NULL
 *                when K == 0.
 * draft_tokens   [B, K] int32 device; may be NULL when K == 0.  A token outside
 *                [0, V) has p = q = 0 and is rejected.
 * uniforms       [B, K+1] float32 device, each in [0, 1).  u[b][i] (i < K)
 *                drives the acceptance test at position i; u[b][K] drives the
 *                final (correction or bonus) draw.
 * temperature    [B] float32 device; T <= 0 (or NaN) selects greedy for the row.
 * B >= 1, K in [0, SV_MAX_K], V >= 1.
 * topk_draft     0 or >= V: dense draft; otherwise keep the topk_draft largest
 *                draft logits per position (at most SV_MAX_TOPK).
 * dtype          sv_dtype of both logit tensors.
 * out_tokens     [B, K+1] int32 device: accepted drafts, the final token,
 *                then -1 padding.
 * num_accepted   [B] int32 device: number of accepted drafts, 0..K.  A row
 *                whose internal hand-off between work-groups did not complete
 *                within 100 ms (it completes in microseconds in any correct
 *                launch; the bound only guarantees termination) gets -1 here
 *                and -1 in every out_tokens slot.
 * workspace      device scratch of at least *workspace_bytes bytes, 256-byte
 *                aligned, zero-filled before its first use with a given
 *                shape (B, K, V, topk_draft, dtype), e.g. by hipMemset to 0.
 *                Every call leaves the regions its shape's layout needs
 *                zeroed again (its counters return to zero), so calls of the
 *                same shape can reuse it without clearing; a call of another
 *                shape lays the regions out differently and needs it
 *                zero-filled first.  Calls that overlap in time must use
 *                different workspaces.  NULL requests the size only:
 *                *workspace_bytes is set to the size required and nothing is
 *                launched.
 * workspace_bytes in: bytes available at workspace; out (size query): bytes
 *                required.  Must not be NULL.
 * stream         HIP stream to enqueue on (0 = null stream).
 *
 * Device data is not validated (that would need a synchronisation): logits
 * that are all -inf in a position, or NaN anywhere, give unspecified tokens
 * but every memory access stays in bounds.
 */
int spec_verify(const void* target_logits, const void* draft_logits,
                const int32_t* draft_tokens, const float* uniforms,
                const float* temperature, int B, int K, int V, int topk_draft,
                int dtype, int32_t* out_tokens, int32_t* num_accepted,
                void* workspace, size_t* workspace_bytes, hipStream_t stream);

/*
 * spec_verify_probe - spec_verify plus diagnostics, for parity tests.  Not
 * part of the serving API.
 *
 * probs_out  [B, K, 2] float32 device or NULL: (p_i(d_i), q_i(d_i)) for every
 *            position i < K of sampling rows (also after the first
 *            rejection); 0 for greedy rows.
 * mass_out   [B] float32 device or NULL: total weight S of the distribution
 *            the final token was drawn from (residual mass after a rejection,
 *            about 1 for the bonus); 0 for greedy rows.
 * Other arguments and return codes as spec_verify.
 */
int spec_verify_probe(const void* target_logits, const void* draft_logits,
                      const int32_t* draft_tokens, const float* uniforms,
                      const float* temperature, int B, int K, int V,
                      int topk_draft, int dtype, int32_t* out_tokens,
                      int32_t* num_accepted, void* workspace,
                      size_t* workspace_bytes, hipStream_t stream,
                      float* probs_out, float* mass_out);

/*
 * spec_verify_relaxed - spec_verify with a lossy relaxed acceptance rule in
 * place of u*q < p ("Acceptance Is Not Speed (arXiv:2610.23818): ...",
 * newsaint.id: section 1 describes verification that tolerates q > p within
 * a divergence budget, section 6 gives the budget's rule and a support guard,
 * section 7 recommends a strict support filter).  For each draft d_i of a
 * sampling row, in order:
 *   1. support guard: reject if d_i is outside [0, V), if its target rank
 *      1 + #{x : l_i(x) > l_i(d_i)} exceeds max_rank (max_rank = 0 disables
 *      the rank check), or if p_i(d_i) < min_prob;
 *   2. strict branch: accept if p_i(d_i) > 0 and q_i(d_i) <= p_i(d_i);
 *   3. otherwise accept iff u_i * q < gamma, gamma = min(p + sqrt(2 alpha p
 *      (1 - p)), 1) with p = p_i(d_i), q = q_i(d_i).
 * The first rejection ends the prefix as in spec_verify, and the correction
 * is drawn from the same residual norm(max(0, p_n - q_n)) (the pages leave
 * the correction under relaxed rules open; this is the plain reading).
 * Greedy rows (T <= 0) and the bonus draw are unchanged.  The output
 * distribution is no longer the target's: the rule is lossy by design.
 *
 * alpha     >= 0 divergence budget (0 with max_rank = 0 and min_prob = 0
 *           gives exactly spec_verify's decisions).
 * max_rank  >= 0 largest accepted target rank (0 = no rank check).  With a
 *           rank check the statistics pass also counts, per target position,
 *           the logits above l(d_i) (one compare per target logit).
 * min_prob  in [0, 1]: smallest accepted p_i(d_i).
 * probs_out, mass_out as spec_verify_probe (may be NULL).
 * Other arguments as spec_verify.  SV_ERR_ARG also for a negative or NaN
 * alpha, a negative max_rank or min_prob outside [0, 1].
 */
int spec_verify_relaxed(const void* target_logits, const void* draft_logits,
                        const int32_t* draft_tokens, const float* uniforms,
                        const float* temperature, int B, int K, int V,
                        int topk_draft, int dtype, float alpha, int max_rank,
                        float min_prob, int32_t* out_tokens,
                        int32_t* num_accepted, void* workspace,
                        size_t* workspace_bytes, hipStream_t stream,
                        float* probs_out, float* mass_out);

/*
 * spec_verify_kl - spec_verify that also returns KL(p_i || q_i), in nats, for
 * every draft position of each sampling row: the distillation signal that
 * test-time speculation takes from the verification step (gist.science
 * summary of paper 2605.09329, section 2: KL between the target's and the
 * drafter's distributions over the verified positions, with position weights
 * applied by the caller).  The value is exact up to fp32 rounding:
 *   KL = E_p[l_t - l_q] / T - ln 2 (fl(M_t s) - fl(M_q s)) - ln Z_t + ln Z_q
 * with the chunk statistics of the verification pass (s = log2(e) / T).
 * The statistics pass pairs each draft position with its target position so
 * that both are read once; tokens and num_accepted equal spec_verify's up to
 * the rounding of p and q (their decisions use the same partial sums).
 *
 * kl_out  [B, K] float32 device: KL(p_i || q_i); NaN for greedy rows (no
 *         sampling distribution); +inf where the draft gives zero mass to a
 *         token the target can produce.  Required when K > 0.
 * A sparse draft (0 < topk_draft < V) is not supported (KL against a
 * truncated draft is +inf): SV_ERR_UNSUPPORTED.  Other arguments and return
 * codes as spec_verify.
 */
int spec_verify_kl(const void* target_logits, const void* draft_logits,
                   const int32_t* draft_tokens, const float* uniforms,
                   const float* temperature, int B, int K, int V,
                   int topk_draft, int dtype, int32_t* out_tokens,
                   int32_t* num_accepted, void* workspace,
                   size_t* workspace_bytes, hipStream_t stream, float* kl_out);

/*
 * spec_verify_early_exit - spec_verify that verifies the positions of a row
 * one after the other and stops reading its logits at the first rejection:
 * no later draft can be committed ("Speculative decoding: memverifikasi
 * token draft sebelum diterima", subsection "Penolakan memendekkan pekerjaan
 * speculative yang berguna").  A row that rejects at position n reads the
 * target and draft logits of positions 0..n only (plus the residual pass of
 * position n), instead of all 2K+1 positions; in exchange its positions are
 * verified in sequence rather than in parallel.  Tokens, counts, the
 * probabilities p_i(d_i), q_i(d_i) and the final mass equal spec_verify's
 * bit for bit.
 *
 * One kernel per call for a dense draft.  topk_draft as spec_verify: a
 * truncated draft's selection does not depend on any decision, so such a
 * call makes every position's selection before the walk (three kernels:
 * position 0's statistics and the drafts' candidate lists, the selections,
 * the walk); it reads all K drafts of a sampling row, and the targets up to
 * the first rejection.  A shape whose row statistics ((2K+1) C 16 + C 128
 * bytes, plus 16 topk_draft for a truncated draft) do not fit the walking
 * kernel's LDS is SV_ERR_UNSUPPORTED.  The workspace has its own size (query
 * with workspace == NULL) and must not be shared with the other entry
 * points: each call leaves it ready for the next call of the same shape (a
 * dense draft leaves it all zero); zero-fill it before a call of another
 * shape.
 * probs_out  [B, K, 2] float32 device or NULL: (p_i(d_i), q_i(d_i)) of every
 *            position the row tested, NaN past its first rejection (and for
 *            greedy rows).
 * mass_out   [B] float32 device or NULL: as spec_verify_probe.
 * Other arguments and return codes as spec_verify.
 */
int spec_verify_early_exit(const void* target_logits, const void* draft_logits,
                           const int32_t* draft_tokens, const float* uniforms,
                           const float* temperature, int B, int K, int V,
                           int topk_draft, int dtype, int32_t* out_tokens,
                           int32_t* num_accepted, void* workspace,
                           size_t* workspace_bytes, hipStream_t stream,
                           float* probs_out, float* mass_out);

/*
 * spec_verify_tree - verify B rows of draft trees against one target pass
 * (RheoSampling 2026, section 4, RheoVerification: sibling candidates are
 * tested one after the other; an accepted candidate is descended into; after
 * a rejection the next sibling is tested against the residual
 * norm(max(0, r - q~)); when every candidate is rejected the final token is
 * drawn from the last residual).
 *
 * A row's tree has N nodes; node 0 is the root (the committed prefix) and
 * every other node c is a candidate token tok[c] drawn, independently of its
 * siblings, from the drafter's distribution at its parent par[c] < c.
 * Children are tested in increasing node index.  With r_0 = p_v at node v,
 * the j-th tested child (0-based) is accepted when u[c] * q_v(d) < r_j(d),
 * where r_j = max(0, p_v - c_j q_v) / W_j, c_0 = 0, W_0 = 1,
 * c_{j+1} = c_j + W_j, W_j = sum_x max(0, p_v(x) - c_j q_v(x)).  A rejection
 * therefore costs one pass over node v's target and draft logits (for the
 * next W).  A leaf reached by acceptance emits a bonus token drawn from its
 * target p_leaf.  Greedy rows (T <= 0) descend into the first child whose
 * token equals the node's target argmax and emit the argmax where none does.
 * Every draw is the inverse CDF of spec_verify with uniform u[b][0].  A chain
 * (par[c] = c - 1) gives exactly spec_verify's result with K = N - 1,
 * draft_tokens[i] = tok[i+1] and uniforms (u[1..N-1], u[0]).
 *
 * target_logits  [B, N, V] device, dtype: the target's next-token logits at
 *                each node (after the path root..node).
 * draft_logits   [B, N, V] device, dtype: the drafter's logits at each node;
 *                read only for nodes with children (other rows may hold any
 *                values) and never for greedy rows.
 * node_tokens    [B, N] int32 device; entry 0 is not read.  A token outside
 *                [0, V) has p = q = 0 and is rejected.
 * parents        [B, N] int32 device; entry 0 is not read.  par[c] must be
 *                < c; a node whose parent is not an earlier node is never
 *                reached.
 * uniforms       [B, N] float32 device in [0, 1): u[c] tests node c, u[0]
 *                drives the final draw.
 * temperature    [B] float32 device; T <= 0 (or NaN) selects greedy.
 * B >= 1, N in [1, SV_MAX_NODES], V >= 1.
 * topk_draft     0 or >= V: dense drafts; otherwise every node's draft is cut
 *                to its topk_draft largest logits (at most SV_MAX_TOPK), as in
 *                spec_verify, and a third kernel selects each node's kept set.
 * out_tokens     [B, N] int32 device: the tokens of the accepted nodes in
 *                path order, then the final token, then -1.
 * out_nodes      [B, N] int32 device: the accepted node indices in path
 *                order, then -1.
 * num_accepted   [B] int32 device: accepted nodes (-1 if a wait for another
 *                work-group's results timed out, which a correct launch
 *                never does).
 * workspace, workspace_bytes, stream as spec_verify (the size depends on
 *                B, N, V and dtype).
 * probs_out      [B, N, 3] float32 device or NULL: (p_v(d), q_v(d), r_j(d))
 *                of every tested node, NaN for nodes not tested.
 * mass_out       [B] float32 device or NULL: total weight of the final
 *                draw's distribution (W for a residual, ~1 for a target), 0
 *                for greedy rows.
 * Every call enqueues two kernels (three with a sparse draft).
 * SV_ERR_UNSUPPORTED also when the row's chunk statistics (2 N C 16 bytes,
 * plus 12 topk_draft bytes) do not fit the walking kernel's LDS.
 */
int spec_verify_tree(const void* target_logits, const void* draft_logits,
                     const int32_t* node_tokens, const int32_t* parents,
                     const float* uniforms, const float* temperature, int B,
                     int N, int V, int topk_draft, int dtype,
                     int32_t* out_tokens, int32_t* out_nodes,
                     int32_t* num_accepted, void* workspace,
                     size_t* workspace_bytes, hipStream_t stream,
                     float* probs_out, float* mass_out);

/*
 * spec_verify_tree_timed - spec_verify_tree (without probes) that also times
 * its kernels: events[0] / events[1] take the start / end of the statistics
 * kernel's dispatch, events[2] / events[3] those of the walking kernel (a
 * sparse draft's selection kernel runs between them, untimed).
 * n_events must be 4.
 */
int spec_verify_tree_timed(const void* target_logits, const void* draft_logits,
                           const int32_t* node_tokens, const int32_t* parents,
                           const float* uniforms, const float* temperature,
                           int B, int N, int V, int topk_draft, int dtype,
                           int32_t* out_tokens, int32_t* out_nodes,
                           int32_t* num_accepted, void* workspace,
                           size_t* workspace_bytes, hipStream_t stream,
                           hipEvent_t* events, int n_events);

/*
 * spec_verify_timed - spec_verify that also times each of its kernels on the
 * caller's stream, for measurement.
 *
 * events     array of n_events events created by the caller (hipEventCreate).
 *            events[0] / events[1] take the start / end timestamps of the
 *            statistics kernel's dispatch, events[2] / events[3] those of the
 *            sparse-draft merge kernel (both recorded after the statistics
 *            kernel when there is none), events[4] / events[5] those of the
 *            finishing kernel (decision, residual mass and final draw).
 *            n_events must be 0 or 6.
 * Other arguments and return codes as spec_verify.
 */
int spec_verify_timed(const void* target_logits, const void* draft_logits,
                      const int32_t* draft_tokens, const float* uniforms,
                      const float* temperature, int B, int K, int V,
                      int topk_draft, int dtype, int32_t* out_tokens,
                      int32_t* num_accepted, void* workspace,
                      size_t* workspace_bytes, hipStream_t stream,
                      hipEvent_t* events, int n_events);

/*
 * spec_verify_noalloc - spec_verify for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc).  Same arguments, semantics and results as spec_verify
 * (bit for bit), without the workspace: the scratch is a static device array
 * of SV_SCRATCH_BYTES inside the library, one per GPU, held until the
 * process ends.  Its device address is looked up once per device, on the
 * first call made with that device current.  Each call clears the part of
 * the scratch its shape uses with a small fill kernel on `stream` (no
 * memory set, so it can be captured) and then enqueues spec_verify's kernels.
 * The call allocates nothing (no hipMalloc, hipFree or allocating library
 * routine).
 *
 * Every call on a GPU shares that GPU's scratch: calls that overlap in time
 * on one GPU (different streams, or graphs replayed concurrently) race and
 * must not be issued; calls serialised on one stream are fine.
 * Returns SV_ERR_SCRATCH, before enqueuing anything, when the shape's
 * workspace (spec_verify's size query) exceeds SV_SCRATCH_BYTES -- a dense
 * draft of 256 rows, K = 7, V = 201,088 needs about 1.7 MB; truncated drafts
 * need about 2 KB per (row, position, vocabulary chunk) more up to
 * topk_draft = 128 (8 bytes per candidate entry, max(256, topk_draft, about
 * 4.5 topk_draft / C + 24) entries per chunk).  SV_ERR_HIP if
 * the scratch's address cannot be obtained.  Other codes as spec_verify.
 */
int spec_verify_noalloc(const void* target_logits, const void* draft_logits,
                        const int32_t* draft_tokens, const float* uniforms,
                        const float* temperature, int B, int K, int V,
                        int topk_draft, int dtype, int32_t* out_tokens,
                        int32_t* num_accepted, hipStream_t stream);

/*
 * spec_verify_launches - how many kernels a spec_verify (or _probe, _relaxed,
 * _timed) call of this shape enqueues: 2 for a dense draft (statistics,
 * finishing), 3 with a truncated draft (statistics, selection, finishing);
 * spec_verify_noalloc enqueues one more (the fill of its scratch).  A
 * negative value is minus an sv_status for a shape spec_verify refuses.
 */
int spec_verify_launches(int B, int K, int V, int topk_draft, int dtype);

/*
 * spec_verify_plan - the vocabulary split the library would use for a shape:
 * *chunks vocabulary chunks per (row, position), each *chunk_len ids long
 * (the last one may be shorter).  For tests that need inputs spanning several
 * chunks and a ragged tail.  Returns SV_OK or SV_ERR_ARG / SV_ERR_UNSUPPORTED.
 */
int spec_verify_plan(int B, int K, int V, int topk_draft, int dtype,
                     int* chunks, int* chunk_len);

/* Static description of a status code (never NULL). */
const char* spec_verify_status_string(int status);

/* ------------------------------------------------------------------------
 * Operators around a verification step
 *
 * One step of a serving program: attention of the step's tokens (the last
 * committed token and its drafts: a chain or a tree) over the row's cache
 * (spec_verify_attention), the model's remaining layers, penalties, biases
 * and grammar masks on the logits that come of it
 * (spec_verify_adjust_logits), spec_verify or spec_verify_tree, then the
 * accepted path's keys and values into the cache (spec_verify_commit: the
 * cache follows the committed prefix, "Speculative decoding: memverifikasi
 * token draft sebelum diterima", subsection "KV cache harus mengikuti token
 * yang di-commit"), and eviction of the blocks that drew the least attention
 * (spec_verify_evict).
 *
 * A prompt enters in one call (spec_verify_append), or as chains of up to
 * SV_MAX_K + 1 tokens that are all accepted.  Keys are rotated by their
 * positions before they meet the cache (spec_verify_rotate,
 * spec_verify_append).
 *
 * The rules at the top of this file hold: device pointers owned by the
 * caller, no allocation, no synchronisation, kernels only on `stream`, whose
 * device must be the current one; device data is not validated, but every
 * memory access stays in bounds for any values in the arrays.  Rows and
 * entries that a call's description leaves out are left as they were.
 * ------------------------------------------------------------------------ */

/*
 * sv_controls - what spec_verify_adjust_logits applies.  NULL members are
 * left out.  All pointers are device pointers.
 */
typedef struct {
  /* Tokens that count for the penalties: row b's are history[b *
   * history_stride + 0 .. history_lens[b]), of which the first
   * prompt_lens[b] are the prompt (prompt_lens NULL: none).  Lengths are
   * taken as at least 0 and at most history_stride, or history_width (below)
   * where that is not 0.  A token outside [0, V)
   * is ignored.  history may be NULL (no tokens but the drafted ones). */
  const int32_t* history;
  const int32_t* history_lens;
  const int32_t* prompt_lens;
  int64_t history_stride;
  const float* repetition; /* [B] r > 0, or NULL (1) */
  const float* presence;   /* [B], or NULL (0)       */
  const float* frequency;  /* [B], or NULL (0)       */
  /* Row b's biases are bias_ids / bias_values[b * bias_stride + 0 ..
   * bias_lens[b]) (bias_lens NULL: bias_stride entries).  Where a token is
   * listed more than once its last entry counts; ids outside [0, V) are
   * ignored. */
  const int32_t* bias_ids;
  const float* bias_values;
  const int32_t* bias_lens;
  int64_t bias_stride;
  /* Grammar masks [num_masks, ceil(V / 32)]: bit x % 32 of word x / 32 is 1
   * where token x is allowed.  Position i of row b goes by mask row
   * mask_rows[b * P + i], none if that is outside [0, num_masks);
   * mask_rows NULL: by mask row b * P + i. */
  const uint32_t* mask;
  const int32_t* mask_rows;
  int num_masks;
  /* Entries of a row's history that may be read, where rows lie further apart
   * than they are long: in [0, history_stride]; 0 means history_stride. */
  int64_t history_width;
} sv_controls;

/*
 * spec_verify_adjust_logits - penalties for repeated tokens, biases and
 * grammar masks on the logits of every position of a step, before they are
 * verified.
 *
 * Position i of row b follows the row's history and the drafted tokens
 * before it: of a chain (parents NULL) tokens[b][0 .. i-1], of a tree the
 * tokens of the nodes on the path from the root to node i, node i included
 * and the root (whose token ends the history) left out.  So one call serves
 * target logits [B, K+1, V] or draft logits [B, K, V] with the draft_tokens
 * of spec_verify, or either logits of spec_verify_tree with its node_tokens
 * and parents.  With n(x) the occurrences of token x in the history past the
 * prompt and on that path:
 *   l1 = l / r where x occurs at all (prompt included) and l > 0, l r where
 *        it occurs and l <= 0, l elsewhere
 *   l2 = l1 - frequency n(x) - presence [n(x) > 0]
 *   l3 = l2 + bias(x)
 *   out = l3 where x is allowed, -inf elsewhere
 * in float32, rounded once to dtype.  Logits that nothing applies to keep
 * their bits.  A mask that allows no token leaves a position all -inf, for
 * which spec_verify's result is unspecified.
 *
 * logits       element (b, i, x) at b * row_stride + i * stride + x, of the
 *              stated dtype and aligned to it; strides in elements, stride >=
 *              V.
 * out          likewise, with out_row_stride and out_stride.  It may be the
 *              logits themselves with the same strides (then only what
 *              changes is written, and only what a penalty or bias changes
 *              is read); otherwise it must not overlap them.
 * tokens       [B, tokens_stride] int32, tokens_stride >= P - 1 (P for a
 *              tree); NULL where no penalty is given or P == 1.
 * parents      [B, P] int32 as in spec_verify_tree, or NULL: a chain.  The
 *              path of a node whose parent is not an earlier node starts at
 *              that node.
 * B >= 1, P in [1, SV_MAX_K + 1] (SV_MAX_NODES with parents), V >= 1.
 * One kernel, no workspace.  SV_ERR_ARG, SV_ERR_UNSUPPORTED (P too large; a
 * history_width or bias_stride beyond 2^30 - 1024; 2^24 and more rows times
 * parts of 4096 ids, of 2048 where bias_stride passes 2048) or SV_ERR_HIP.
 */
int spec_verify_adjust_logits(const void* logits, int64_t row_stride,
                              int64_t stride, const int32_t* tokens,
                              int64_t tokens_stride, const int32_t* parents,
                              const sv_controls* controls, int B, int P, int V,
                              int dtype, void* out, int64_t out_row_stride,
                              int64_t out_stride, hipStream_t stream);

/* How a cache's values are held in 8 bits: OCP e4m3 (no infinities) or
 * two's-complement int8; a value stands for code * its block's scale. */
typedef enum { SV_E4M3 = 0, SV_INT8 = 1 } sv_kind;

#define SV_MAX_BLOCKS 65536

/*
 * sv_cache - a paged cache of B rows.  A row's committed tokens are cut into
 * blocks of `page` tokens.  Full blocks are held in 8 bits, one page each,
 * with a scale for each block and kv head; the tokens after the last full
 * block (the tail) are held in bf16, so nothing is ever quantised twice and a
 * rejected draft leaves no trace.  All pointers are device pointers; the
 * pages, tails and scales are written by spec_verify_commit and
 * spec_verify_append only.
 *
 * k_pages      [num_pages, Hkv, page, D] codes
 * v_pages      [num_pages, Hkv, D, page] codes: a channel's tokens side by
 *              side, as the matrix instructions take them
 * k_scale, v_scale [num_pages, Hkv] float32, positive (a NaN makes every
 *              output that sees the block NaN; attention takes a v_scale below
 *              2^-126 as 2^-126)
 * k_tail, v_tail [B, tail, Hkv, D] bf16 rings: the row's token number p lies in
 *              slot p % tail.  tail is a multiple of page.
 * block_table  [B, max_blocks] int32: the page of each block; entries past a
 *              row's blocks are its reserve.  A block whose entry is outside
 *              [0, num_pages) is not seen by attention.
 * Two counters [B] int32 go with a cache, and are passed to each call:
 * positions[b], the tokens committed to row b so far, and blocks[b], the full
 * blocks it keeps.  positions[b] % page tokens lie in the tail; positions[b]
 * / page - blocks[b] blocks have been evicted.
 * Pages, tails 16-byte aligned.  page in {16, 32, 64, 128, 256}, D in {64,
 * 128}, B <= 65536, Hkv <= 4096, max_blocks <= SV_MAX_BLOCKS, tail <= 2^20.
 */
typedef struct {
  uint8_t* k_pages;
  uint8_t* v_pages;
  float* k_scale;
  float* v_scale;
  uint16_t* k_tail;
  uint16_t* v_tail;
  int32_t* block_table;
  int B, num_pages, Hkv, D, page, max_blocks, tail, kind;
} sv_cache;

/*
 * spec_verify_attention - attention of a step's T new tokens per row (the
 * last committed token's successor positions: the root and its drafts) over
 * the row's cache and over each other.
 *
 * Query (b, t, h) goes with kv head h / (H / Hkv).  It sees every full block
 * of row b, the tail, and of the new tokens those before it and itself (a
 * chain, parents NULL) or those on its path from the root, itself included (a
 * tree; the path of a node whose parent is not an earlier node starts at that
 * node).  With s = scale q.k over what it sees:
 *   out = sum softmax(s) v
 *   weights[b][t][j] = the softmax mass of block j, summed over the H heads
 * What a query does not see does not reach it, infinities and NaN included.
 * Scores and softmax statistics are float32; q, the new tokens and the tail
 * enter as bf16 and the codes exactly, whatever their scales; a probability is
 * rounded to 11 bits beside a code, or by at most 2^-21 of the largest one of
 * its 64 cached keys (the row's keys 64 i .. 64 i + 63; 2^-16 where these are
 * of several pages), and to 16 bits beside a tail or new token's value; what
 * is 2^-100 of the largest may be lost; the output is rounded to bf16.
 *
 * q            element (b, t, h, d) at b * q_row + t * q_tok + h * D + d, bf16
 * k_new, v_new element (b, t, h, d) at b * kv_row + t * kv_tok + h * D + d,
 *              bf16.  All three may be views of one projection's output; 16-byte
 *              aligned, strides multiples of 8.
 * positions, blocks [B] int32, see sv_cache.
 * parents      [B, T] int32 or NULL.
 * query_lens   [B] int32 or NULL: row b has only that many (0 .. T) new
 *              tokens.  What lies behind them in q, k_new and v_new is not
 *              read, and in out and weights not written; a row of 0 is idle.
 * T in [1, SV_MAX_K + 1] ([1, SV_MAX_NODES] with parents), H a multiple of
 * Hkv (at most 256 times it), scale positive and finite.  B (max_blocks * page
 * / 64 + 10) ceil(T * H / Hkv / 16) < 2^30.
 * out          [B, T, H, D] bf16 contiguous.  Neither it nor weights may
 *              overlap the other, the workspace, a row of q, k_new or v_new,
 *              or another input.
 * weights      [B, T, max_blocks] float32 or NULL; 0 for blocks that a row does
 *              not have.  Fewer than 2^32 of them.
 * workspace, workspace_bytes  as spec_verify, but only its first 4 * B * Hkv *
 *              ceil(T * H / Hkv / 16) bytes need to be zero-filled before its
 *              first use with a given shape (B, T, H and Hkv, parents or not,
 *              weights or not, and the cache's D, page, max_blocks); left ready
 *              for the next call of that shape, not to be used by two calls at
 *              once.
 * One kernel, two with weights.
 */
int spec_verify_attention(const void* q, int64_t q_row, int64_t q_tok,
                          const void* k_new, const void* v_new, int64_t kv_row,
                          int64_t kv_tok, const sv_cache* cache,
                          const int32_t* positions, const int32_t* blocks,
                          const int32_t* parents, const int32_t* query_lens,
                          int T, int H, float scale, void* out, float* weights,
                          void* workspace, size_t* workspace_bytes,
                          hipStream_t stream);

/*
 * sv_prefix - pages that several rows share: what their prompts have in
 * common.  Rows starts[i] .. starts[i + 1] - 1 begin with prefix i, the first
 * blocks[i] pages of table[i]; other rows have none.  A row's own blocks, tail
 * and new tokens follow it: positions[b] counts the prefix's tokens too,
 * blocks[b] and block_table[b] only the row's own blocks (the prefix's are, to
 * its counters, blocks that were evicted), so spec_verify_commit, _append and
 * _evict go on as they do without one.  The prompt's tokens past the last full
 * block belong in each row's tail.  No row may have a prefix's page in reserve.
 *
 * table        [count, max_blocks] int32 pages of the cache; an entry outside
 *              [0, num_pages) is not seen.
 * blocks       [count] int32.
 * starts       [count + 1] int32, ascending (a prefix may have no rows).
 * count in [1, 65536], max_blocks in [1, SV_MAX_BLOCKS].
 */
typedef struct {
  const int32_t* table;
  const int32_t* blocks;
  const int32_t* starts;
  int count, max_blocks;
} sv_prefix;

/*
 * spec_verify_attention_prefix - spec_verify_attention of rows that share
 * prefixes: each query sees its row's prefix too, and softmax and weights are
 * over both.  A prefix's keys are read once for all its rows.  Beside its
 * codes a probability is rounded to 11 bits, to at least 8 where it is less
 * than 2^-16 of the largest (each times its value scale) of 64 keys.
 *
 * weights[b][t][j] are those of the row's own blocks.
 * prefix       NULL: spec_verify_attention.
 * Other arguments as spec_verify_attention, but the workspace's size also
 * depends on prefix->max_blocks (for SV_MAX_BLOCKS it is the largest): one that
 * is large enough serves every prefix of a shape, and calls without one.
 * (B T H / Hkv / 128 + count) Hkv < 2^23, B T H D < 2^34.
 * Three kernels, four with weights.
 */
int spec_verify_attention_prefix(
    const void* q, int64_t q_row, int64_t q_tok, const void* k_new,
    const void* v_new, int64_t kv_row, int64_t kv_tok, const sv_cache* cache,
    const sv_prefix* prefix, const int32_t* positions, const int32_t* blocks,
    const int32_t* parents, const int32_t* query_lens, int T, int H,
    float scale, void* out, float* weights, void* workspace,
    size_t* workspace_bytes, hipStream_t stream);

/*
 * spec_verify_commit - the accepted path's keys and values enter the cache.
 *
 * Row b commits its root and its accepted drafts: n = num_accepted[b] + 1 of
 * its new tokens, the first n of a chain (nodes NULL), or token 0 and then
 * nodes[b][0 .. n-2], spec_verify_tree's out_nodes.  They follow the tail;
 * each block that this completes is quantised into the page that the row's
 * block table has in reserve, block_table[b][blocks[b]] first, and the
 * tokens after the last full block go to their slots of the tail ring.  The
 * tail's old tokens stay where they are and the counters are put out, so a
 * step can be undone by keeping the counters from before it.
 *
 * A block's scale is, with a the largest magnitude of its head's page * D
 * values: e4m3, the smallest power of two of at least a / 448; int8, a / 127
 * rounded to float32; in both at least 2^-126, and 1 where a is 0.  Its codes
 * are the values over the scale, rounded to nearest even exactly.  A block
 * that holds an infinity or NaN gets a NaN scale (and codes 0).
 *
 * A row is left as it was, its counters repeated, where num_accepted is
 * outside [0, T - 1] (spec_verify's -1 among it), a node outside [0, T), a
 * counter out of range, or a completed block has no page (its table entry is
 * past max_blocks or outside [0, num_pages)): an active row always advances.
 *
 * k_new, v_new, kv_row, kv_tok, T as spec_verify_attention.
 * num_accepted [B] int32; nodes [B, nodes_stride] int32 or NULL, nodes_stride
 *              >= T - 1.
 * cache        with tail >= page - 1 + T.  No page may be in reserve for two
 *              rows, nor in reserve for one and among the blocks of another.
 *              B (2 + 2 Hkv + max_blocks / 256) < 2^24.
 * positions_out, blocks_out [B] int32; both may be the inputs themselves (then
 *              a second kernel updates them).
 * weights      [B, T, max_blocks] float32 (spec_verify_attention's) or NULL.
 * totals, totals_out [B, max_blocks] float32, both or none: totals_out[b][j]
 *              is totals[b][j] plus the weights of block j from the committed
 *              tokens for the blocks that row b had, 0 for the rest.  They may
 *              be the same array.  So a total counts what a block drew since it
 *              was complete, not what its tokens drew in the tail: a new block
 *              starts from 0, and spec_verify_evict's keep_last keeps it until
 *              it has drawn some.
 * Beyond that no output may overlap an input or another output.
 */
int spec_verify_commit(const void* k_new, const void* v_new, int64_t kv_row,
                       int64_t kv_tok, int T, const int32_t* num_accepted,
                       const int32_t* nodes, int64_t nodes_stride,
                       const sv_cache* cache, const int32_t* positions,
                       const int32_t* blocks, int32_t* positions_out,
                       int32_t* blocks_out, const float* weights,
                       const float* totals, float* totals_out,
                       hipStream_t stream);

/*
 * spec_verify_evict - blocks that drew little attention leave the cache.
 *
 * Where row b has more than `budget` blocks, the blocks[b] - budget of least
 * totals leave, of those that are neither among its first keep_first nor its
 * last keep_last (all of these if they are fewer); of equal totals the
 * earlier block leaves first, and a NaN counts as above every number.  The
 * row's table becomes the pages of the blocks kept, then those evicted, then
 * its old reserve, each in their order: the evicted pages are the next ones
 * that spec_verify_commit fills.  totals follow the blocks kept; the rest are
 * 0.  No page is read or moved.  (A key's position is in its values, so a
 * block's place in the table does not matter to attention.)
 *
 * totals       [B, max_blocks] float32
 * block_table  [B, max_blocks] int32
 * blocks       [B] int32
 * totals_out, table_out, blocks_out  as these; each may be its input itself
 *              (table_out only up to max_blocks = 16384, else
 *              SV_ERR_UNSUPPORTED).  Beyond that no output may overlap an input
 *              or another output.
 * evicted      [B] int32: how many blocks left.
 * budget, keep_first, keep_last >= 0; 1 <= max_blocks <= SV_MAX_BLOCKS; B <
 * 2^22.
 * One kernel, no workspace.
 */
int spec_verify_evict(const float* totals, const int32_t* block_table,
                      const int32_t* blocks, int B, int max_blocks, int budget,
                      int keep_first, int keep_last, float* totals_out,
                      int32_t* table_out, int32_t* blocks_out,
                      int32_t* evicted, hipStream_t stream);

/*
 * sv_rotary - the rotation of queries and keys by their positions.  The
 * first `dims` channels of a head are dims / 2 pairs: channels i and i + dims
 * / 2, or 2 i and 2 i + 1 where interleaved is 1.  Pair i (a, b) of a token at
 * position p becomes
 *   (a cos x - b sin x, b cos x + a sin x),  x = p freqs[i]
 * with x (up to 2^52 in magnitude), its cosine and its sine in 64 bits, the
 * last two rounded to float32, the products and sums in float32 and the result rounded to bf16.  The other
 * channels stay as they are.
 *
 * freqs        [dims / 2] float32 device.  dims a multiple of 16, at most D.
 * ids          [num_axes, B, T] int32 device, or NULL.  Positions of their
 *              own for each token, one number for each axis (time, height and
 *              width of a picture's or video's tokens); pair i goes by axis
 *              axes[i] (taken into [0, num_axes)).  NULL: the position that
 *              each call describes.
 * axes         [dims / 2] int32 device, or NULL (axis 0).  Needs ids.
 * num_axes     1 .. 16; read only with ids.
 */
typedef struct {
  const float* freqs;
  const int32_t* ids;
  const int32_t* axes;
  int num_axes, dims, interleaved;
} sv_rotary;

/*
 * spec_verify_rotate - the queries and keys of a step rotated by their
 * positions, as spec_verify_attention takes them.
 *
 * Token t of row b is at position positions[b] + t, of a tree (parents given)
 * at positions[b] + the number of steps on its path from the root (0 where the
 * path starts at the node itself), or where rotary->ids says.
 *
 * q            element (b, t, h, d) at b * q_row + t * q_tok + h * D + d, bf16;
 *              k likewise, with Hkv heads.  Views of one projection's output
 *              will do; 16-byte aligned, strides multiples of 8.
 * q_out, k_out likewise.  Each may be its input itself, with the same strides;
 *              beyond that neither may overlap the other or an input (the
 *              views of one tensor may lie between each other).
 * positions    [B] int32, the tokens before the step (a cache's); may be NULL
 *              with ids.
 * parents      [B, T] int32 or NULL, as in spec_verify_attention.
 * query_lens   [B] int32 or NULL: row b has only that many (0 .. T) tokens;
 *              what lies behind them is not read and not written.
 * B, T, H, Hkv >= 1, H and Hkv at most 65536, T at most SV_MAX_NODES with
 * parents, fewer than 2^24 fours of tokens in all rows; D a multiple of 16, at
 * most 512.  One kernel, no workspace.
 */
int spec_verify_rotate(const void* q, int64_t q_row, int64_t q_tok,
                       const void* k, int64_t k_row, int64_t k_tok,
                       const sv_rotary* rotary, const int32_t* positions,
                       const int32_t* parents, const int32_t* query_lens,
                       int B, int T, int H, int Hkv, int D, void* q_out,
                       int64_t qo_row, int64_t qo_tok, void* k_out,
                       int64_t ko_row, int64_t ko_tok, hipStream_t stream);

/*
 * spec_verify_append - a prompt's keys and values enter the cache, the keys
 * rotated on the way: what spec_verify_rotate and then spec_verify_commit of
 * chains that are all accepted would leave, bit for bit, for any number of
 * tokens.
 *
 * Row b appends its first lens[b] tokens (lens NULL: all T), token t at
 * position positions[b] + t or where rotary->ids says.  A row is left as it
 * was, its counters repeated, where lens[b] is outside [0, T], a counter is
 * out of range or a completed block has no page.
 *
 * k, v         element (b, t, h, d) at b * kv_row + t * kv_tok + h * D + d,
 *              bf16, as spec_verify_attention's k_new and v_new.  Tokens behind
 *              lens[b] are not read.
 * rotary       NULL: the keys are rotated already (or need not be).
 * cache        with any tail.  The tokens after the last full block overwrite
 *              the tail's old ones where the ring is shorter than page - 1 +
 *              lens[b]; such an append cannot be undone by keeping the counters
 *              from before it.  Pages in reserve as spec_verify_commit has it.
 * k_out        the keys as they enter the cache, at b * ko_row + t * ko_tok +
 *              h * D + d, or NULL; may be k itself with the same strides.
 *              Rows that are left as they were, and what lies behind lens[b],
 *              are not written.
 * positions_out, blocks_out [B] int32; both may be the inputs themselves (then
 *              a second kernel updates them).  Beyond that no output, the cache's
 *              pages, scales and tails among them, may overlap an input or
 *              another output.
 * T in [1, 2^24]; B (page - 1 + T) / page Hkv < 2^24.
 */
int spec_verify_append(const void* k, const void* v, int64_t kv_row,
                       int64_t kv_tok, int T, const int32_t* lens,
                       const sv_rotary* rotary, const sv_cache* cache,
                       const int32_t* positions, const int32_t* blocks,
                       int32_t* positions_out, int32_t* blocks_out,
                       void* k_out, int64_t ko_row, int64_t ko_tok,
                       hipStream_t stream);

/*
 * spec_verify_sample - tokens drawn from logits: drafts (several siblings of a
 * node at once), or the next tokens of rows without drafts.
 *
 * Position i of row b goes by the row's rules.  With its tokens in the order
 * of their logits (larger first, of equal ones the lower id first), w(x) =
 * exp((l(x) - max l) / temperature[b]) and the mass of a set the sum of its
 * w:
 *   top_k   the first top_k[b] tokens stay (0 or less, V or more: all)
 *   top_p   of those, each before which less than top_p[b] of their mass lies;
 *           the first one always (1 or more, NaN: all)
 *   min_p   of those, each with w >= min_p[b], taken as at most 1 (0 or less,
 *           NaN: all)
 * Draw j is the smallest kept id x for which the mass of the kept ids up to x
 * exceeds uniforms[b][i][j] times the mass of all kept: spec_verify's draw,
 * and with top_k alone spec_verify's truncated draft.
 * Weights are formed in float64, to 2^-39 of each, and are 0 under 2^-1000, so
 * that such a token is not drawn.  Where rules cut a row the weights added up
 * are whole multiples of 2^-43.  A cut by mass or a draw is that of exact
 * weights unless a border lies within 2^-37 of the row's mass or, where rules
 * cut the row, 2^-43 times the number of tokens added up.  Sums of whole
 * multiples do not depend on their order.  A sum over a whole row, by which
 * rows without rules are drawn from and top_p goes without a top_k, is float64's
 * over parts of the row, which depend on B P and the row's alignment: so near a
 * border its result may change with the batch.
 * Rows with T <= 0 (or NaN) take the largest logit's lowest id.  A NaN logit
 * counts as -inf and -inf is never drawn; where there is nothing else the
 * token is -1 and its logprob -inf.
 *
 * logits       element (b, i, x) at b * row_stride + i * stride + x, of the
 *              stated dtype and aligned to it; strides in elements, stride >=
 *              V.
 * uniforms     [B, P, n] float32 in [0, 1) (taken into it).
 * temperature  [B] float32; top_k [B] int32, top_p, min_p [B] float32, or
 *              NULL.
 * tokens       [B, P, n] int32.
 * logprobs     [B, P, n] float32 or NULL: ln of each token's part of the kept
 *              mass, 0 for greedy rows.
 * workspace, workspace_bytes  as spec_verify, but it need not be zero-filled.
 * B, P >= 1; V in [1, 2^20]; n in [1, SV_MAX_NODES]; fewer than 2^24 parts of
 * 16,384 logits (8192 of float32) in all rows.  Two kernels.
 */
int spec_verify_sample(const void* logits, int64_t row_stride, int64_t stride,
                       const float* uniforms, const float* temperature,
                       const int32_t* top_k, const float* top_p,
                       const float* min_p, int B, int P, int V, int n,
                       int dtype, int32_t* tokens, float* logprobs,
                       void* workspace, size_t* workspace_bytes,
                       hipStream_t stream);

/*
 * spec_verify_truncate - the logits of tokens that spec_verify_sample's rules
 * leave out become -inf, the others keep their bits: spec_verify on target (or
 * draft) logits cut so verifies against the distribution that
 * spec_verify_sample draws from.  NaN counts as -inf, and becomes it, in every
 * row that a rule applies to.  Greedy rows, and rows whose rules are all off
 * (top_k 0 or less or V or more, top_p 1 or more, min_p 0 or less, or NaN), are
 * not changed.
 *
 * out          element (b, i, x) at b * out_row_stride + i * out_stride + x.  It
 *              may be the logits themselves with the same strides; otherwise it
 *              must not overlap them.
 * Other arguments as spec_verify_sample; fewer than 2^24 parts of 8192 logits
 * (4096 of float32) in all rows.  Two or three kernels.
 */
int spec_verify_truncate(const void* logits, int64_t row_stride,
                         int64_t stride, const float* temperature,
                         const int32_t* top_k, const float* top_p,
                         const float* min_p, int B, int P, int V, int dtype,
                         void* out, int64_t out_row_stride, int64_t out_stride,
                         void* workspace, size_t* workspace_bytes,
                         hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */

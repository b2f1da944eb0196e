/*
 * specverify -- batched speculative-sampling verify step for AMD Instinct
 * MI355X (gfx950), C ABI.
 *
 * One call verifies a batch of B sequences, each with up to K drafted tokens:
 *
 *   1. temperature softmax over the vocabulary for every target position
 *      0..L_b and every draft position 0..L_b-1 of row b;
 *   2. optionally the top-p (nucleus) filter on each of those distributions;
 *   3. for j = 0..L_b-1 the acceptance test u < min(1, p'(x_j)/q'(x_j)), where
 *      the first failing j is the row's first rejection n_b (n_b = L_b if
 *      none fails);
 *   4. one more token: on a rejection, drawn from max(0, p'_n - q'_n)/Z by
 *      inverse CDF; otherwise a bonus token drawn from p'_L.
 *
 * The method is the one on the page "Speculative Decoding للمحترف: ضاعف سرعة
 * Llama 70B لـ 2.4x بدون فقد token واحد": section "المفهوم بالتقريب" (accept
 * agreed tokens, reject the first disagreeing one and resample it), section
 * "التعريف الرياضي من Leviathan et al." (the equation for the acceptance
 * probability alpha(x) = min(1, p_target(x)/p_draft(x)) and the equation for
 * the corrected distribution p'(x) = max(0, p_target(x) - p_draft(x))/Z),
 * section "كود شغّال على vLLM" (the knobs K, temperature and top_p).  The bonus
 * token is the one of the page "Faster LLM Inference via Sequential Monte
 * Carlo", section 2 (the scoring step over K+1 positions).  Per-row draft
 * lengths follow the page "HiSpec: Hierarchical Speculative Decoding for LLMs",
 * section 2 (per-sequence acceptance in a batch without padding).
 *
 * Uniforms come from Philox4x32-10 (Salmon et al., SC'11) with key = (seed low
 * word, seed high word) and counter = (row, position, 0, 0): output word 0
 * gives the acceptance uniform, word 1 the resampling uniform, each as
 * (word >> 8) * 2^-24.  Any implementation following that contract reproduces
 * the outputs bit for bit, decisions lying within rounding of a boundary
 * aside.  Precision: the softmax normalisers behind the acceptance tests are
 * float32 exponentials summed per lane and wave in float32 (relative error
 * below 1.2e-6 each, so below 2.4e-6 on p'(x)/q'(x)); the draw of step 4 is
 * float64 throughout (its own normalisers of the two rows at n, float64
 * exponentials and masses), so its token is the exact inverse-CDF token
 * unless u*Z lies within about 1e-13*Z of a boundary.
 *
 * Memory: every pointer argument is caller-owned device memory unless stated
 * otherwise.  Inputs are only read; outputs are written in full for every row.
 * The library owns a small scratch buffer per (device, stream), grown on first
 * use and kept until spec_verify_release().  Calls are asynchronous on the
 * given stream and never synchronise the host (except a first call on a
 * stream, or a call that outgrows the cached scratch, which allocates).
 *
 * Graphs: a call that does not allocate may be captured into a HIP graph:
 * each kernel of a call rewrites, before any reader needs it, all scratch
 * that later kernels of the same call read, so replays are independent.  A
 * call that would have to grow the scratch while its stream is being
 * captured returns SV_ECAPTURE and enqueues nothing (make one call of the
 * largest shape on that stream before capturing).  A buffer outgrown later
 * is kept, not freed, so graphs captured earlier stay valid;
 * spec_verify_release() frees every buffer and so invalidates every graph
 * that holds a call of this library.
 *
 * Concurrency: concurrent calls on the same stream from several host threads
 * are not supported.  Calls on different streams may run concurrently, each
 * on its stream's own scratch.  No workgroup of a call waits for another
 * workgroup to start: the row pass splits a logit row over workgroups, and
 * the one that completes the row's arrival count draws the token from the
 * records the others left, so any number of calls, and any other work on the
 * device, can share it.  A row whose record is found missing or foreign (a
 * corrupted scratch; not otherwise possible) reports out_n_accepted = -2 and
 * every token -1 (an SMC particle: bonus -2).
 *
 * Testing: with the environment variable SPECVERIFY_FAIL_LAUNCH set to a
 * non-zero value every call fails as a failed kernel launch does (SV_EHIP,
 * message through spec_verify_strerror) before touching the device.
 * SPECVERIFY_AMB_BAND (a number) replaces the relative error the row pass
 * assumes for the float32 kept-mass ratio when it classifies ids before the
 * exact ratio is known: 0 sends every row through the exact second round, a
 * wide band fills the ambiguous groups.  The result is the same either way;
 * only the path (and its time) changes.  SPECVERIFY_VERIFY_LOOKS (0 to 64) is
 * how often a workgroup of spec_verify_tree looks for another's partial sum
 * before it computes it itself; the result is the same again.
 */
#ifndef SPECVERIFY_H
#define SPECVERIFY_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPECVERIFY_ABI_VERSION 1
#define SPECVERIFY_MAX_K 16
/* Largest vocabulary of the calls that draw a token (spec_verify,
 * spec_verify_probe, spec_smc_step, spec_hispec_verify; beyond it SV_ESHAPE).
 * Greedy verify and the draft producer take V up to 2^24. */
#define SPECVERIFY_MAX_V (1 << 21)

/* Element type of a logits tensor. */
typedef enum { SV_F32 = 0, SV_BF16 = 1 } sv_dtype;

/* Describes a device tensor of logits [B, P, V] whose V axis is contiguous.
 * Element (b, p, v) lives at data + (b*stride_b + p*stride_p + v) elements.
 * data must be aligned to the element size; strides may be anything >= 0
 * (rows need not start on 16-byte boundaries). */
typedef struct {
    const void* data;
    int32_t dtype;       /* sv_dtype */
    int32_t B, P, V;     /* P = K+1 for target logits, K for draft logits */
    int64_t stride_b;    /* elements */
    int64_t stride_p;    /* elements */
} sv_logits;

/* Status codes.  Negative values are errors. */
enum {
    SV_OK = 0,
    SV_EINVAL = -1,   /* NULL pointer, bad temperature or top_p, bad stride */
    SV_ESHAPE = -2,   /* B, K or V out of range, or the two tensors disagree */
    SV_EDTYPE = -3,   /* unknown dtype, or target and draft dtypes differ */
    SV_EHIP = -4,     /* a HIP runtime call failed; see spec_verify_strerror */
    SV_ENOMEM = -5,   /* an allocation failed (scratch, or host memory) */
    SV_EALIGN = -6,   /* a pointer is not aligned to its element size */
    SV_ECAPTURE = -7, /* the stream is being captured and the scratch would have to grow */
    SV_ETOOBIG = -8   /* spec_verify_noalloc: the call needs more than its fixed scratch;
                         tree and cache calls: the workspace is too small */
};

/* Probe record layout (float64), per row b and position j in [0, K]:
 *   [0] target max logit          [1] target sum_v exp((l_v - max)/T)
 *   [2] draft max logit           [3] draft sum_v exp((l_v - max)/T)
 *   [4] p'(x_j), filtered target  [5] q'(x_j), filtered draft
 *   [6] kept target mass (1 when top-p is off)
 *   [7] kept draft mass  (1 when top-p is off)
 * and per row b:
 *   [0] Z, the mass the final token is drawn from
 *   [1] t = u * Z, the inverse-CDF threshold
 *   [2] u, the resampling uniform
 *   [3] n, the first-rejection index
 * Entries for positions a row does not evaluate are NaN. */
#define SV_PROBE_POS 8
#define SV_PROBE_ROW 4

/*
 * spec_verify -- the verify step (steps 1-4 above) for B rows.
 *
 * target_logits   [B, K+1, V] target logits, bf16 or fp32;
 *                 1 <= B <= 2^22, 1 <= V <= SPECVERIFY_MAX_V.
 * draft_logits    [B, K, V] draft logits, same dtype, B and V; 1 <= K <= 16.
 * draft_tokens    device int32 [B, K], contiguous; entry (b, j) is the drafted
 *                 id at position j, read only for j < L_b.
 * draft_len       device int32 [B] with L_b in [0, K], or NULL for L_b = K.
 *                 Positions >= L_b (and target positions > L_b) are never read.
 * temperature     > 0, finite; logits are divided by it before the softmax.
 * top_p           in (0, 1]; 1 switches the nucleus filter off.
 * seed            64-bit Philox key.
 * out_tokens      device int32 [B, K+1], contiguous: the n_b accepted drafted
 *                 ids, then the resampled or bonus token, then -1.
 * out_n_accepted  device int32 [B]: n_b in [0, L_b], or -1 for an invalid row
 *                 (-2: see Concurrency above; not otherwise possible).
 * stream          hipStream_t to run on (NULL = the default stream).
 *
 * Errors: arguments the host can check return SV_EINVAL / SV_ESHAPE /
 * SV_EDTYPE / SV_EALIGN and launch nothing;
 * SV_ECAPTURE as described under Graphs.  Data errors cannot be reported
 * synchronously: a row whose L_b lies outside [0, K], whose drafted id at some
 * j < L_b lies outside [0, V), or one of whose needed logit rows holds a NaN, a
 * +inf or only -inf, gets out_n_accepted = -1 and out_tokens = -1 throughout.
 * Launch failures return SV_EHIP.
 */
int spec_verify(const sv_logits* target_logits, const sv_logits* draft_logits,
                const int32_t* draft_tokens, const int32_t* draft_len,
                float temperature, float top_p, uint64_t seed,
                int32_t* out_tokens, int32_t* out_n_accepted, void* stream);

/*
 * spec_verify_noalloc -- spec_verify for callers that cannot allocate device
 * memory (code being captured into a HIP graph, tight serving loops, hosts
 * that forbid allocation).  Same arguments, kernels and outputs as
 * spec_verify, but the scratch (statistics records, row states, candidate
 * lists, row-pass records) lives in one fixed device array of
 * SPECVERIFY_NOALLOC_SCRATCH_BYTES per device, held until the process ends,
 * so no call allocates or frees anything.  A call needing more scratch
 * returns SV_ETOOBIG and launches nothing (B = 64, K = 5, V = 128256 needs
 * about 0.4 MiB, 12.5 MiB with top-p).  Every call on a device shares that
 * device's array: calls that overlap on one device (different streams, or
 * threads) race and must not be issued; each call rewrites, before reading,
 * all the scratch it uses, so nothing needs clearing between calls.  Errors
 * otherwise as spec_verify.
 */
#define SPECVERIFY_NOALLOC_SCRATCH_BYTES (16 << 20)
int spec_verify_noalloc(const sv_logits* target_logits, const sv_logits* draft_logits,
                        const int32_t* draft_tokens, const int32_t* draft_len,
                        float temperature, float top_p, uint64_t seed,
                        int32_t* out_tokens, int32_t* out_n_accepted, void* stream);

/*
 * spec_verify_probe -- spec_verify plus the intermediate values behind each
 * decision, for testing.  probe_pos: device float64 [B, K+1, SV_PROBE_POS];
 * probe_row: device float64 [B, SV_PROBE_ROW]; layouts above.  Same errors as
 * spec_verify; the probe pointers must not be NULL.
 */
int spec_verify_probe(const sv_logits* target_logits, const sv_logits* draft_logits,
                      const int32_t* draft_tokens, const int32_t* draft_len,
                      float temperature, float top_p, uint64_t seed,
                      int32_t* out_tokens, int32_t* out_n_accepted,
                      double* probe_pos, double* probe_row, void* stream);

/*
 * spec_greedy_verify -- greedy verify: the temperature -> 0 limit of
 * spec_verify (page "Speculative Decoding للمحترف", section "المفهوم بالتقريب":
 * accept the drafted tokens the target agrees with, take the target's token at
 * the first disagreement), plus the k ids that rank after the emitted token
 * in the logits it came from (the LogitSpec page, gist.science 2507.01449,
 * section 2: candidates for the token after next; the page uses k = 60).
 *
 * target_logits   [B, K+1, V] target logits, bf16 or fp32; 1 <= K <= 16.
 * draft_tokens, draft_len: as for spec_verify (no draft logits are needed).
 * k               0 <= k <= 64.
 * out_tokens      device int32 [B, K+1]: the n accepted ids, the target's
 *                 argmax at position n (ties to the lower id), then -1.
 * out_n_accepted  device int32 [B]: n = the first j < L_b whose drafted id is
 *                 not the target's argmax (L_b if none), -1 for an invalid row.
 * out_topk        device int32 [B, k] (NULL when k = 0): the ids ranked 2..k+1
 *                 by logit at position n (descending, ties to the lower id),
 *                 -1 past V.
 *
 * Invalid rows (as for spec_verify, on the target rows 0..L_b) give n = -1
 * and -1 in every output.  Errors as spec_verify, SV_EINVAL for k outside
 * [0, 64] or out_topk NULL with k > 0.
 */
int spec_greedy_verify(const sv_logits* target_logits, const int32_t* draft_tokens,
                       const int32_t* draft_len, int32_t k, int32_t* out_tokens,
                       int32_t* out_n_accepted, int32_t* out_topk, void* stream);

/*
 * spec_hispec_verify -- the two-stage (hierarchical) verify step (page
 * "HiSpec: Hierarchical Speculative Decoding for LLMs", section 2: an
 * early-exit model's intermediate layer verifies the drafts first and rejects
 * early; the final layer verifies what passed; applying the lossless rule in
 * both stages makes the output follow the final layer exactly).
 *
 * final_logits    [B, K+2, V] final-layer logits at the positions of the
 *                 provisional sequence (positions past n1 + 1 are not read).
 * inter_logits    [B, K+1, V] intermediate-layer logits.
 * draft_logits    [B, K, V] draft-layer logits; all three the same dtype, B
 *                 and V; 1 <= K <= 15.
 * draft_tokens, draft_len, temperature, top_p, seed: as for spec_verify.
 * out_tokens      device int32 [B, K+2]: the n accepted tokens, then the
 *                 final layer's corrected or bonus token, then -1.
 * out_n_accepted  device int32 [B]: n (stage 2's accepted count), -1 for an
 *                 invalid row.
 * out_n_stage1    device int32 [B] or NULL: n1, the drafts the intermediate
 *                 layer accepted.
 *
 * Stage 1 is spec_verify(inter, draft): n1 accepted drafts and one token.
 * Stage 2 is spec_verify(final, inter) on those n1 + 1 tokens, with its
 * uniforms from Philox counter (row, position, 1, 0).  Errors as spec_verify.
 */
int spec_hispec_verify(const sv_logits* final_logits, const sv_logits* inter_logits,
                       const sv_logits* draft_logits, const int32_t* draft_tokens,
                       const int32_t* draft_len, float temperature, float top_p,
                       uint64_t seed, int32_t* out_tokens, int32_t* out_n_accepted,
                       int32_t* out_n_stage1, void* stream);

/*
 * spec_smc_step -- one reweight-and-resample step of SMC-SD over N particles
 * (page "Faster LLM Inference via Sequential Monte Carlo", section 2: every
 * particle is extended by K draft tokens and scored by the target, which also
 * yields one bonus token per particle; importance weights follow the ratio of
 * target to draft probabilities; when the effective sample size falls below a
 * threshold the particles are resampled).
 *
 * target_logits   [N, K+1, V] target logits, bf16 or fp32 (B of the
 *                 descriptor = N particles).
 * draft_logits    [N, K, V] draft logits, same dtype, N and V; 1 <= K <= 16.
 * draft_tokens    device int32 [N, K], contiguous: each particle's K drafted ids.
 * logw_in         device float64 [N]: log-weights before the step (any
 *                 common offset; -inf marks a dead particle).
 * temperature     > 0, finite; divides both models' logits (no top-p).
 * ess_fraction    resample when ESS < ess_fraction * N (0.5 is the usual
 *                 choice; <= 0 never, > 1 always resamples); not NaN.
 * seed            64-bit Philox key.  Bonus draw of particle i: word 1 of
 *                 counter (i, K, 0, 0), as the verify step's bonus; systematic
 *                 resampling offset u0: word 0 of counter (0, 0, 1, 0).
 * out_bonus       device int32 [N]: the bonus token drawn from the target at
 *                 position K by inverse CDF; -1 for an invalid particle.
 * out_logw        device float64 [N]: logw_in + sum_j (log p_j(x_j) -
 *                 log q_j(x_j)); all 0 after a resampling; -inf for an invalid
 *                 particle.  May be the same buffer as logw_in.
 * out_ancestor    device int32 [N]: the particle that slot k continues (k
 *                 itself without resampling; systematic: the first particle
 *                 whose cumulative normalised weight exceeds (k + u0)/N).
 * out_ess         device float64 [1]: (sum w)^2 / sum w^2 before resampling,
 *                 w = exp(logw - max); 0 when no particle is valid.
 * out_resampled   device int32 [1]: 1 if the step resampled.
 * stream          hipStream_t to run on (NULL = the default stream).
 *
 * A particle is invalid when a drafted id lies outside [0, V), a needed logit
 * row holds a NaN, a +inf or only -inf, or its input log-weight is NaN or
 * +inf; it never becomes an ancestor.  Host-checkable errors return
 * SV_EINVAL / SV_ESHAPE / SV_EDTYPE / SV_EALIGN and launch nothing.
 */
int spec_smc_step(const sv_logits* target_logits, const sv_logits* draft_logits,
                  const int32_t* draft_tokens, const double* logw_in,
                  float temperature, double ess_fraction, uint64_t seed,
                  int32_t* out_bonus, double* out_logw, int32_t* out_ancestor,
                  double* out_ess, int32_t* out_resampled, void* stream);

/*
 * spec_draft_produce -- the synthetic draft producer of the two-batch
 * schedule (page "MineDraft: A Framework for Batch Parallel Speculative
 * Decoding", section 2: two batches alternate, one verified while the other
 * is drafted, roles swapping every step).  The pages give no drafter; this
 * stand-in derives a batch's drafts from its target logits so that a caller
 * can run it on one stream while spec_verify runs on another:
 *
 *   draft[b, j, v] = round(float32(target[b, j, v]) + delta(b, j, v)), j < K,
 *   delta = ((h >> 5) - 1024) / 512 with h the 16-bit half (v & 1; 0 = low)
 *   of word (v & 7) >> 1 of Philox4x32-10 at counter (v >> 3, b, j, 3), key
 *   (seed low, seed high); round = round to nearest even into the logits'
 *   format (NaN stays NaN);
 *   out_tokens[b, j] = the lowest id holding the largest draft[b, j, :], or
 *   -1 when that row holds a NaN (a greedy drafter).
 *
 * target_logits  [B, P, V], bf16 or fp32; positions 0..K-1 are read.
 * K              1 <= K <= P.
 * draft_out      device buffer of the target's dtype, written at element
 *                b*out_stride_b + j*out_stride_p + v (strides in elements,
 *                >= 0); its rows must not overlap one another or the
 *                target (the library does not check this).
 * out_tokens     device int32 [B, K], contiguous.
 *
 * Errors as spec_verify: SV_EINVAL (NULL pointer, negative stride),
 * SV_ESHAPE (K outside [1, P], B or V out of range), SV_EDTYPE, SV_EALIGN,
 * SV_ENOMEM, SV_EHIP; nothing is launched on a host-checked error.  Uses the
 * stream's scratch like every other call: calls on one stream run in order.
 */
int spec_draft_produce(const sv_logits* target_logits, int32_t K, uint64_t seed,
                       void* draft_out, int64_t out_stride_b, int64_t out_stride_p,
                       int32_t* out_tokens, void* stream);

/*
 * ---- The tree round --------------------------------------------------------
 *
 * Drafts that form a tree (page "LogitSpec", gist.science 2507.01449, section
 * 2: a draft tree with its attention mask; a chain is the tree whose parent of
 * node i is node i - 1) over a paged key/value cache (page "HiSpec", section 2:
 * block tables; page "Faster LLM Inference via Sequential Monte Carlo",
 * section 2: particles that share and copy cache pages):
 *
 *   spec_tree_attention   every node attends to the cache and its ancestors;
 *   spec_verify_tree      the target's probabilities accept a path of the tree;
 *   spec_cache_commit     the accepted path's rows go into the cache;
 *   spec_cache_fork       the slots of a batch continue their ancestors (the
 *                         out_ancestor of spec_smc_step), or are freed.
 *
 * A tree has N <= SPECVERIFY_MAX_NODES nodes.  Node 0 is the last token of the
 * sequence, whose keys and values are not in the cache yet; node i > 0 is a
 * drafted token after node parent[i] < i.  Level order is not required.
 *
 * A sequence's cache is its row of the block table: row j of the sequence lies
 * in slot j % page_size of page table[j / page_size].
 *
 * These calls take a workspace from the caller (its size from the functions
 * below; contents need no preparation and mean nothing after the call), so
 * they never allocate and any of them may be captured.  Two calls that may run
 * at the same time, captured ones included, need workspaces of their own.
 */
#define SPECVERIFY_MAX_NODES 64
#define SPECVERIFY_MAX_PAGES (1 << 20)
enum { SV_F16 = 2 };  /* a dtype of the attention and the cache */

/*
 * spec_tree_attention -- for every sequence b, node i and query head e,
 *
 *   out[b, i, e] = sum_j softmax_j(scale * q[b, i, e] . k_j) v_j
 *
 * over the cache rows j < len[b] of key head e / (heads / kv_heads) and over
 * the nodes j that are i or one of its ancestors.  Softmax statistics and sums
 * are float32; the weights are rounded to the input type before they meet V
 * (fp16: absolutely, by at most 2^-32 of the row's largest weight, where they
 * are below 2^-21 of it).
 *
 * With window > 0, node i at depth d has position len + d and sees the cache
 * rows with len + d - j < window, the first `sinks` cache rows, and the nearest
 * `window` of itself and its ancestors.  window = 0: everything.
 *
 * dtype          SV_BF16 or SV_F16, of all tensors.
 * B, N           1 <= B <= 65536 sequences, 1 <= N <= 64 nodes; B * kv_heads
 *                below 2^24, and with t = N * heads / kv_heads / 128, rounded
 *                up, above 1: B * kv_heads, rounded up to eights, times t too.
 * heads, kv_heads  query and key heads; heads <= 1024, a multiple of kv_heads.
 * dim            a multiple of 8, at most 128.
 * q, out         [B, N, heads, dim]; k_tree, v_tree [B, N, kv_heads, dim];
 *                strides in elements for (sequence, node, head).
 * k_cache, v_cache  [pages, page_size, kv_heads, dim]; strides for (page,
 *                slot, head); page_size a power of two, at most 1024.
 *                The last axis of every tensor is contiguous; data and strides
 *                are multiples of 16 bytes; strides are >= 0, below 64 GB; those of
 *                axes of one are not looked at.
 * table          device int32 [B, width], row stride table_stride.  An entry
 *                outside [0, pages) hides its rows.  width * page_size <= 2^28
 *                (with 1024 key heads of more than 32 rows each, 2^28 - 64).
 * len            device int32 [B], rows in the cache (clamped to [0, width *
 *                page_size]).
 * parent         device int32 [B, N], contiguous; parent[b, 0] is not read.  A
 *                parent outside [0, i) ends the line: node i has no ancestors.
 * n_nodes        device int32 [B] or NULL (N for all), clamped to [0, N].  The
 *                output of an absent node is zero.
 * scale          finite.
 * workspace      at least spec_tree_attention_workspace(args) bytes, aligned
 *                to 16 bytes (may be NULL if that is 0).
 *
 * What a node does not see never reaches its output, whatever it holds (NaN
 * and infinities included).  out must not overlap the inputs, nor its rows each
 * other.
 *
 * Errors: SV_EINVAL (NULL, negative stride, out with a stride of 0 along an
 * axis longer than one, scale not finite, window or sinks < 0),
 * SV_ESHAPE, SV_EDTYPE, SV_EALIGN, SV_ETOOBIG (workspace too small), SV_EHIP.
 */
typedef struct {
    int32_t dtype;
    int32_t B, N, heads, kv_heads, dim;
    const void* q;
    int64_t q_stride[3];
    const void* k_tree;
    const void* v_tree;
    int64_t k_tree_stride[3], v_tree_stride[3];
    const void* k_cache;
    const void* v_cache;
    int64_t k_cache_stride[3], v_cache_stride[3];
    int32_t pages, page_size, width;
    const int32_t* table;
    int64_t table_stride;
    const int32_t* len;
    const int32_t* parent;
    const int32_t* n_nodes;
    float scale;
    int32_t window, sinks;
    void* out;
    int64_t out_stride[3];
    void* workspace;
    int64_t workspace_bytes;
} sv_tree_attention;

int spec_tree_attention(const sv_tree_attention* args, void* stream);

/* Bytes of workspace the call needs, from its sizes (pointers are not looked
 * at); a negative status for sizes the call refuses. */
int64_t spec_tree_attention_workspace(const sv_tree_attention* args);

/*
 * spec_verify_tree -- verification of a tree of drafted tokens against the
 * target's probabilities, from given random numbers: for callers with their
 * own sampler (penalties, top-k, grammars), whose distributions are not the
 * tempered softmax spec_verify computes.  With p and q the target's and the
 * draft's row at the current node (node 0 at first), its children are tested
 * in the order of their numbers:
 *
 *   with draft_probs (children drawn independently from q; the acceptance rule
 *   and the corrected distribution of spec_verify, applied again after every
 *   refusal to what is left of p):
 *       accept x iff  u S q(x) < p(x) - a q(x);  a = 0, S = 1 at first, after
 *       a refusal a += S and S = sum_v max(0, p(v) - a q(v));
 *   without (children chosen, not drawn): accept x iff u S < p(x); a refusal
 *       takes p(x) out of S and x out of p; x refused before is refused again.
 *
 * An accepted child becomes the current node.  Where all are refused, or there
 * are none, one more token is drawn by inverse CDF in id order at u_final from
 * what is left: max(0, p - a q), or p without the refused ids (p itself where
 * nothing is left of it).  All in float64.
 *
 * target_probs   [B, N, V] (the descriptor's P = N <= 64): row i the target's
 *                distribution after node i.  fp32 or bf16.  V <= SPECVERIFY_MAX_V.
 * draft_probs    [B, P, V], same dtype, P <= N: row i the distribution the
 *                children of node i were drawn from; or NULL.
 * tokens         device int32 [B, N]: the nodes' ids (node 0's is not read).
 * parent         device int32 [B, N] (node 0's is not read).
 * n_nodes        device int32 [B] or NULL (N for all).
 * u_accept       device float32 [B, N]: node i's uniform (node 0's is not read).
 * u_final        device float32 [B].
 * out_tokens     device int32 [B, N]: the n accepted ids, the last token, -1.
 * out_nodes      device int32 [B, N]: the path: node 0, the n accepted nodes, -1.
 * out_n_accepted device int32 [B]: n.
 *                Outputs must not overlap the inputs or each other.  B < 2^22.
 *
 * A sequence is invalid (n = -1 and -1 throughout) when n_nodes lies outside
 * [1, N], a node's parent outside [0, i) (with draft_probs, outside [0, P)),
 * its id outside [0, V), its uniform or u_final outside [0, 1), or when a
 * probability at a drafted id, or in a row that is read whole (the last node's
 * row, and rows whose S is needed), is negative, infinite or NaN, or the last
 * row has no positive entry.
 *
 * workspace      at least spec_verify_tree_workspace bytes, aligned to 8.
 *
 * Errors as spec_verify, SV_ETOOBIG for too small a workspace.
 */
int spec_verify_tree(const sv_logits* target_probs, const sv_logits* draft_probs, const int32_t* tokens,
                     const int32_t* parent, const int32_t* n_nodes, const float* u_accept, const float* u_final,
                     int32_t* out_tokens, int32_t* out_nodes, int32_t* out_n_accepted, void* workspace,
                     int64_t workspace_bytes, void* stream);

/* Bytes of workspace the call needs, by its sizes and whether it has
 * draft_probs; 0 for large batches and without them (then NULL will do). */
int64_t spec_verify_tree_workspace(int32_t B, int32_t N, int32_t V, int32_t dtype, int32_t draft);

/*
 * A paged cache of `layers` layers and the block tables of B sequences.  The
 * tables are the whole state: a page is in use exactly if a live entry (one of
 * the first ceil(len / page_size) of a row) names it, and free otherwise.
 */
typedef struct {
    void* k;                /* [layers, pages, page_size, heads, dim] */
    void* v;
    int32_t dtype;          /* SV_F32, SV_BF16 or SV_F16; rows are moved, not computed with */
    int32_t layers, pages, page_size, heads, dim;
    int64_t k_stride[4], v_stride[4];  /* layer, page, slot, head */
    const int32_t* table;   /* [B, width], row stride table_stride */
    int64_t table_stride;
    const int32_t* len;     /* [B] */
    int32_t B, width;
} sv_cache;

/*
 * spec_cache_commit -- append the accepted path of every sequence's tree:
 * rows nodes[b, 0..n] of k_tree, v_tree ([layers, B, N, heads, dim], strides
 * for layer, sequence, node, head) become the cache rows len..len+n, for n =
 * n_accepted[b]; a negative n appends nothing.  nodes NULL: rows 0..n (a
 * chain: the out_n_accepted of spec_verify).  A partly filled last page is
 * filled up, and further pages are taken lowest free page first, in the order
 * of the sequences.  A partly filled last page that is appended to must be
 * named by no other live entry (spec_cache_fork leaves it so).
 *
 * out_table [B, width] (row stride out_stride) and out_len [B] receive the new
 * tables, -1 behind the live entries; they may be table and len themselves
 * (same stride), and must not overlap them otherwise.
 *
 * out_status  device int32 [1]: 0; or the number of pages that were lacking;
 *             or -1 when a length, count, node or live page number is out of
 *             range, a table row too short, or a partly filled page that is to
 *             be appended to is shared.  Unless 0, nothing is appended and
 *             tables and lengths go out as they came in.
 *
 * dim * element size, strides (of axes longer than one) and data are multiples of 16 bytes; pages <=
 * SPECVERIFY_MAX_PAGES; page_size a power of two, at most 1024; B, layers <=
 * 65534; width * page_size <= 2^28; a page, and a sequence's N rows, of one layer
 * at most 16 GB.  The cache's rows must not overlap each other or the tree's (a stride of
 * 0 along an axis of the cache longer than one is refused).  workspace:
 * spec_cache_workspace bytes.
 */
int spec_cache_commit(const sv_cache* cache, const void* k_tree, const void* v_tree, const int64_t k_tree_stride[4],
                      const int64_t v_tree_stride[4], int32_t N, const int32_t* nodes, const int32_t* n_accepted,
                      int32_t* out_table, int64_t out_stride, int32_t* out_len, int32_t* out_status, void* workspace,
                      int64_t workspace_bytes, void* stream);

/*
 * spec_cache_fork -- slot k continues sequence ancestor[k] (its own: k; -1:
 * the slot is freed).  Full pages are shared; a partly filled last page stays
 * with the lowest slot that continues its sequence and is copied, in every
 * layer, to the lowest free pages for the others.  Pages that no slot names
 * any more are free.  Outputs, status and limits as spec_cache_commit, with
 * out_table and out_len apart from table and len.
 */
int spec_cache_fork(const sv_cache* cache, const int32_t* ancestor, int32_t* out_table, int64_t out_stride,
                    int32_t* out_len, int32_t* out_status, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace a commit of at most N rows per sequence, or a fork (N =
 * 0), needs. */
int64_t spec_cache_workspace(int32_t B, int32_t N, int32_t page_size);

/*
 * ---- Latent rows -----------------------------------------------------------
 *
 * Models whose heads share one row per token: its first elements are the latent
 * vector that keys and values are made of, the rest a part that carries
 * positions.  A paged cache holds that row only, [pages, page_size, dim].  It is
 * committed and forked like any cache (spec_cache_commit, spec_cache_fork), its
 * row's two halves given as k and v.
 */
#define SPECVERIFY_MAX_LATENT 576

/*
 * spec_latent_attention -- attention on the rows themselves (the absorbed form:
 * queries multiplied into the latent space, results to be multiplied out of
 * it; spec_head_product does both).  For every sequence b, node i and head e,
 *
 *   out[b, i, e] = sum_j softmax_j(scale * q[b, i, e] . c_j) c_j[0 .. dim_v)
 *
 * over the cache rows j < len[b] and the nodes j that are i or one of its
 * ancestors, c_j their rows.  Trees, tables and lengths are spec_tree_attention's,
 * and so are statistics and roundings.
 *
 * dtype          SV_BF16 or SV_F16, of all tensors.
 * B, N           1 <= B <= 65536 sequences, 1 <= N <= 64 nodes.
 * heads          at most 1024; B, rounded up to eights, times N * heads / 64, rounded up, below 2^23.
 * dim, dim_v     multiples of 8; dim <= SPECVERIFY_MAX_LATENT, dim_v <= dim and 512.
 * q              [B, N, heads, dim]; out [B, N, heads, dim_v]; strides in
 *                elements for (sequence, node, head).
 * rows           [B, N, dim], the nodes' own rows (not in the cache yet);
 *                strides for (sequence, node).
 * cache          [pages, page_size, dim]; strides for (page, slot).
 *                The last axis of every tensor is contiguous; data and strides
 *                are multiples of 16 bytes; strides as spec_tree_attention's.
 * table, table_stride, len, n_nodes, width, scale, workspace  as spec_tree_attention.
 * parent         device int32 [B, N], or NULL: node i's parent is node i - 1.
 *
 * What a node does not see never reaches its output.  A node that sees a node
 * (itself included) with an infinity or NaN among its row's first dim_v elements
 * gets NaN.  The output of an absent node is zero.  out must not overlap the
 * inputs, nor its rows each other.
 *
 * Errors as spec_tree_attention.
 */
typedef struct {
    int32_t dtype;
    int32_t B, N, heads, dim, dim_v;
    const void* q;
    int64_t q_stride[3];
    const void* rows;
    int64_t rows_stride[2];
    const void* cache;
    int64_t cache_stride[2];
    int32_t pages, page_size, width;
    const int32_t* table;
    int64_t table_stride;
    const int32_t* len;
    const int32_t* parent;
    const int32_t* n_nodes;
    float scale;
    void* out;
    int64_t out_stride[3];
    void* workspace;
    int64_t workspace_bytes;
} sv_latent_attention;

int spec_latent_attention(const sv_latent_attention* args, void* stream);

/* Bytes of workspace the call needs, from its sizes (pointers are not looked
 * at); a negative status for sizes the call refuses. */
int64_t spec_latent_attention_workspace(const sv_latent_attention* args);

/*
 * spec_head_product -- a product per head, out[t, h, m] = sum_k x[t, h, k]
 * w[h, m, k]: queries into the latent space (w: the key weights, transposed
 * once to [heads, latent, dim_k]) and results out of it (w: the value weights
 * [heads, dim_v, latent]).  Sums are float32, rounded once.
 *
 * dtype          SV_BF16 or SV_F16, of all tensors.
 * T              tokens, 0 (nothing is done) to 2^24; heads <= 1024; K and M
 *                multiples of 8, at most 65536; tiles of 128 outputs by 128
 *                tokens (32 where T <= 32), over the heads, fewer than 2^24 - 8.
 * x, out         [T, heads, K], [T, heads, M], strides for (token, head); w
 *                [heads, M, K], strides for (head, row).  The last axis of every
 *                tensor is contiguous; data and strides are multiples of 16
 *                bytes.  out must not overlap the inputs, nor its rows each other.
 *
 * Errors: SV_EINVAL (NULL, negative stride, out with a stride of 0 along an axis
 * longer than one), SV_ESHAPE, SV_EDTYPE, SV_EALIGN, SV_EHIP.
 */
typedef struct {
    int32_t dtype;
    int32_t T, heads, K, M;
    const void* x;
    int64_t x_stride[2];
    const void* w;
    int64_t w_stride[2];
    void* out;
    int64_t out_stride[2];
} sv_head_product;

int spec_head_product(const sv_head_product* args, void* stream);

/*
 * spec_latent_prompt -- attention of prompts (the expanded form): keys and values
 * are made of the cache rows per head, for row s of a sequence
 *
 *   k_s = (w_k[h] c_s, e_s),  v_s = w_v[h] c_s,
 *
 * c_s the row's first `latent` elements and e_s the dim_p behind them, and a
 * token at position p attends to rows 0..p:
 *
 *   out[t, h] = sum_{s <= p} softmax_s(scale * q[t, h] . k_s) v_s.
 *
 * The rows q_start[b] .. q_start[b + 1] of q are the last tokens of sequence b, at
 * positions len[b] - n .. len[b] - 1; their rows, and those of a prefix before
 * them, are in the cache.  Keys are rounded to the input type; values and weights
 * to float16's 11 bits in either type.  A row's values (per head) are kept times a
 * power of two where the largest finite one lies outside [2^-14, 2^11): a value's
 * error is half a step, or 2^-15 of that largest one where this is more; that of a
 * weight times its row's power, half a step or 2^-32 of the largest such product that
 * the token sees.  Statistics are float32.
 *
 * dtype          SV_BF16 or SV_F16, of all tensors.
 * T              query tokens, 0 (nothing is done) to 2^24; B <= 65536; heads <= 1024.
 * dim_k, dim_v   at most 128, dim_p at most 64, latent + dim_p <=
 *                SPECVERIFY_MAX_LATENT; multiples of 8; dim_p may be 0.
 * rows           at least the sum of the lengths, at most 2^26: the caller's
 *                bound, by which the workspace is sized.  The output of a
 *                sequence that does not fit is NaN.
 * q, out         [T, heads, dim_k + dim_p], [T, heads, dim_v]; strides for
 *                (token, head).
 * cache          [pages, page_size, latent + dim_p]; strides for (page, slot).
 * w_k, w_v       [heads, dim_k, latent], [heads, dim_v, latent]; strides for
 *                (head, row).  Data and strides of all these are multiples of
 *                16 bytes, last axes contiguous.
 * table, table_stride, len, width, scale  as spec_tree_attention.
 * q_start        device int32 [B + 1], rising within [0, T]; a sequence whose
 *                bounds do not rise so has no queries (no two sequences may share
 *                rows of q).  Rows of out that belong to no sequence are left as they
 *                are; a query that sees nothing is zero.
 * workspace      at least spec_latent_prompt_workspace(args) bytes, aligned to 16:
 *                about 2 heads rows (dim_k + dim_v), as the keys and values of all
 *                rows, the prefixes' too, are made by every call.
 *
 * What a token does not see (later rows, other sequences, pages outside the pool)
 * never reaches its output.  Where it sees infinities or NaN, expanded keys beyond
 * the type's range included, its output is infinite or NaN.  (Launches have fewer
 * than 2^32 threads: the 128-row tiles of `rows` times the 128-wide tiles of heads *
 * dim_k and of heads * dim_v, and (T / 128 + min(B, T)) * heads, are below 2^24 - 8.)
 *
 * Errors as spec_tree_attention.
 */
typedef struct {
    int32_t dtype;
    int32_t T, B, heads, latent, dim_k, dim_p, dim_v, rows;
    const void* q;
    int64_t q_stride[2];
    const void* cache;
    int64_t cache_stride[2];
    int32_t pages, page_size, width;
    const int32_t* table;
    int64_t table_stride;
    const int32_t* len;
    const int32_t* q_start;
    const void* w_k;
    int64_t w_k_stride[2];
    const void* w_v;
    int64_t w_v_stride[2];
    float scale;
    void* out;
    int64_t out_stride[2];
    void* workspace;
    int64_t workspace_bytes;
} sv_latent_prompt;

int spec_latent_prompt(const sv_latent_prompt* args, void* stream);

/* Bytes of workspace the call needs, from its sizes; a negative status for sizes
 * the call refuses. */
int64_t spec_latent_prompt_workspace(const sv_latent_prompt* args);

/*
 * spec_cache_reserve -- room for n_new[b] more rows of every sequence (new
 * requests' prompts, behind a length of 0; the next token of running ones) and
 * where these rows go.  A partly filled last page is filled up, further pages are
 * taken lowest free page first, in the order of the sequences; a page is in use
 * if a live entry of the tables names it.
 *
 * table, len     device int32 [B, width] (row stride table_stride) and [B].
 * n_new          device int32 [B]; a negative count is 0.
 * pages, page_size, width  the cache's (no tensor is needed); limits as spec_cache_commit's.
 *                B <= 65534; B * (width / 64 + 1) < 2^31.
 * rows           the length of the lists below: at least the sum of the counts.
 * out_table, out_len  as spec_cache_commit's: the new tables, -1 behind the live
 *                entries, and lengths; they may be table and len themselves.
 * out_start      device int32 [B + 1]: sequence b's new rows are entries
 *                out_start[b] .. out_start[b + 1] of the lists.
 * out_slots, out_position  device int32 [rows]: the new rows' slots, page *
 *                page_size + place in the page, and their positions in the
 *                sequence (its old length on); -1 behind the last one.
 * out_status     device int32 [1]: 0; the number of pages that were lacking; or -1
 *                when a length, a live page number or `rows` is out of range, a
 *                table row too short, or a partly filled page that is to be
 *                appended to is named by another live entry.  Unless 0, tables
 *                and lengths go out as they came in, out_start is 0 and the lists -1.
 * workspace      at least spec_cache_reserve_workspace bytes, aligned to 4.
 *
 * Outputs must not overlap each other, nor (but for the two that may be) the
 * inputs.  Errors as spec_cache_commit.
 */
int spec_cache_reserve(const int32_t* table, int64_t table_stride, const int32_t* len, const int32_t* n_new, int32_t B,
                       int32_t width, int32_t pages, int32_t page_size, int32_t rows, int32_t* out_table,
                       int64_t out_stride, int32_t* out_len, int32_t* out_start, int32_t* out_slots,
                       int32_t* out_position, int32_t* out_status, void* workspace, int64_t workspace_bytes,
                       void* stream);

int64_t spec_cache_reserve_workspace(int32_t B, int32_t page_size, int32_t rows);

/*
 * spec_cache_write -- row t of `a`, and row t of `b` behind it, become the cache row
 * in slot slots[t]; a slot outside the cache (-1) takes nothing.  For latent rows a
 * is the latent part and b the part that carries positions; dim_b may be 0 (b is
 * not looked at).  No two tokens may have the same slot, and a and b must not
 * overlap the cache.
 *
 * cache          [pages, page_size, dim_a + dim_b], strides for (page, slot); a
 *                [T, dim_a], b [T, dim_b], strides between rows; SV_F32, SV_BF16 or
 *                SV_F16.  Dimensions (at most 65536), strides and data are multiples of
 *                16 bytes.  0 <= T <= 2^28.
 * slots          device int32 [T].
 *
 * Errors: SV_EINVAL (NULL, negative stride, a stride of 0 in the cache), SV_ESHAPE,
 * SV_EDTYPE, SV_EALIGN, SV_EHIP.
 */
typedef struct {
    void* cache;
    int64_t cache_stride[2];
    int32_t dtype, pages, page_size;
    int32_t T, dim_a, dim_b;
    const void* a;
    int64_t a_stride;
    const void* b;
    int64_t b_stride;
    const int32_t* slots;
} sv_cache_rows;

int spec_cache_write(const sv_cache_rows* args, void* stream);

/*
 * ---- Beam search -----------------------------------------------------------
 *
 * spec_beam_select -- the W best continuations of a sequence's W beams.  Beam w's
 * candidates are the ids v with a logit above -inf, at
 *
 *   scores[b, w] + x[v] - log sum_u exp(x[u]),  x = logits[b, w],
 *
 * and a finished beam has one, the token `end` at scores[b, w].  The W largest come
 * out best first: by the scores in float64, equal ones by beam, then within a beam by
 * logit (also where float64 scores cannot tell two apart), then by id; with equal
 * logits that is the order of w * V + v.  A beam whose score is -inf (at the first
 * step all but one), +inf or NaN, or whose logits hold a NaN, +inf or nothing above
 * -inf, has no candidates; its logits are not read where the score is -inf or the
 * beam finished.
 *
 * logits         [B, W, V] (the descriptor's P = W <= SPECVERIFY_MAX_BEAMS); B * W <=
 *                65535, V <= 2^24.
 * scores         device float32 [B, W].
 * finished       device int32 [B, W], non-zero: finished; or NULL.
 * end            the token that finishes a beam, or -1 (then finished is NULL).
 * out_tokens     device int32 [B, W].
 * out_ancestor   device int32 [B * W]: b * W + the beam continued, as
 *                spec_cache_fork and spec_beam_reorder take it.
 * out_scores     device float32 [B, W], rounded once.  The logarithm is off by at most
 *                2^-20 of the share of probability that the ids beside the beam's
 *                first one have (by a float64 rounding where two beams' candidates are
 *                close, as these sums are taken again).
 * out_finished   device int32 [B, W]: 1 where the token is `end` or the beam was finished.
 *                Where there are fewer candidates than beams: -1, -1, -inf and 0.
 *                Outputs must not overlap the inputs or each other.
 * workspace      at least spec_beam_workspace bytes, aligned to 8.
 *
 * Errors as spec_verify, SV_ETOOBIG for too small a workspace.
 */
#define SPECVERIFY_MAX_BEAMS 64
int spec_beam_select(const sv_logits* logits, const float* scores, const int32_t* finished, int32_t end,
                     int32_t* out_tokens, int32_t* out_ancestor, float* out_scores, int32_t* out_finished,
                     void* workspace, int64_t workspace_bytes, void* stream);

int64_t spec_beam_workspace(int32_t B, int32_t W, int32_t V);

/*
 * spec_beam_reorder -- row k of dst becomes row ancestor[k] of src (a beam's
 * history, or any state kept by rows; pages follow by spec_cache_fork).  Rows are
 * row_bytes long, strides are in bytes; an ancestor outside [0, rows) makes row k
 * of dst zero.  src and dst must not overlap, nor the rows of dst each other;
 * rows that lie at multiples of 16 bytes are the fastest.  rows <= 65535.
 *
 * Errors: SV_EINVAL (NULL, src == dst, a negative stride, rows of dst that overlap),
 * SV_ESHAPE, SV_EALIGN (ancestor), SV_EHIP.
 */
int spec_beam_reorder(const void* src, int64_t src_stride, void* dst, int64_t dst_stride, int64_t row_bytes,
                      int32_t rows, const int32_t* ancestor, void* stream);

/* Human-readable text for a status code (for SV_EHIP, the last HIP error). */
const char* spec_verify_strerror(int status);

/* Frees every cached scratch buffer.  The caller must ensure no call is in
 * flight on any stream. */
void spec_verify_release(void);

/* Returns SPECVERIFY_ABI_VERSION. */
int spec_verify_abi_version(void);

/* Kernel timing for measurement.  While enabled, every launch carries a pair
 * of HIP events on its stream, attached to the kernel's dispatch.
 * spec_verify_profile_read synchronises those events and writes, for each of
 * the n kernel kinds (0 statistics pass, 1 nucleus selection, 2 row pass:
 * decision and resample, or the SMC particle pass, 3 SMC resampling, 4 the
 * synthetic draft producer, 5 tree attention, 6 its join, 7 the clearing of tree
 * verification's workspace, 8 tree verification, 9 cache plan, 10 cache copies, 11
 * latent attention, 12 its join, 13 products per head, 14 the prompts' places, 15
 * their keys and values, 16 their rows' powers of two and the values of such rows
 * once more, 17 the prompts' attention, 18 beam statistics, 19 beam selection, 20
 * reordered rows, 21 reservation plan, 22 its outputs, 23 rows into their slots), the
 * summed duration in milliseconds and the number of launches since the last read; it
 * returns the number of kinds written.  Host arrays ms[n], launches[n]. */
int spec_verify_profile_enable(int enable);
int spec_verify_profile_read(double* ms, int64_t* launches, int n);

/* Measurement helper (not part of the verify step): reads every 16-byte
 * vector of the device buffer buf[0..bytes) once, with the statistics pass's
 * access pattern (workgroups of 256 threads, `unroll` in {2, 4, 8} vectors per
 * thread), so that timing it on `stream` gives the streaming-read ceiling the
 * verify kernels are measured against.  sink: device uint32[1024], written
 * only to keep the loads alive.  buf must be 16-byte aligned. */
int spec_verify_stream_read(const void* buf, int64_t bytes, uint32_t* sink, int unroll, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_H */

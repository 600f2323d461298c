/*
 * sdv.h -- C ABI of libsdv: batched lossless draft verification with
 * test-time self-selection, for speculative decoding with diffusion drafters,
 * on one NVIDIA GB300 (sm_103a).
 *
 * What one call computes, for every sequence b of a batch of B, given K
 * candidate drafts of gamma tokens each:
 *
 *   1. Temperature softmax of every verifier row p(.|s, x_<j) (j = 0..gamma)
 *      and drafter row q_j (j = 0..gamma-1) over the full vocabulary V.
 *      ("SpecDiff-2: Scaling Diffusion Drafter Alignment For Faster
 *      Speculative Decoding", section 2: the verifier scores all positions in
 *      parallel and exposes q(.|s) and p(.|s).)
 *   2. Per drafted token the acceptance ratio a = min(1, p(x)/q(x)), and per
 *      draft the expected accepted streak S_k = sum_j prod_{i<=j} a_i
 *      (same page, Figure 2 and section 3: position-wise acceptance and
 *      accepted streaks).
 *   3. Self-selection: sel = argmax_k S_k, ties to the lowest k (same page,
 *      section 5.2: K drafts from one denoising pass are ranked by a
 *      streak-oriented verifier score and the best is verified; the verifier
 *      probabilities of the ranking are reused for acceptance).
 *   4. The standard left-to-right acceptance rule on draft sel: token j is
 *      accepted when q <= p, else when u_j < p/q; the first rejection ends the
 *      scan (same page, section 2; "DiffuSpec: Unlocking Diffusion Language
 *      Models for Speculative Decoding", section 3).
 *   5. At the first rejection L < gamma, a replacement token drawn from the
 *      normalised residual max(0, p_L - q_L) (same passages); when all gamma
 *      tokens are accepted, a bonus token drawn from p_gamma.
 *
 * Random numbers: Philox4x32-10 (Salmon et al., SC'11) with key
 * (seed & 0xffffffff, seed >> 32) and counter (j, b, 0, 0); word 0 gives the
 * acceptance uniform u_j, word 1 the sampling uniform w_j, each as
 * (word >> 8) * 2^-24.  The uniforms do not depend on k.  Inverse-CDF draws
 * return the first id v whose cumulative mass exceeds w * (total mass).
 *
 * Layout: every tensor is contiguous, row-major, on the device of the
 * context unless stated otherwise.
 *   p_logits  [B][K][gamma+1][V]  bf16 or fp32
 *   q_logits  [B][K][gamma][V]    same dtype as p_logits ([B][gamma][V] with
 *                                 SDV_FLAG_SHARED_Q, see sdv_create_ex)
 *   drafts    [B][K][gamma]       int32 token ids
 *   out_sel, out_accept_len, out_next_token  [B] int32
 * V * sizeof(element) must be a multiple of 16 bytes and both logit buffers
 * 16-byte aligned (every row then starts on a 16-byte boundary).
 *
 * Ownership: the caller owns every tensor.  A context owns its workspace
 * (allocated by sdv_create, freed by sdv_destroy) and borrows the stream.
 *
 * Errors: argument errors are returned synchronously and nothing is
 * enqueued.  Data errors found on the device (a draft id outside [0, V), a row
 * holding NaN or +inf or only -inf, a per-sequence temperature that is not a
 * finite positive number) set the outputs of that sequence to -1 and are
 * reported by the next sdv_sync.  A context is not thread-safe; use one
 * context per stream.  Outputs are a pure function of (inputs, temperature,
 * seed).
 *
 * CUDA graphs: sdv_verify, sdv_verify_ex, sdv_verify_len, sdv_verify_qstat,
 * sdv_cps, sdv_cps_ex, sdv_cps_prune, sdv_cps_beam and sdv_adl_step check
 * their arguments on the host and enqueue kernels; they allocate nothing,
 * copy nothing and never wait.  Each may therefore be captured into a CUDA graph, in any capture
 * mode, when the stream it launches on (the context's, for the verify calls:
 * see sdv_set_stream) is the capturing stream, with kernel timing off.  Make
 * one uncaptured call of each shape first (the path search may set a kernel
 * attribute on its first call with a large lattice).  A replay recomputes the
 * step from the current contents of the captured buffers, with the scalars of
 * the capture (temperature, seed, tau, ...).  sdv_verify_host and sdv_sync
 * wait for the stream and cannot be captured.
 */
#ifndef SDV_H
#define SDV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct sdv_ctx sdv_ctx;

typedef enum {
    SDV_OK = 0,
    SDV_ERR_ARG = 1,          /* bad argument; nothing was enqueued              */
    SDV_ERR_CUDA = 2,         /* a CUDA runtime call failed, or a device wait    */
                              /* gave up after its iteration limit               */
    SDV_ERR_OOM = 3,          /* workspace allocation failed                     */
    SDV_ERR_DEVICE_DATA = 4,  /* bad draft id / non-finite row / bad per-seq T   */
    SDV_ERR_SCRATCH = 5       /* sdv_verify_static: the shape needs more scratch */
                              /* than SDV_STATIC_SCRATCH_BYTES                   */
} sdv_status;

/* SDV_BF16 and SDV_F32 are the logit types of a verification step.  SDV_F16 is
 * also a type of queries, keys and values, and SDV_E4M3 one of a cache's cells
 * (see sdv_kv_cache). */
typedef enum { SDV_BF16 = 0, SDV_F32 = 1, SDV_F16 = 2, SDV_E4M3 = 3 } sdv_dtype;

/*
 * Create a context for batches of shape (B, K, gamma, V) on the current CUDA
 * device, enqueuing on `stream` (a cudaStream_t; NULL = the legacy default
 * stream).  Requires B >= 1, K >= 1, gamma >= 1, V >= 1, V * elt % 16 == 0.
 * Allocates the workspace (partial row statistics, per-sequence tasks, a
 * status word: a few MB at most).  The select pass holds about
 * K * (20 * gamma + 12) bytes per sequence in shared memory; a shape beyond
 * the device's per-block limit (227 KB on GB300, where K = 64 at gamma = 128
 * fits) is refused with SDV_ERR_ARG.  On error *out is NULL.
 */
sdv_status sdv_create(sdv_ctx** out, int B, int K, int gamma, int V,
                      sdv_dtype dtype, void* stream);

/*
 * Layout flags for sdv_create_ex.
 *
 * SDV_FLAG_SHARED_Q: the K drafts of a sequence are sampled from the
 * position-wise marginals of one denoising pass ("SpecDiff-2: Scaling
 * Diffusion Drafter Alignment For Faster Speculative Decoding", section 5.2),
 * so the drafter rows do not depend on k: q_logits is [B][gamma][V] and row
 * (b, j) serves every draft k.  Each marginal row is read once, which cuts the
 * drafter bytes K-fold.  Results equal those of the full layout with q
 * broadcast over k.
 */
#define SDV_FLAG_SHARED_Q 1u

/*
 * SDV_FLAG_GREEDY: greedy acceptance, which verifies the selected draft
 * without drafting probabilities (same page, section 5.2 and appendix B.4;
 * usable with drafters of another tokenizer).  No drafter rows are read:
 * q_logits may be NULL.  a_j = p_j(x_j), the streak score is
 * S_k = sum_j prod_{i<=j} p_i(x_i), token j is accepted when u_j < p_j(x_j),
 * and at the first rejection L the replacement is drawn from p_L with x_L
 * zeroed out (renormalised); with every token accepted, the bonus token comes
 * from p_gamma.  out_lse is then [B][K][gamma+1].  Cannot be combined with
 * SDV_FLAG_SHARED_Q.
 */
#define SDV_FLAG_GREEDY 2u

/*
 * SDV_FLAG_SHARED_PREFIX_ROW: the verifier row at position 0 of every draft
 * conditions only on the shared prefix s (same page, section 5.2: the K
 * drafts extend one prefix), so it is one row per sequence: row (b, 0, 0) of
 * p_logits serves every draft k and rows (b, k > 0, 0) are not read (their
 * contents do not matter).  p_logits keeps its [B][K][gamma+1][V] shape.
 * Results equal those of the full layout with row (b, 0, 0) copied to every
 * k.  Combines with either flag above.
 */
#define SDV_FLAG_SHARED_PREFIX_ROW 4u

/* sdv_create with layout flags (0 = the full [B][K][gamma][V] q layout). */
sdv_status sdv_create_ex(sdv_ctx** out, int B, int K, int gamma, int V,
                         sdv_dtype dtype, void* stream, unsigned flags);

/*
 * Enqueue one verification step with one temperature for all sequences
 * (temperature > 0, finite; it scales both p and q).  Returns after
 * enqueuing; the outputs are valid once the stream has reached this point.
 */
sdv_status sdv_verify(sdv_ctx* ctx, const void* p_logits, const void* q_logits,
                      const int32_t* drafts, float temperature, uint64_t seed,
                      int32_t* out_sel, int32_t* out_accept_len,
                      int32_t* out_next_token);

/*
 * As sdv_verify, plus:
 *   temperature_per_seq  device float [B] or NULL (NULL: use `temperature`)
 *   out_scores           device float [B][K] expected streaks, or NULL
 *   out_lse              device float [B][K][2 gamma + 1] row log-sum-exp of
 *                        l / T (p rows j = 0..gamma, then q rows j = 0..gamma-1),
 *                        or NULL
 */
sdv_status sdv_verify_ex(sdv_ctx* ctx, const void* p_logits, const void* q_logits,
                         const int32_t* drafts, float temperature,
                         const float* temperature_per_seq, uint64_t seed,
                         int32_t* out_sel, int32_t* out_accept_len,
                         int32_t* out_next_token, float* out_scores,
                         float* out_lse);

/*
 * As sdv_verify_ex, with a draft length per sequence ("DiffuSpec: Unlocking
 * Diffusion Language Models for Speculative Decoding", sections 4.2-4.3: the
 * draft length adapts per step, and a path ends at its first EOS).
 *   draft_len  device int32 [B], 0 <= draft_len[b] <= gamma (required)
 * The arrays keep their gamma stride; for sequence b only the drafts at
 * positions j < draft_len[b] count, so the caller may leave the rest as
 * they are.  The streak scores and the acceptance scan run over those
 * positions, and with all of them accepted the bonus token comes from the
 * verifier row at position draft_len[b], drawn with that position's uniform.
 * Rows past a sequence's length are not read: the p rows j > draft_len[b] and
 * the q rows j >= draft_len[b].  Their out_lse entries are NaN.  The result
 * for b equals that of sdv_verify_ex on the drafts cut to draft_len[b].  A
 * length outside [0, gamma] is a data error for that sequence: its outputs
 * are -1, and sdv_sync reports SDV_ERR_DEVICE_DATA.
 */
sdv_status sdv_verify_len(sdv_ctx* ctx, const void* p_logits, const void* q_logits,
                          const int32_t* drafts, const int32_t* draft_len, float temperature,
                          const float* temperature_per_seq, uint64_t seed, int32_t* out_sel,
                          int32_t* out_accept_len, int32_t* out_next_token, float* out_scores,
                          float* out_lse);

/*
 * As sdv_verify_len (draft_len may be NULL: every draft has gamma tokens),
 * with the drafter rows' softmax statistics supplied by the caller instead of
 * computed here.  In a decode step the path search has just streamed the same
 * marginals (sdv_cps_ex writes these statistics), so the verification reads
 * the q rows only at the drafted tokens and, for a rejection, in the residual
 * draw: one full pass over the marginals per step instead of two.
 *   q_row_stat  device float [rows_q][4], 16-byte aligned, one entry per q
 *               row in q_logits' row order ([B][gamma] with
 *               SDV_FLAG_SHARED_Q, else [B][K][gamma]):
 *               {m, s, c, 0} with c = 1.4426950408889634f / T, an fp32
 *               division (T the row's sequence's temperature), m the row's
 *               largest logit and s = sum over the row of 2^((logit - m) * c)
 * The result is that of sdv_verify_len up to the rounding of s (the sum is
 * taken in another order).  An entry whose c differs from the c this call
 * computes for its sequence is a data error for that sequence (outputs -1,
 * SDV_ERR_DEVICE_DATA from sdv_sync).  A row whose m or s is not finite, or
 * s <= 0, is a bad row as for sdv_verify_ex.  Not with SDV_FLAG_GREEDY
 * (which reads no q rows): SDV_ERR_ARG.
 */
sdv_status sdv_verify_qstat(sdv_ctx* ctx, const void* p_logits, const void* q_logits,
                            const int32_t* drafts, const int32_t* draft_len,
                            const float* q_row_stat, float temperature,
                            const float* temperature_per_seq, uint64_t seed, int32_t* out_sel,
                            int32_t* out_accept_len, int32_t* out_next_token, float* out_scores,
                            float* out_lse);

/*
 * End-to-end variant for callers whose data lives in HOST memory: copies the
 * inputs to device buffers owned by the context (allocated on the first call,
 * the size of one batch's inputs), runs sdv_verify_ex, copies the three
 * outputs back and waits for the stream.  All pointers are host pointers
 * (pinned memory gives full copy bandwidth); temperature_per_seq may be NULL.
 * Returns the status of the step, as sdv_sync would.
 */
sdv_status sdv_verify_host(sdv_ctx* ctx, const void* p_logits_host,
                           const void* q_logits_host, const int32_t* drafts_host,
                           float temperature, const float* temperature_per_seq_host,
                           uint64_t seed, int32_t* out_sel_host,
                           int32_t* out_accept_len_host,
                           int32_t* out_next_token_host);

/*
 * Wait for the context's stream and return the device-side status of every
 * step enqueued since the previous sdv_sync (then cleared): SDV_OK,
 * SDV_ERR_DEVICE_DATA or SDV_ERR_CUDA.  SDV_ERR_CUDA with the text "a bounded
 * device wait gave up" means that the sampling pass waited for its row copy
 * longer than its poll limit; it then wrote -1 to all three outputs of the
 * sequences concerned, and the context stays usable.
 */
sdv_status sdv_sync(sdv_ctx* ctx);

/* Text of the last error seen by this context ("" if none).  The pointer is
 * valid until the next call on the context. */
const char* sdv_last_error(const sdv_ctx* ctx);

/* Free the workspace and the context (NULL is a no-op).  Waits for the
 * context's stream first. */
void sdv_destroy(sdv_ctx* ctx);

/* Launch plan of a context, for tests and benchmarks: CTAs of the row pass,
 * 16-byte vectors per row chunk, chunks per row, CTAs per sequence (cluster
 * size) of the sampling pass.  Any pointer may be NULL. */
sdv_status sdv_plan(const sdv_ctx* ctx, int* rowpass_ctas, int64_t* chunk_vectors,
                    int* chunks_per_row, int* sample_cluster);

/*
 * Fault-path test hook (not part of the method; the pages have no
 * counterpart).  With SDV_HOOK_SAMPLE_NO_COPY set, the sampling pass of later
 * steps arms its barrier for the row copy but issues no copy and polls only a
 * few times, so that its bounded wait runs out with nothing in flight: the
 * step writes -1 to every sequence's three outputs and sdv_sync returns
 * SDV_ERR_CUDA ("a bounded device wait gave up").  This is how the timeout
 * path is tested without faulting or hanging a GPU.  hooks = 0 restores
 * normal steps; unknown bits give SDV_ERR_ARG.
 */
#define SDV_HOOK_SAMPLE_NO_COPY 1u
sdv_status sdv_set_test_hooks(sdv_ctx* ctx, unsigned hooks);

/* Replace the stream of a context (a cudaStream_t): later calls enqueue on
 * it.  The caller orders it after work already enqueued on the old stream.
 * To capture a step into a CUDA graph, set the capturing stream first. */
sdv_status sdv_set_stream(sdv_ctx* ctx, void* stream);

/*
 * Kernel timing.  While enabled, every step records CUDA events on the
 * context's stream before the row pass and after each of its three kernels
 * (row pass, select/scan, sample), for up to 65536 steps.  sdv_profile_read
 * waits for the recorded steps, writes the mean device time in milliseconds
 * of each kernel to ms_avg[0..2] and the number of steps to *steps, and
 * clears the record.  Enabling with enable = 0 stops recording.
 */
sdv_status sdv_profile_enable(sdv_ctx* ctx, int enable);
sdv_status sdv_profile_read(sdv_ctx* ctx, float* ms_avg, int* steps);

/*
 * Causal-consistency path search over drafter marginals ("DiffuSpec:
 * Unlocking Diffusion Language Models for Speculative Decoding", section 4.2;
 * the page's settings, section 5.3: beam 3, mmax 15, tau 0.8).  Produces
 * left-to-right drafts from one denoising pass's position-wise marginals:
 *   1. each row q[b][j] is pruned to the shortest list of its most likely
 *      tokens (probability of softmax(q / T) descending, ties to the lower id)
 *      whose mass reaches tau, at most mmax tokens; a token of probability
 *      zero (logit -inf) is never a candidate;
 *   2. the lattice ends at the first position whose most likely token is
 *      eos_id, which is kept alone as the last token (eos_id < 0: no cut);
 *   3. the paths a beam of width `beam` keeps over the lattice, scoring a
 *      path by the sum of its log-probabilities (drafter confidence; the
 *      page's causal fluency proxy is not specified there and is not used).
 *      The temperature and each position's normaliser are common to all of a
 *      sequence's paths, so paths rank by the sum of their raw logits (in
 *      fp64, exact for bf16 logits); equal sums go to the path whose
 *      candidate ranks come first lexicographically.  With a score that sums
 *      over positions the beam keeps the `beam` best paths of the lattice,
 *      and these are found best first rather than position by position.  The
 *      result is those paths, best first, each with its log-probability
 *      summed in fp32 in a fixed order.
 * The paths serve as the K = beam drafts of a verification step
 * (SDV_FLAG_SHARED_Q, with the same q).
 * Arguments: q_marginals device [B][gamma][V] bf16 or fp32 (16-byte aligned,
 * V * elt % 16 == 0); temperature, or device temperature_per_seq [B];
 * 0 <= tau <= 1; 1 <= mmax <= 16; 1 <= beam <= 16; gamma <= 1024;
 * eos_id < V.  Outputs (device, caller-owned): out_cand_ids / out_cand_logp /
 * out_cand_logit [B][gamma][mmax] (candidate ids, natural-log probabilities
 * and raw logits; -1 / -inf / -inf past the count), out_ncand [B][gamma] (0
 * past the lattice), out_paths [B][beam][gamma] (-1 past the lattice or past
 * npaths), out_path_logp [B][beam] (-inf past npaths), out_npaths [B],
 * out_lat_len [B] or NULL.  A row holding NaN, +inf or only -inf gets no
 * candidates and its sequence no path.  Stateless: allocates nothing, only
 * enqueues on `stream`.
 */
sdv_status sdv_cps(int B, int gamma, int V, sdv_dtype dtype, void* stream,
                   const void* q_marginals, float temperature,
                   const float* temperature_per_seq, float tau, int mmax, int beam,
                   int eos_id, int32_t* out_cand_ids, float* out_cand_logp,
                   float* out_cand_logit, int32_t* out_ncand, int32_t* out_paths,
                   float* out_path_logp, int32_t* out_npaths, int32_t* out_lat_len);

/*
 * sdv_cps that also writes every marginal row's softmax statistics, as the
 * pruning pass computes them, to out_row_stat (device float [B][gamma][4],
 * 16-byte aligned, or NULL): {m, s, c, 0} with c = 1.4426950408889634f / T
 * (fp32), m the row's largest logit and s = sum of 2^((logit - m) * c).  sdv_verify_qstat takes
 * them so that the verification of the paths does not stream the marginals a
 * second time.
 */
sdv_status sdv_cps_ex(int B, int gamma, int V, sdv_dtype dtype, void* stream,
                      const void* q_marginals, float temperature,
                      const float* temperature_per_seq, float tau, int mmax, int beam,
                      int eos_id, int32_t* out_cand_ids, float* out_cand_logp,
                      float* out_cand_logit, int32_t* out_ncand, int32_t* out_paths,
                      float* out_path_logp, int32_t* out_npaths, int32_t* out_lat_len,
                      float* out_row_stat);

/*
 * The two halves of sdv_cps, for callers that inspect or reuse the pruned
 * lattice.  sdv_cps_prune is step 1 for every row (no EOS cut): it reads
 * q_marginals / temperature(_per_seq) and writes out_cand_ids, out_cand_logp,
 * out_cand_logit and out_ncand exactly as sdv_cps documents them, before the
 * cut.  sdv_cps_beam is steps 2-3: it reads the lattice (as sdv_cps_prune
 * wrote it: each position's candidates in decreasing order of logit, at most
 * mmax of them; a count of 0 or less leaves the sequence without a path),
 * trims it in place at an EOS end (one candidate at the EOS
 * position, none past it) and writes the paths.  V is only used to check
 * eos_id.  Argument rules, ownership and errors as for sdv_cps; sdv_cps is
 * sdv_cps_prune followed by sdv_cps_beam on `stream`.
 */
sdv_status sdv_cps_prune(int B, int gamma, int V, sdv_dtype dtype, void* stream,
                         const void* q_marginals, float temperature,
                         const float* temperature_per_seq, float tau, int mmax,
                         int32_t* out_cand_ids, float* out_cand_logp, float* out_cand_logit,
                         int32_t* out_ncand);
sdv_status sdv_cps_beam(int B, int gamma, int V, int mmax, int beam, int eos_id, void* stream,
                        int32_t* cand_ids, float* cand_logp, float* cand_logit, int32_t* ncand,
                        int32_t* out_paths, float* out_path_logp, int32_t* out_npaths,
                        int32_t* out_lat_len);

/*
 * Adaptive draft length ("DiffuSpec: Unlocking Diffusion Language Models for
 * Speculative Decoding", section 4.3 and appendix C).  The page states the
 * controller's inputs and direction only; this is the plainest rule that
 * fits it.  Per sequence, a window of the last `window` steps records the
 * draft length k used, the EOS-aware generated length g (tokens up to and
 * including the first EOS of the chosen draft, e.g. sdv_cps's lattice length)
 * and the accepted length a (e.g. sdv_verify's out_len); g is clamped to
 * [0, k] and a to [0, g].  Acceptance keeps pace when the window's a sum to
 * its g; generation fills the drafts when its g sum to its k.  The next
 * length is k + up if both hold, k if only the first holds (generation
 * saturated: EOS before the end of the draft), k - down otherwise, clamped to
 * [kmin, kmax].
 * Limits: 1 <= window <= 64; 1 <= kmin <= kmax <= 2^20; 0 <= up, down <= 2^20.
 * sdv_adl_state_words(window): int32 words of one sequence's state (-1 for a
 * bad window).  The state [B][words] is caller-owned and starts zeroed; its
 * layout is private to the library.
 * sdv_adl_step_host: host pointers; k [B] holds the lengths just used and
 * receives the next ones.  SDV_ERR_ARG for bad limits or any k outside
 * [kmin, kmax] (then nothing is updated).
 * sdv_adl_step: the same on device pointers, enqueued on `stream` (one thread
 * per sequence); a sequence whose k lies outside [kmin, kmax] is left as it
 * is and sets bit 16 in *status (device int32, may be NULL), which the caller
 * clears.  Host-checked argument errors return SDV_ERR_ARG.
 */
#define SDV_ADL_MAX_WINDOW 64
#define SDV_STATUS_BAD_LENGTH 16
int sdv_adl_state_words(int window);
sdv_status sdv_adl_step_host(int B, int window, int kmin, int kmax, int up, int down,
                             const int32_t* gen_len, const int32_t* acc_len, int32_t* k,
                             int32_t* state);
sdv_status sdv_adl_step(int B, int window, int kmin, int kmax, int up, int down, void* stream,
                        const int32_t* gen_len, const int32_t* acc_len, int32_t* k,
                        int32_t* state, int32_t* status);

/*
 * sdv_verify_static -- the step of sdv_verify_ex for callers that cannot
 * allocate device memory.  The pages have no counterpart to this entry point:
 * it exists for deployment, not for the method.
 *
 * Who needs it: code that must not call cudaMalloc -- a process whose device
 * memory belongs entirely to another allocator (a serving engine's pool, which
 * would otherwise see memory vanish behind its back), a plug-in loaded into
 * such a process, code that runs where allocation is forbidden.  sdv_create
 * allocates a workspace; this call does not.  It takes no context and
 * allocates nothing: no cudaMalloc, no cudaFree, no allocating library
 * routine.
 *
 * Scratch: the row-pass partials, per-sequence tasks and status word live in
 * one static device array of SDV_STATIC_SCRATCH_BYTES (8 MiB), which every GPU
 * that loads libsdv holds until the process exits.  A shape whose scratch does
 * not fit is rejected with SDV_ERR_SCRATCH before anything is enqueued (as a
 * guide: partials take 8 bytes per row chunk, at least one chunk per row, so
 * B*K*(2*gamma+1) must stay below about one million rows).
 *
 * Set-up: the first call on a device, with that device current, looks up the
 * device address of the array (cudaGetSymbolAddress), the device's limits,
 * and raises the kernels' shared-memory limits; later calls on that device
 * do none of this.
 *
 * Arguments: as sdv_verify_ex, with the shape (B, K, gamma, V, dtype) and the
 * stream (a cudaStream_t, NULL = legacy default stream) passed on every call;
 * all tensors are caller-owned device memory (logits 16-byte aligned, the
 * int32 / float arrays 4-byte aligned).  Outputs are the same values
 * sdv_verify_ex writes.  Argument errors -- including a host pointer or a
 * misaligned one -- return SDV_ERR_ARG and nothing is enqueued.  The call only
 * enqueues; there is no sdv_sync for it: a sequence with bad data (draft id
 * out of range, non-finite row, bad per-sequence temperature), or whose
 * sampling pass gave up waiting for its row copy, gets -1 in all three
 * outputs.
 *
 * Sharing: every call uses the same array and leaves its contents behind (the
 * status word is cleared at the start of each call; the rest is written before
 * it is read).  Calls that overlap on the GPU -- on two streams or from two
 * host threads -- race on the array; the caller must serialise them.
 */
#define SDV_STATIC_SCRATCH_BYTES (8u << 20)
sdv_status sdv_verify_static(int B, int K, int gamma, int V, sdv_dtype dtype, void* stream,
                             const void* p_logits, const void* q_logits,
                             const int32_t* drafts, float temperature,
                             const float* temperature_per_seq, uint64_t seed,
                             int32_t* out_sel, int32_t* out_accept_len,
                             int32_t* out_next_token);

/* ------------------------------------------------------------------------
 * The verifier's layer around a step: a tree of drafted tokens, rotary
 * positions, a paged cache of keys and values, attention of the tree over that
 * cache, and the sampling parameters of every draft position.
 *
 * "SpecDiff-2: Scaling Diffusion Drafter Alignment For Faster Speculative
 * Decoding", appendix B.8: the K drafts are flattened into one tree, which the
 * verifier scores in one forward pass with a branch-aware attention mask, the
 * cache of the shared prefix being reused.  The page gives no layouts; those
 * below are this library's.
 *
 * All entry points here are stateless: they check their arguments on the host
 * (SDV_ERR_ARG: nothing was enqueued; pointers that are not memory of the
 * current device among them), allocate nothing, only enqueue on
 * `stream`, and can be captured into a CUDA graph (after one uncaptured call of
 * each shape).  Strides are in elements, and the innermost one is 1.  Data
 * errors that only the device can see (a page id outside the cache, a length
 * outside its limits) set bits of *status (device int32, which the caller
 * clears; NULL: not reported); what such an entry does to the outputs is said
 * at each call, and no memory outside the caller's buffers is touched.
 * --------------------------------------------------------------------- */
#define SDV_STATUS_BAD_TOKEN 1      /* a token id outside [0, V)                      */
#define SDV_STATUS_BAD_ROW 2        /* a row with a NaN or +infinity, or nothing finite */
#define SDV_STATUS_BAD_PARAM 4      /* a sampling parameter outside its range         */
#define SDV_STATUS_TIMEOUT 8        /* a bounded device wait gave up                  */
#define SDV_STATUS_BAD_PAGE 64      /* a page id outside [0, pages)                   */
#define SDV_STATUS_NO_PAGES 128     /* the free pages ran out                         */

/*
 * The tree of K drafts.  Node 0 is the sequence's last committed token (the
 * root, whose key and value are not in the cache yet); the other nodes are the
 * drafts' tokens, drafts that begin with the same tokens sharing their nodes.
 * Nodes are numbered draft by draft, left to right, so a node's ancestors come
 * before it.  N = 1 + K * gamma nodes have room.
 *   root       device int32 [B]
 *   drafts     device int32 [B][K][gamma]
 *   draft_len  device int32 [B], 0 <= draft_len[b] <= gamma, or NULL (gamma)
 * Outputs (device int32, caller-owned):
 *   tokens     [B][N] token of each node (-1 past the sequence's nodes)
 *   depth      [B][N] distance from the root (a node's position is the number
 *              of committed tokens in the cache + depth); 0 past the nodes
 *   mask       [B][N][ceil(N / 32)] bit m % 32 of word m / 32 of node i's row:
 *              node m is i itself or one of its ancestors (rows past the
 *              nodes are 0)
 *   nodes      [B][K][gamma] node of draft k's token j (-1 for j >= draft_len)
 *   rows       [B][K][gamma + 1] node whose logits are the verifier's row
 *              (b, k, j): the root for j = 0, the node of token j - 1 else
 *              (the root past the length)
 *   count      [B] nodes of the tree
 * A draft_len outside [0, gamma] gives that sequence the root alone and sets
 * SDV_STATUS_BAD_LENGTH.  K <= 64, gamma <= 128.
 */
sdv_status sdv_tree_build(int B, int K, int gamma, void* stream, const int32_t* root,
                          const int32_t* drafts, const int32_t* draft_len, int32_t* tokens,
                          int32_t* depth, int32_t* mask, int32_t* nodes, int32_t* rows,
                          int32_t* count, int32_t* status);

/*
 * Rotary frequencies, on the host: inv_freq[i] = base^(-2i / R) for i < R / 2
 * (R even, 2 <= R <= 512; base > 0), scaled for contexts longer than the
 * `original` length by `factor` >= 1:
 *   SDV_ROPE_PLAIN   unchanged
 *   SDV_ROPE_LINEAR  every frequency divided by factor (positions interpolated)
 *   SDV_ROPE_BASE    base * factor^(R / (R - 2)) in the place of base (R >= 4)
 *   SDV_ROPE_PARTS   frequencies that turn at least `fast` times within
 *                    `original` positions stay, those that turn at most `slow`
 *                    times are divided by factor, with a linear ramp over the
 *                    number of turns between them (fast > slow >= 0,
 *                    original >= 1); *attn_factor, which multiplies cosine and
 *                    sine, is 0.1 ln(factor) + 1 (1 for the other kinds)
 * Computed in 64 bits, rounded once.  attn_factor may be NULL.
 */
#define SDV_ROPE_PLAIN 0
#define SDV_ROPE_LINEAR 1
#define SDV_ROPE_BASE 2
#define SDV_ROPE_PARTS 3
sdv_status sdv_rope_freqs(int R, double base, int scaling, double factor, double original,
                          double fast, double slow, float* inv_freq, float* attn_factor);

/*
 * Rotary positions for the queries [T][Hq][D] and keys [T][Hk][D] of T tokens.
 * Pair i < R / 2 of token t's head, (x_i, x_{i + R/2}) or with `interleaved`
 * (x_{2i}, x_{2i + 1}), turns by the angle positions[t] * inv_freq[i]:
 *   (a, b) -> factor * (a cos - b sin, b cos + a sin)
 * and elements R..D-1 are copied.  Angles are off by 2^-26 of a turn at most, at
 * any int32 position (for |inv_freq| up to 2^40); arithmetic is fp32 with one
 * rounding at the end.
 *   dtype      SDV_BF16, SDV_F16 or SDV_F32
 *   q_st, q_sh strides of a token and of a head (k_*, oq_*, ok_* alike)
 *   k, out_k   NULL with Hk = 0: queries alone
 *   out_q may be q with the same strides (in place), and out_k k; buffers that
 *   overlap in any other way give undefined values
 * 2 <= R <= D <= 4096, R even, R <= 512, T >= 0, 1 <= Hq + Hk <= 4096, Hq >= 1.
 * positions and inv_freq are device arrays ([T] int32, [R / 2] float).
 */
sdv_status sdv_rope(int64_t T, int Hq, int Hk, int D, int R, int interleaved, sdv_dtype dtype,
                    void* stream, const void* q, int64_t q_st, int64_t q_sh, const void* k,
                    int64_t k_st, int64_t k_sh, const int32_t* positions, const float* inv_freq,
                    float factor, void* out_q, int64_t oq_st, int64_t oq_sh, void* out_k,
                    int64_t ok_st, int64_t ok_sh);

/*
 * A paged cache of one layer's keys and values.  k and v are
 * [pages][kv_heads][page_size][head_dim] cells, each page contiguous and
 * page_stride elements after the one before (so k and v may be the halves of
 * one [pages][2][...] buffer); k and v 16-byte aligned, page_stride * cell size
 * a multiple of 16 bytes.  Position t of sequence b is place t % page_size of
 * page block_table[b][t / page_size].
 *
 * dtype SDV_BF16 or SDV_F16: cells hold the values; k_exp and v_exp are NULL.
 * dtype SDV_E4M3: a cell row (one position, one head) is held in e4m3 in units
 * of a power of two of its own, 2^(exp - 127), with exp in k_exp / v_exp,
 * uint8 [pages][kv_heads][page_size], exp_page_stride after one another
 * (a row holds the smallest power, no less than 2^-126, that brings its
 * largest magnitude to at most 448; exp 255: the row is not a number).  A
 * magnitude of 2^128 - 2^123 and more rounds to 2^128, which may count as infinite.
 * head_dim is a multiple of 16, at most 256; page_size >= 1.
 */
typedef struct sdv_kv_cache {
    void* k;
    void* v;
    uint8_t* k_exp;
    uint8_t* v_exp;
    int64_t page_stride;
    int64_t exp_page_stride;
    int pages;
    int page_size;
    int kv_heads;
    int head_dim;
    sdv_dtype dtype;
} sdv_kv_cache;

/*
 * Pages for new tokens, from request lengths.  The free pages are a stack,
 * free_list[0 .. *free_count - 1], and sequence b holds the first held[b] pages
 * of its row of block_table.  For positions start[b] .. start[b] + count[b] - 1
 * (count NULL: N) it needs ceil((start[b] + count[b]) / page_size) pages; those
 * it lacks are taken from the stack's top, sequence by sequence in order, and
 * go to its row, and held and *free_count follow.  Where the stack does not last,
 * a sequence for which it no longer does takes nothing (SDV_STATUS_NO_PAGES), nor
 * does any after it that lacks a page.
 *   free_list  device int32 [pages]
 *   free_count device int32 [1], held device int32 [B]
 *   block_table device int32 [B][max_pages]
 *   depth      device int32 [B][N] (sdv_tree_build's) or NULL: n
 *   base       device int32 [B] or NULL: 0 (a shared prefix's length)
 *   positions  device int32 [B][N] or NULL: base[b] + start[b] + depth[b][n], as
 *              sdv_rope takes them; 0 from count[b] on
 *   slots      device int64 [B][N] or NULL: place (start[b] + n) of the cache,
 *              page * page_size + place in the page; -1 from count[b] on and
 *              where there is no page (or a bad one)
 * A held outside [0, max_pages], a negative start, a count outside [0, N], or a
 * sum beyond max_pages * page_size sets SDV_STATUS_BAD_LENGTH, and the sequence
 * takes nothing and has no slots; *free_count outside [0, pages] sets it too, and
 * no sequence takes anything.  An entry of the list outside [0, pages) sets
 * SDV_STATUS_BAD_PAGE and is handed out as it is (the cache's entry points refuse
 * it).  N <= 2^20, B <= 2^20, max_pages * page_size <= 2^30.
 */
sdv_status sdv_pages_extend(int B, int N, int pages, int page_size, int max_pages, void* stream,
                            int32_t* free_list, int32_t* free_count, int32_t* block_table,
                            int32_t* held, const int32_t* start, const int32_t* count,
                            const int32_t* depth, const int32_t* base, int32_t* positions,
                            int64_t* slots, int32_t* status);

/*
 * Give back the pages behind the first keep[b] positions of each sequence (0:
 * all it holds): its entries of block_table from place ceil(keep[b] / page_size)
 * on go to the stack and become -1, and held and *free_count follow.  A keep
 * beyond what is held changes nothing.  They go back in the order that returns the
 * stack to what it was when they were just taken by sdv_pages_extend.  A negative
 * keep or a held outside [0, max_pages] sets SDV_STATUS_BAD_LENGTH, and the
 * sequence keeps all; so does a *free_count that is out of range or would exceed
 * `pages`, and all keep all.  An entry outside [0, pages) sets SDV_STATUS_BAD_PAGE
 * and goes back as it is.
 */
sdv_status sdv_pages_release(int B, int pages, int page_size, int max_pages, void* stream,
                             int32_t* free_list, int32_t* free_count, int32_t* block_table,
                             int32_t* held, const int32_t* keep, int32_t* status);

/*
 * Write the keys and values of up to N new positions per sequence: row n of
 * sequence b goes to position start[b] + n, for n < count[b] (NULL: N).
 *   k, v       device [B][N][kv_heads][D] of `dtype` (SDV_BF16 or SDV_F16; the
 *              cache's dtype, unless that is SDV_E4M3), strides (sb, sn, sh)
 *   block_table device int32 [B][max_pages]
 *   start, count  device int32 [B]
 * A value is rounded once, to nearest even, when the cache is e4m3; a row that
 * holds a NaN or an infinity is then stored as not a number.  A position
 * outside [0, max_pages * page_size) or a count outside [0, N] sets
 * SDV_STATUS_BAD_LENGTH, a bad page SDV_STATUS_BAD_PAGE; those rows are not
 * written (a bad count writes nothing of its sequence).  Two rows that go to
 * one cell leave either.
 */
sdv_status sdv_kv_write(const sdv_kv_cache* cache, int B, int N, sdv_dtype dtype, void* stream,
                        const void* k, int64_t k_sb, int64_t k_sn, int64_t k_sh, const void* v,
                        int64_t v_sb, int64_t v_sn, int64_t v_sh, const int32_t* block_table,
                        int max_pages, const int32_t* start, const int32_t* count,
                        int32_t* status);

/*
 * Read positions start[b] .. start[b] + count[b] - 1 back into contiguous
 * out_k, out_v [B][N][kv_heads][D] of `dtype` (as for sdv_kv_write); rows past
 * count[b] become 0.  What an e4m3 row stands for is exact in bf16 (but for
 * magnitudes below 2^-133) and rounded once to fp16 (overflow to infinity).
 * Rows of a bad position, page or count become NaN, with the status bits of
 * sdv_kv_write.  Outputs are 16-byte aligned.
 */
sdv_status sdv_kv_read(const sdv_kv_cache* cache, int B, int N, sdv_dtype dtype, void* stream,
                       void* out_k, void* out_v, const int32_t* block_table, int max_pages,
                       const int32_t* start, const int32_t* count, int32_t* status);

/*
 * After a verification step: keep the accepted path.  The tree's cells sit at
 * positions start[b] + node; the cells of draft sel[b]'s accepted tokens move
 * to start[b] + 1 + j, j < accept_len[b] (the root's are in place), from node
 * nodes[b][sel[b]][j] (as sdv_tree_build numbers them: at least 1 and growing
 * with j).  Cells are moved as they are, with their exponents.
 *   out_len  device int32 [B] or NULL: start[b] + 1 + accept_len[b]
 * A sequence with sel = -1 (a data error of the step), or whose accept_len,
 * positions, nodes or pages are out of range (the status bits of sdv_kv_write;
 * SDV_STATUS_BAD_LENGTH for the nodes), gets out_len = start[b]; cells moved
 * before a bad one stay moved.  out_len may be the start array itself.
 */
sdv_status sdv_kv_commit(const sdv_kv_cache* cache, int B, int K, int gamma, void* stream,
                         const int32_t* block_table, int max_pages, const int32_t* start,
                         const int32_t* nodes, const int32_t* sel, const int32_t* accept_len,
                         int32_t* out_len, int32_t* status);

/*
 * Attention of the nodes of a tree over the cache.  Sequence b has
 * ctx_len[b] committed positions and count[b] <= N nodes (NULL: N) whose keys
 * and values are at positions ctx_len[b] + m (sdv_kv_write).  Node i sees every
 * committed position, and node m when bit m of its mask row is set (mask NULL:
 * when m <= i, a causal chain; so N = 1 is the decode step of one token and
 * ctx_len = 0 the first chunk of a prompt).  With s_j = scale * q_i . k_j over
 * what it sees,
 *   out_i = sum_j softmax(s)_j v_j      lse_i = ln sum_j e^{s_j}
 * in fp32 sums; a node that sees nothing has out = 0, lse = -inf, and so have
 * the nodes from count[b] on.
 *   q      device [B][N][Hq][D] of `dtype` (SDV_BF16 or SDV_F16; the cache's
 *          dtype, unless that is SDV_E4M3), strides (sb, sn, sh); Hq a multiple
 *          of the cache's kv_heads, query head h reading kv head
 *          h / (Hq / kv_heads)
 *   mask   device int32, rows of ceil(N / 32) words, one row per node;
 *          mask_sb words from one sequence's to the next (0: all have the same)
 *   out    device [B][N][Hq][D] of `dtype`, contiguous, 32-byte aligned
 *   lse    device float [B][N][Hq] contiguous, or NULL
 *   workspace  device memory of at least sdv_tree_attn_workspace(...) bytes,
 *          32-byte aligned, that no other call uses until this one is done
 * Probabilities are rounded to 16 bits for their product with the values; all
 * sums are fp32.  Over an e4m3 cache that product may be taken in fp16 of the
 * probability times the value row's power of two: a row where this is below
 * 2^-20 of the node's largest counts with fewer digits, below 2^-31 not at all.
 * What a node does not see has no influence on it, whatever it
 * holds.  A NaN, an infinite value and a score of +infinity that it does see make
 * its output not finite (which elements, and NaN or infinite, is not fixed).  A
 * score of -infinity (an infinite key in a 16-bit cache; an e4m3 row with an
 * infinity is not a number) has weight 0, and a node that sees no other score has
 * out = 0, lse = -inf as if it saw nothing.  A sequence whose
 * ctx_len, count or ctx_len + count is out of range gets NaN in out and lse;
 * the cells of a bad page count as not a number; both set the status bits of
 * sdv_kv_write.
 * sdv_tree_attn_workspace: bytes for calls of any shape on the current device
 * (0: the device cannot be asked).
 */
size_t sdv_tree_attn_workspace(void);
sdv_status sdv_tree_attn(const sdv_kv_cache* cache, int B, int N, int Hq, sdv_dtype dtype,
                         void* stream, const void* q, int64_t q_sb, int64_t q_sn, int64_t q_sh,
                         const int32_t* block_table, int max_pages, const int32_t* ctx_len,
                         const int32_t* count, const int32_t* mask, int64_t mask_sb, float scale,
                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                         int32_t* status);

/*
 * The same attention for sequences that share prefixes, each prefix read once
 * for all of its sequences.  The B sequences form `groups` groups of B / groups
 * (a whole number), in order; those of group j follow a prefix of prefix_len[j]
 * positions whose keys and values are on pages of their own, position t at place
 * t % page_size of page prefix_table[j][t / page_size].  What a sequence adds
 * begins on a new page: node i of sequence b sees the whole prefix of its group,
 * then what it sees in sdv_tree_attn, which all other arguments are as for.
 * (sdv_kv_write and sdv_kv_commit take block_table and ctx_len; a node's position
 * for sdv_rope is prefix_len + ctx_len + depth.)
 *   prefix_table  device int32 [groups][max_prefix_pages]
 *   prefix_len    device int32 [groups], 0 <= prefix_len <= max_prefix_pages * page_size
 *   workspace     at least sdv_prefix_attn_workspace(B, N, Hq, head_dim) bytes,
 *                 32-byte aligned, that no other call uses until this one is done
 * The nodes of a group whose prefix_len is out of range get NaN in out and lse
 * (nodes from count[b] on stay 0 and -inf); the other failures are those of
 * sdv_tree_attn.  B * N * Hq <= 2^31, and (B / groups) * N query rows of a kv head
 * at most 2^28.  Results of the two parts are joined in fp32.
 * sdv_prefix_attn_workspace: 0 for a bad shape, or when the device cannot be
 * asked.
 */
size_t sdv_prefix_attn_workspace(int B, int N, int Hq, int head_dim);
sdv_status sdv_prefix_attn(const sdv_kv_cache* cache, int B, int groups, int N, int Hq, sdv_dtype dtype,
                           void* stream, const void* q, int64_t q_sb, int64_t q_sn, int64_t q_sh,
                           const int32_t* prefix_table, int max_prefix_pages,
                           const int32_t* prefix_len, const int32_t* block_table, int max_pages,
                           const int32_t* ctx_len, const int32_t* count, const int32_t* mask,
                           int64_t mask_sb, float scale, void* out, float* lse, void* workspace,
                           size_t workspace_bytes, int32_t* status);

/*
 * Fault-path test hook of later sdv_tree_attn and sdv_prefix_attn calls of the
 * process (not part of the method).  With SDV_HOOK_ATTN_NO_COPY the kernels that
 * load by tile copies (head_dim <= 128, page_size a multiple of 8) leave the copies
 * of the first block's second tile out and poll fewer times, so that its bounded
 * waits run out with nothing of it in flight: the rows that this block had still to
 * write become NaN and *status gets SDV_STATUS_TIMEOUT.  hooks = 0 restores normal
 * calls; unknown bits give SDV_ERR_ARG.
 */
#define SDV_HOOK_ATTN_NO_COPY 2u
sdv_status sdv_set_attn_test_hooks(unsigned hooks);

/*
 * The sampling parameters of every draft position, before sdv_verify.  Row
 * (b, k, j) of the verifier's logits follows the tokens of sequence b and the
 * first j tokens of draft k, so its penalties count both:
 *   c = counts[b][v] + #{i < j : drafts[b][k][i] = v}
 *   x = the logit in fp32
 *   x = x > 0 ? x / repetition[b] : x * repetition[b]   where c > 0 or v is in
 *                                                       the prompt
 *   x = x - frequency[b] * c - presence[b] * [c > 0] + sum of v's biases
 *   x = -inf                                            where v is not allowed
 * rounded once to the logits' type.  (For bf16 logits the quotient may be the
 * product with the rounded reciprocal: one rounding of fp32 more.)
 *   logits     device [B][K][gamma + 1][V], or with `rows`
 *              [B][nsrc][V] (a tree's logits), 16-byte aligned
 *   rows       device int32 [B][K][gamma + 1] source row within the sequence's
 *              nsrc, or NULL (nsrc is then not used).  An id outside
 *              [0, nsrc) sets SDV_STATUS_BAD_LENGTH and gives a row of NaN
 *   drafts     device int32 [B][K][gamma] (ids outside [0, V) count nowhere)
 *   counts     device int32 [B][V], 16-byte aligned, or NULL: 0
 *   prompt     device int32 [B][ceil(V / 32)] bits (v % 32 of word v / 32), or
 *              NULL: none
 *   repetition, frequency, presence  device float [B], or NULL: 1, 0, 0
 *   bias_ids, bias  device int32 / float [B][M] with M >= 0, or NULL with
 *              M = 0; ids outside [0, V) are passed over, repeated ids add up
 *              in their order
 *   allow      device int32 [B][K][gamma + 1][ceil(V / 32)] bits, or NULL: all
 *   out        device [B][K][gamma + 1][V] of the logits' type, 16-byte
 *              aligned; without `rows` it may be logits itself
 * dtype SDV_BF16 or SDV_F32; V * elt % 16 == 0.
 */
sdv_status sdv_logits_process(int B, int K, int gamma, int V, sdv_dtype dtype, void* stream,
                              const void* logits, int nsrc, const int32_t* rows,
                              const int32_t* drafts, const int32_t* counts, const int32_t* prompt,
                              const float* repetition, const float* frequency,
                              const float* presence, int M, const int32_t* bias_ids,
                              const float* bias, const int32_t* allow, void* out,
                              int32_t* status);

/*
 * After a verification step: add the committed tokens to counts [B][V], those
 * of draft sel[b] at positions j < accept_len[b] and next_token[b].  A sequence
 * with sel = -1 adds nothing; sel, accept_len or a token out of range sets
 * SDV_STATUS_BAD_LENGTH / SDV_STATUS_BAD_TOKEN and that token (or for sel and
 * accept_len the sequence) is not counted.
 */
sdv_status sdv_counts_commit(int B, int K, int gamma, int V, void* stream, const int32_t* drafts,
                             const int32_t* sel, const int32_t* accept_len,
                             const int32_t* next_token, int32_t* counts, int32_t* status);

/*
 * Draws from rows of logits, and their truncation.  Rows r / per share one entry
 * of the parameters.  A row's tokens are ordered by falling logit, equal ones by
 * index, and token i weighs
 *   w_i = 2^44 e^((x_i - max x) / temperature)
 * as a whole number, the nearest or the one next to it.
 * Of that order a row keeps a first part, cut in turn by
 *   min_p  to the tokens with x_i >= max x + temperature * ln(min_p)
 *   top_k  to the first top_k
 *   top_p  to those before which less than top_p * W lies, W being the weight of
 *          what the others keep
 * and a logit of -infinity is never kept.  temperature 0 keeps the first token
 * alone.  W and its products with top_p and u are exact, so that what is kept and
 * drawn does not depend on how a row is shared out.
 *   logits     device [rows] of V logits, row_stride elements apart (0 with one
 *              row, or to draw from one row several times)
 *   temperature  device float [rows / per], 0 or 2^-64 .. 2^64, or NULL: 1
 *   top_k      device int32 [rows / per], >= 0 (0: all), or NULL
 *   top_p      device float [rows / per], in (0, 1], or NULL: 1
 *   min_p      device float [rows / per], in [0, 1], or NULL: 0
 *   kept       device int32 [rows] or NULL: how many tokens the row keeps
 * dtype SDV_BF16 or SDV_F32; any V <= 2^19, aligned to an element; rows a multiple
 * of per, below 2^31.  A row that holds a NaN or +infinity, or nothing finite,
 * sets SDV_STATUS_BAD_ROW; a parameter outside its range sets
 * SDV_STATUS_BAD_PARAM: kept is then 0, and the outputs what is said below.
 *
 * sdv_sample: the token of each row where the running sum of kept weights passes
 * u * (their sum).
 *   uniform    device float [rows], u in [0, 1)
 *   tokens     device int32 [rows]; -1 for a bad row
 *   logprob    device float [rows] or NULL: ln(w / (sum of kept weights)), with the
 *              nearest whole number for the drawn token's w; NaN for a bad row
 *
 * sdv_logits_truncate: the logits, -infinity where a token is not kept (a bad
 * row: NaN), unscaled: sdv_verify on such rows, with the same temperatures, is
 * lossless for the truncated distribution.
 *   out        device [rows] of V, out_stride elements apart; it may be logits
 *              with the same stride (in place), and must not overlap it otherwise
 */
sdv_status sdv_sample(int64_t rows, int per, int V, sdv_dtype dtype, void* stream, const void* logits,
                      int64_t row_stride, const float* temperature, const int32_t* top_k,
                      const float* top_p, const float* min_p, const float* uniform, int32_t* tokens,
                      float* logprob, int32_t* kept, int32_t* status);
sdv_status sdv_logits_truncate(int64_t rows, int per, int V, sdv_dtype dtype, void* stream,
                               const void* logits, int64_t row_stride, const float* temperature,
                               const int32_t* top_k, const float* top_p, const float* min_p, void* out,
                               int64_t out_stride, int32_t* kept, int32_t* status);

#ifdef __cplusplus
}
#endif

#endif /* SDV_H */

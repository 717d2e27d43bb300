/*
 * dspark.h -- C ABI of the MI355X (gfx950) DSpark draft-and-verify hot path.
 *
 * Pages cited (titles as published):
 *   [P1] "DSpark: Confidence-Scheduled Speculative Decoding with
 *        Semi-Autoregressive Generation 요약 설명" (summary page)
 *   [P2] "DSpark: Confidence-Scheduled Speculative Decoding with
 *        Semi-Autoregressive Generation" (notes page, "DSpark 핵심 기술")
 *
 * Conventions shared by every entry point
 *   - Tensor arguments are DEVICE pointers, row-major, owned by the caller.  The
 *     library keeps no pointer after the work it enqueued has completed and
 *     allocates no memory on the hot path (scratch comes from the caller's
 *     workspace, sized by the *_workspace_bytes queries).
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Every
 *     call is asynchronous on it; outputs are valid after the stream syncs.
 *     Calls on different streams must use different workspaces.
 *   - Arguments are checked on the host before anything is enqueued.  On error
 *     the call returns a negative dspark_status, enqueues nothing, leaves the
 *     outputs untouched and records a message for dspark_last_error().
 *   - Values the host cannot see (token ids, confidences, logits) are
 *     preconditions: token ids must lie in [0, V), confidences in [0, 1], and
 *     the logits U, T and the weights finite (a logit may be -inf to mask an
 *     entry); out-of-range values or NaN give unspecified results but every
 *     memory access stays in bounds (token ids are clamped before they index
 *     W1).
 *   - dtype: DSPARK_F32 (binary32) or DSPARK_BF16 (bfloat16 bit patterns) for
 *     U, T, W1 and W2.  The Markov-head rank must be 256 (the pages' default).
 *   - Random numbers: Philox4x32-10 (Salmon et al., SC'11) with key words
 *     (seed mod 2^32, seed >> 32) and counter (i>>2, k, r, stream), taking word
 *     i&3 of the output; r is the request index, k the 1-based block position
 *     and i the element index within the stream (a token id or a block index,
 *     below).  Uniform u = ((w>>9) + 1/2) 2^-23; Gumbel variate
 *     G(stream, r, k, i) = -ln(-ln u).
 *   - Categorical draws: every token the library samples is a two-level
 *     Gumbel-max draw from softmax(w) over a row of V log-weights w (entries may
 *     be -inf).  The vocabulary is cut into blocks b of 32 tokens
 *     [32b, 32b+32), the last one shorter when 32 does not divide V, and
 *       block  b* = argmax_b ( log sum_{v in b} exp(w_v) + G(S, r, k, b) ),
 *       token  x  = argmax_{v in b*} ( w_v + G(S + 4, r, k, v) ),
 *     the lowest block, then the lowest token, winning exact ties (a block with
 *     no finite entry never wins).  P(x = v) = softmax(w)_v exactly.  The
 *     streams S (block) / S + 4 (member) are 0 / 4 for the draft, 2 / 6 for the
 *     residual draw and 3 / 7 for the bonus draw; stream 1 holds the acceptance
 *     uniforms (element i = 0).  The library takes each decision in binary64 on
 *     the stored inputs; its binary32 screening only skips blocks that a
 *     proven error bound shows cannot win.
 *   - No C++ exception crosses this interface.
 */
#ifndef DSPARK_H_
#define DSPARK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DSPARK_OK = 0,
  DSPARK_ERR_ARG = -1,        /* null pointer or negative / zero size */
  DSPARK_ERR_SHAPE = -2,      /* unsupported dimension */
  DSPARK_ERR_DTYPE = -3,      /* unknown dtype */
  DSPARK_ERR_WORKSPACE = -4,  /* workspace missing, too small or misaligned */
  DSPARK_ERR_RANGE = -5,      /* host-visible value out of range */
  DSPARK_ERR_HIP = -6         /* HIP runtime error while enqueuing */
} dspark_status;

typedef enum { DSPARK_F32 = 0, DSPARK_BF16 = 1 } dspark_dtype;

/* One decoding round's problem: R requests, gamma block positions, vocabulary
 * V, Markov-head rank, storage dtype and the round's random seed.
 * Limits: 1 <= R <= 65536, 1 <= gamma <= 64, 1 <= V < 2^26, R*gamma <= 2^20. */
typedef struct {
  int32_t R;
  int32_t gamma;
  int32_t V;
  int32_t rank;
  int32_t dtype;
  int32_t reserved;  /* must be 0 */
  uint64_t seed;
} dspark_problem;

/* Bytes of the packed W2 operand (see dspark_pack_w2). Returns 0 on bad input. */
size_t dspark_w2_packed_bytes(const dspark_problem* p);

/* Repack the Markov-head factor W2 [rank, V] into the vocabulary-major layout
 * the kernels stream (a once-per-model weight preparation, not part of a round).
 * W2p must hold dspark_w2_packed_bytes(p) bytes, 256-byte aligned.  With
 * n = ceil(V/32) tiles of 32 tokens:
 *   bf16: tile t holds 16 steps x 64 lanes x 8 values, entry
 *         ((t*16 + s)*64 + l)*8 + e = W2[128*(l/32) + 8*s + e][32*t + pi(l%32)],
 *         pi(m) = 16*((m>>2)&1) + 4*(m>>3) + (m&3), zero beyond V (n*16 KB).
 *   f32:  W2 transposed, [n*32, rank], zero rows beyond V.
 * Then n floats: tile t's max |W2[i][v]| over i < rank and its tokens v < V
 * (the factor of the contraction's error bound). */
int dspark_pack_w2(const dspark_problem* p, const void* W2, void* W2p, void* stream);

/* Workspace bytes needed by dspark_draft_step and dspark_verify for problem p
 * (one buffer serves both when they run on one stream). 0 on bad input. */
size_t dspark_workspace_bytes(const dspark_problem* p);

/* Stage 1 -- Markov-head semi-autoregressive draft sampling.  [P1 §3.1; P2]
 * For k = 1..gamma and every request r, with x_0 = anchors[r]:
 *   z_v = U[r,k-1,v] + sum_i W1[x_{k-1}, i] W2[i, v]      (rank-256 bias B_k)
 *   lse[r,k-1]  = log sum_v exp(z_v)                     (p^d_k = softmax(z))
 *   x_k         = the two-level draw from softmax(z) with streams 0 / 4 at (r, k)
 *   logq[r,k-1] = z_{x_k} - lse[r,k-1]                   (log p^d_k(x_k))
 * U: [R, gamma, V] dtype; W1: [V, 256] dtype; W2p: packed W2; anchors: [R] int32.
 * Outputs: tokens [R, gamma] int32, lse and logq [R, gamma] float64.
 * logpd: NULL, or float32 [R, gamma, V] that receives log p^d_k(v) = z_v - lse
 * of every position (a parity / debugging output that costs a full write;
 * z in binary32, the difference in binary64 rounded to binary32).
 * ws: dspark_workspace_bytes(p) bytes, 256-byte aligned. */
int dspark_draft_step(const dspark_problem* p, const void* U, const void* W1, const void* W2p,
                      const int32_t* anchors, int32_t* tokens, double* lse, double* logq,
                      float* logpd, void* ws, size_t ws_bytes, void* stream);

/* dspark_draft_step without a workspace, for callers that cannot allocate
 * device memory (code under graph capture, tight serving loops, harnesses that
 * forbid allocation).  Same arguments, outputs and results as
 * dspark_draft_step; the draft's scratch (split records and the next
 * position's matrix-core operands) is a fixed 8 MiB device array of the
 * library instead, one per GPU, held until the process ends.  The call
 * allocates nothing and records no timing events.  Problems whose draft
 * scratch exceeds 8 MiB are rejected with DSPARK_ERR_WORKSPACE (every R up to
 * 8192 fits at V <= 2^20).  The array of the current device is used: calls
 * that overlap on one GPU (on different streams, or from different threads)
 * race on it and must be ordered by the caller; a call may start once the
 * previous call's work on that GPU has been enqueued before it on the same
 * stream, or has completed.  Nothing in the array needs to start at zero. */
int dspark_draft_step_noalloc(const dspark_problem* p, const void* U, const void* W1,
                              const void* W2p, const int32_t* anchors, int32_t* tokens,
                              double* lse, double* logq, float* logpd, void* stream);

/* Stage 2 -- standard speculative rejection sampling with bonus token, and the
 * analytic acceptance c*.  [P1 요약, §3.2.1; P2 배경]
 * For request r with verify length l_r = lengths[r] (all gamma if lengths is
 * NULL), for k = 1..l_r:
 *   p^d_k = softmax(U[r,k-1] + W1[x_{k-1}] W2) (recomputed; lse_d from stage 1)
 *   p^t_k = softmax(T[r,k-1])
 *   cstar[r,k-1] = sum_v min(p^d_k, p^t_k) = 1 - ||p^d_k - p^t_k||_1 / 2
 *   accept x_k iff ln u < ln p^t_k(x_k) - logq[r,k-1], u = uniform(stream 1, r, k, v=0)
 * n_accept[r] = number of leading accepted positions.  If a position k* <= l_r
 * is rejected, out_token[r] = the two-level draw from the normalised
 * max(0, p^t_{k*} - p^d_{k*}) (log-weights ln max(0, p^t - p^d)) with streams
 * 2 / 6 at (r, k*), or from p^t_{k*} with the same streams if no entry has
 * p^t > p^d in binary64; otherwise out_token[r] = the two-level draw from
 * softmax(T[r,l_r]) = p^t_{l_r+1} with streams 3 / 7 at (r, l_r + 1) (bonus).
 * T: [R, gamma+1, V] dtype (row gamma is the bonus row).  tokens, lse_d, logq:
 * stage-1 outputs.  lengths: [R] int32 in [0, gamma] or NULL.
 * Outputs: cstar [R, gamma] float32 (NaN for k > l_r); n_accept, out_token [R]
 * int32; accept_mask [R, gamma] uint8 or NULL (1 accepted, 0 rejected, 255 not
 * decided); lse_t [R, gamma+1] float64 or NULL (NaN where not computed). */
int dspark_verify(const dspark_problem* p, const void* U, const void* W1, const void* W2p,
                  const int32_t* anchors, const int32_t* tokens, const double* lse_d,
                  const double* logq, const void* T, const int32_t* lengths, float* cstar,
                  int32_t* n_accept, int32_t* out_token, uint8_t* accept_mask, double* lse_t,
                  void* ws, size_t ws_bytes, void* stream);

/* Confidence head with Sequential Temperature Scaling.  [P1 §3.2.1]
 * c[r,k-1] = 1 / (1 + exp(-(w . [h[r,k-1,:]; W1[x_{k-1},:]]) / temps[k-1])),
 * evaluated in float64 and rounded to float32.  h: [R, gamma, H] bfloat16;
 * w: [H + 256] float32; temps: [gamma] float32 (> 0); W1 [V, 256] in p->dtype;
 * anchors [R], tokens [R, gamma] int32.  Output c: [R, gamma] float32.
 * Limits: 1 <= H <= 65536. */
int dspark_confidence(const dspark_problem* p, int32_t H, const uint16_t* h, const float* w,
                      const float* temps, const void* W1, const int32_t* anchors,
                      const int32_t* tokens, float* c, void* stream);

/* Stages 3-4 -- prefix-survival products and the hardware-aware prefix
 * scheduler (Algorithm 1).  [P1 §3.2.2]
 *   a[r,j-1] = a[r,j-2] * c[r,j-1] in binary32, a[r,0] = c[r,0]
 *   candidates (r, j) in order of the key (-a[r,j-1], r, j); start from l = 0,
 *   B = R, tau = R, Theta = R * sps[R-1]; take candidates while
 *   Theta' = tau' * sps[B'-1] > Theta (strict), B' = B + 1, tau' = tau + a;
 *   stop at the first non-improvement (causal).  tau is accumulated exactly in
 *   units of 2^-38 (each a rounded to nearest-even), Theta = double(tau) * SPS.
 * c: [R, gamma] float32 in [0, 1]; sps: [n_sps] float32, sps[B-1] = SPS(B),
 * n_sps >= R*(gamma+1).  Outputs: a [R, gamma] float32; lengths [R] int32;
 * stats [4] float64 = (B, tau, Theta, n_selected); theta_path [R*gamma+1]
 * float64 or NULL (Theta before any candidate, then after each examined
 * candidate up to and including the stopping one, NaN afterwards).
 * Limit: R*gamma <= 16384.  No workspace is needed. */
int dspark_schedule(int32_t R, int32_t gamma, const float* c, const float* sps, int32_t n_sps,
                    float* a, int32_t* lengths, double* stats, double* theta_path, void* stream);

/* Production variant of the scheduler: capacity.  [P1 §5.2]
 * The deployed scheduler sets a round's capacity K from confidences two
 * rounds old and leaves out the early-stopping break, so that the search is
 * not caught in a local optimum at a throughput cliff of an irregular SPS(B).
 * Here: a = prefix products of c (as in dspark_schedule), candidates in the
 * same survival order, Theta_i = tau_i * sps[R+i-1] after the first i
 * candidates (i = 0..R*gamma, tau as in dspark_schedule); K = the smallest i
 * with the largest Theta_i, written to K[0] on the device (a later round reads
 * it there with no host synchronisation).  lengths [R]: the top-K verify
 * lengths on these same confidences; stats [4] = (B, tau, Theta, K) at K;
 * theta_path [R*gamma+1] float64 or NULL: every Theta_i.  sps entries must be
 * finite and >= 0.  Limit: R*gamma <= 16384. */
int dspark_schedule_capacity(int32_t R, int32_t gamma, const float* c, const float* sps,
                             int32_t n_sps, float* a, int32_t* K, int32_t* lengths,
                             double* stats, double* theta_path, void* stream);

/* Production variant of the scheduler: top-K.  [P1 §5.2]
 * Verify the first min(K[0], R*gamma) candidates (K[0] < 0 counts as 0) in the
 * survival order of this round's c; K is a device int32 (normally written by
 * dspark_schedule_capacity two rounds earlier).  a [R, gamma] float32;
 * lengths [R] int32 (prefixes, since a request's survival never rises);
 * stats [4] = (B, tau, Theta, taken), Theta = tau * sps[B-1].
 * Limit: R*gamma <= 16384. */
int dspark_schedule_topk(int32_t R, int32_t gamma, const float* c, const int32_t* K,
                         const float* sps, int32_t n_sps, float* a, int32_t* lengths,
                         double* stats, void* stream);

/* Static-threshold verify lengths.  [P1 §4.3.3]
 * a = binary32 prefix products of c [R, gamma]; lengths[r] = the largest j
 * with a[r,i-1] >= theta (compared in binary64) for every i <= j.
 * theta must not be NaN.  Limits: 1 <= R <= 65536, 1 <= gamma <= 64. */
int dspark_schedule_threshold(int32_t R, int32_t gamma, const float* c, double theta, float* a,
                              int32_t* lengths, void* stream);

/* Acceptance statistics of one verified round.  [P1 §4.3.1, §4.3.3]
 * accept_mask [R, gamma] (dspark_verify's: 1 accepted, 0 rejected, 255 not
 * verified) or NULL.  Position k counts only rollouts whose positions 1..k-1
 * were all accepted: reached[k-1] = requests with positions 1..k-1 accepted
 * and position k verified, accepted[k-1] = those that accepted position k
 * (int64 [gamma] each).  Threshold sweep (n_thr in [0, 1024]; a [R, gamma]
 * survival products, n_accept [R] the accepted lengths of a verify of all
 * gamma positions, thresholds [n_thr] float64): sweep_verified[g] = sum_r
 * l_r(thresholds[g]) with l_r as in dspark_schedule_threshold, and
 * sweep_accepted[g] = sum_r min(n_accept[r], l_r) -- the tokens a verify
 * limited by that threshold checks and accepts.  One workgroup for the mask and
 * one per threshold; no workspace. */
int dspark_acceptance_stats(int32_t R, int32_t gamma, const uint8_t* accept_mask, const float* a,
                            const int32_t* n_accept, const double* thresholds, int32_t n_thr,
                            int64_t* reached, int64_t* accepted, int64_t* sweep_verified,
                            int64_t* sweep_accepted, void* stream);

/* Sequential Temperature Scaling fit.  [P1 §3.2.1]
 * Calibrates the prefix survival on N held-out rollouts by a left-to-right
 * grid search: for j = 1..gamma, with the temperatures of positions < j fixed,
 *   a_j(T) = fl32(a_{j-1} * fl32(1 / (1 + exp(-s[n,j-1] / T)))) (binary64
 *            sigmoid rounded to binary32; a_0 = 1),
 *   N * ECE_j(T) = sum over bins b of |sum_{n in b} (y[n,j-1] - a_j(T))|, bins
 *            = min(floor(a * bins), bins - 1) over [0, 1], every a rounded to
 *            the nearest multiple of 2^-40 (exact integer sums),
 * and T_j = the grid value with the smallest ECE (lowest index on ties).
 * s: [N, gamma] float64 confidence-head scores (the logit before the sigmoid);
 * y: [N, gamma] uint8 survival labels (1 iff positions 1..j were all
 * accepted); grid: [G] float64 candidate temperatures (> 0).
 * Outputs: temps [gamma] float32 (T_j); ece_units, ece1_units [gamma] int64:
 * N * ECE in units of 2^-40 at T_j and at T = 1 (earlier positions
 * calibrated); a [N, gamma] float32, the calibrated survival.
 * ws: dspark_sts_workspace_bytes(N, gamma, G, bins) bytes, 256-byte aligned
 * (0 = bad sizes).  Limits: 1 <= N <= 2^20, 1 <= gamma <= 64, 1 <= G <= 1024,
 * 1 <= bins <= 64.  3 * gamma + 1 launches. */
size_t dspark_sts_workspace_bytes(int32_t N, int32_t gamma, int32_t G, int32_t bins);
int dspark_sts_fit(int32_t N, int32_t gamma, const double* s, const uint8_t* y, int32_t G,
                   const double* grid, int32_t bins, float* temps, int64_t* ece_units,
                   int64_t* ece1_units, float* a, void* ws, size_t ws_bytes, void* stream);

/* The tokens a verified round emits, in order.  [P1 요약]
 * ids[r, k] = tokens[r, k] for k < n_accept[r], out_token[r] at k = n_accept[r]
 * and -1 behind it; position k's distribution is row k of T.  tokens [R, gamma],
 * n_accept, out_token [R], ids [R, gamma + 1] int32; n_accept is clamped to
 * [0, gamma].  Limits: 1 <= R <= 65536, 1 <= gamma <= 64. */
int dspark_emitted_tokens(int32_t R, int32_t gamma, const int32_t* tokens, const int32_t* n_accept,
                          const int32_t* out_token, int32_t* ids, void* stream);

/* Log probabilities of given tokens, with the entropy of their distribution
 * and its most likely tokens.  For row r of logits z (V entries, the next row
 * ld entries on, ld >= V; any element-aligned start) and x = ids[r]:
 *   logprob[r] = z_x - lse,  lse = log sum_v exp(z_v)
 *   entropy[r] = -sum_v p_v log p_v (nats), p = softmax(z)
 *   top_ids[r, j], top_logprobs[r, j] = the (j + 1)-th most likely token and
 *       its log probability, j < n_top; the lower token first among equal logits.
 * Finite entries may have any magnitude (masks by the type's lowest value).  An
 * entry may be -inf (masked): its token has log probability -inf and is no
 * alternative; places without one hold id -1 and -inf.  A row whose id lies
 * outside [0, V) is skipped without being read: NaN, ids -1.  A row without a
 * finite entry, or with one that is +inf or NaN, has no distribution: NaN, ids -1.
 * logits: dtype; ids [N] int32; logprob, entropy [N] float32; top_ids int32 and
 * top_logprobs float32 [N, n_top] (NULL if n_top is 0).  Sums in binary64 over
 * binary32 exponentials (16 at a time in binary32).
 * ws: dspark_logprobs_workspace_bytes(N, V, n_top) bytes, 256-byte aligned; 0
 * bytes (ws may be NULL) where a workgroup takes a whole row.
 * Limits: 1 <= N < 2^24, 1 <= V < 2^26, 0 <= n_top <= 64. */
size_t dspark_logprobs_workspace_bytes(int32_t N, int32_t V, int32_t n_top);
int dspark_token_logprobs(int32_t dtype, int32_t N, int32_t V, int64_t ld, const void* logits,
                          const int32_t* ids, int32_t n_top, float* logprob, float* entropy,
                          int32_t* top_ids, float* top_logprobs, void* ws, size_t ws_bytes,
                          void* stream);

/* ---- Paged key/value cache -------------------------------------------------
 * What the target's verify forward pass keeps between rounds, and its pages:
 * a round appends the chunk of tokens it verifies (the anchor and the
 * scheduled drafts) and keeps the accepted ones.  Every length is on the
 * device; no call needs the host to know one.
 *
 * Storage, owned by the caller (E = 16 bytes of elements: 8 bf16, 4 f32):
 *   K [layers, pages, kv_heads, head_dim / E, page_size, E]
 *   V [layers, pages, kv_heads, page_size / E, head_dim, E]   (dtype, 16-byte aligned)
 * (the operand orders of the matrix cores).  Tables (dspark_cache_tables):
 *   table     [slots, max_pages] int32, a slot's pages in order, -1 behind them
 *   lens      [slots] int32, tokens cached
 *   held      [slots] int32, pages held (at least ceil(lens / page_size))
 *   refs      [pages] int32, slots that hold a page
 *   free_bits [ceil(pages / 32)] uint32, bit p % 32 of word p / 32: refs[p] == 0
 *   n_free    [1] int32
 * dspark_cache_init empties them; after that they change through these calls
 * only, on one stream or in an order that the caller keeps.  Pages are taken
 * lowest index first, so that equal calls give equal tables.  Slot ids, page
 * ids and lengths read from the device are checked before they index memory:
 * an invalid page holds no keys, and what would be written to it is dropped.
 * Limits: 1 <= slots <= 4096, 1 <= pages <= 2^24, page_size 16, 32, 64, 128 or
 * 256, 1 <= max_pages <= 2^20, slots * max_pages <= 2^30, max_pages * page_size
 * <= 2^30, 1 <= layers, kv_heads <= 1024, head_dim 64, 128 or 256. */
typedef struct {
  int32_t slots;
  int32_t max_pages;
  int32_t pages;
  int32_t page_size;
  int32_t layers;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t dtype;
} dspark_cache;

typedef struct {
  int32_t* table;
  int32_t* lens;
  int32_t* held;
  int32_t* refs;
  uint32_t* free_bits;
  int32_t* n_free;
} dspark_cache_tables;

/* Empty tables: every slot without tokens, every page free. */
int dspark_cache_init(const dspark_cache* c, const dspark_cache_tables* t, void* stream);

/* Forks: slot dst[i] gets the tokens of slot src[i] by sharing the pages that
 * hold them (one more reference each; nothing is copied).  Pages that src has
 * reserved behind its tokens stay its own.  status[i] = 0, or 1 for a pair that
 * is refused and changes nothing: an index outside [0, slots), a dst that holds
 * pages, a dst that an earlier pair names, or a src that is any pair's dst.
 * src, dst, status [n] int32, 1 <= n <= 4096. */
int dspark_cache_fork(const dspark_cache* c, const dspark_cache_tables* t, int32_t n,
                      const int32_t* src, const int32_t* dst, int32_t* status, void* stream);

/* Pages for add[s] more tokens of every slot (add[s] <= 0: the slot is left
 * alone; lens does not change).  A slot whose next token falls into a page that it
 * shares gets a page of its own for it: cow_src[s], cow_dst[s] name the copy to
 * make (dspark_cache_copy_pages, before the next reserve), -1 for none; when
 * every sharer of the page has an add[s] > 0, the one with the most tokens in it (the
 * lowest slot of several) keeps it: it writes behind the tokens of all others.
 * status[s]: 0; 1 out of pages (slots are served in order until one does not
 * fit; it and the later ones that need pages get none); 2 the table row is too
 * short (the slot gets none).  A slot with a status other than 0 must not
 * append.  add, status, cow_src, cow_dst [slots] int32. */
int dspark_cache_reserve(const dspark_cache* c, const dspark_cache_tables* t, const int32_t* add,
                         int32_t* status, int32_t* cow_src, int32_t* cow_dst, void* stream);

/* Ends a round: lens[s] += keep[s] + plus, clamped to [0, held * page_size], and
 * the pages behind the new length are released (a negative sum rolls back).
 * keep[s] = INT32_MIN leaves the slot alone.  After dspark_verify, keep =
 * n_accept with plus = 1 keeps the anchor and the accepted drafts; the last
 * emitted token is the next round's anchor.  keep [slots] int32. */
int dspark_cache_commit(const dspark_cache* c, const dspark_cache_tables* t, const int32_t* keep,
                        int32_t plus, void* stream);

/* Releases every page of the listed slots and empties them.  An index outside
 * [0, slots) is skipped; one listed twice is released once.  slots [n] int32,
 * 1 <= n <= 4096. */
int dspark_cache_free(const dspark_cache* c, const dspark_cache_tables* t, int32_t n,
                      const int32_t* slots, void* stream);

/* Moves the used pages to the front of the pool: with u pages in use, page
 * src[i] >= u goes to the free page dst[i] < u, both ascending, i < n_moves[0]
 * (-1 behind).  Writes the tables after the moves to `out` (which may be t, or
 * other tables while a round still reads t); the caller then copies the pages
 * (dspark_cache_copy_pages with count = n_moves).  The sources keep their
 * contents.  src, dst [pages] int32, n_moves [1] int32.
 * ws: dspark_cache_compact_workspace_bytes(c) bytes, 256-byte aligned. */
size_t dspark_cache_compact_workspace_bytes(const dspark_cache* c);
int dspark_cache_compact(const dspark_cache* c, const dspark_cache_tables* t,
                         const dspark_cache_tables* out, int32_t* src, int32_t* dst,
                         int32_t* n_moves, void* ws, size_t ws_bytes, void* stream);

/* Copies page src[i] to page dst[i] in K and V of every layer, i < n, or i <
 * min(n, count[0]) if count (device) is given.  Pairs with an index outside
 * [0, pages) are skipped.  No page may be two pairs' dst, or one's dst and
 * another's src.  src, dst [n] int32, 1 <= n <= 2^24. */
int dspark_cache_copy_pages(const dspark_cache* c, void* K, void* V, int32_t n, const int32_t* src,
                            const int32_t* dst, const int32_t* count, void* stream);

/* Writes a chunk's keys and values into one layer's pages.  Tokens are
 * flattened over the slots: slot s has rows offsets[s] .. offsets[s + 1] - 1 of
 * k and v [N, kv_heads, head_dim], row i at position lens[s] + i - offsets[s];
 * rows behind offsets[slots] belong to nobody.  The pages have to be reserved;
 * a token without one is dropped.  offsets [slots + 1] int32, from 0, not
 * falling.  Limits: 1 <= N <= 2^22. */
int dspark_cache_append(const dspark_cache* c, const dspark_cache_tables* t, int32_t layer, void* K,
                        void* V, int32_t N, const void* k, const void* v, const int32_t* offsets,
                        void* stream);

/* Attention of a chunk of new tokens per slot over the cache (after
 * dspark_cache_append wrote the chunk): row i of slot s, head h, sees the
 * positions p <= lens[s] + i - offsets[s] that are on a page of the slot,
 *   out[i, h] = sum_p softmax_p(scale q[i, h] . k[p, g]) v[p, g], g = h / (heads / kv_heads),
 * 0 if there is none.  q, out [N, heads, head_dim] dtype, flattened as in
 * dspark_cache_append; rows behind offsets[slots] are left as they were.  A
 * slot may have no rows.  Scores, sums and outputs accumulate in binary32 (bf16:
 * the weights are rounded to bf16 for the product with v; one rounding at the
 * end).  Keys and values that any of the chunk's tokens sees must be finite and the
 * scaled scores below 5e29 in magnitude; what else the pages hold does not matter.
 * out must not overlap q (a row's keys are shared out over workgroups).
 * max_chunk: the longest chunk expected, >= 1; it chooses the tiling only, any
 * chunk is computed.  scale > 0.  heads a multiple of kv_heads, N * heads <= 2^30.
 * ws: dspark_attend_workspace_bytes(c, N, heads) bytes, 256-byte aligned. */
size_t dspark_attend_workspace_bytes(const dspark_cache* c, int32_t N, int32_t heads);
int dspark_attend(const dspark_cache* c, const dspark_cache_tables* t, int32_t layer, const void* K,
                  const void* V, int32_t N, int32_t heads, const void* q, const int32_t* offsets,
                  float scale, int32_t max_chunk, void* out, void* ws, size_t ws_bytes,
                  void* stream);

/* Device-side check of the values the host cannot see, the preconditions
 * above (a debugging aid, off the hot path: one pass over every tensor given).
 * counts: int64 [6] in device memory, overwritten with the number of
 *   0: anchors [R] outside [0, V)
 *   1: tokens [R, gamma] outside [0, V)
 *   2: entries of U [R, gamma, V] that are NaN or +inf (-inf masks an entry)
 *   3: entries of T [R, gamma+1, V] that are NaN or +inf
 *   4: entries of W1 [V, 256] and W2 [256, V] (as given to dspark_pack_w2)
 *      that are NaN or infinite
 *   5: confidences c [R, gamma] (float32) outside [0, 1] or NaN.
 * Any tensor may be NULL (its count stays 0).  U, T, W1 and W2 are in p->dtype
 * and must be aligned to their element size, the int32 / float32 tensors to 4
 * bytes and counts to 8. */
int dspark_check_inputs(const dspark_problem* p, const void* U, const void* T, const void* W1,
                        const void* W2, const int32_t* anchors, const int32_t* tokens,
                        const float* c, int64_t* counts, void* stream);

/* Message for the last failing call on this thread ("" if none). */
const char* dspark_last_error(void);

/* Per-kernel timing with HIP events (tracing; off by default).
 * dspark_timing_enable(1) clears the record and brackets every kernel the
 * library enqueues from then on with a pair of events on that kernel's
 * stream; dspark_timing_enable(0) stops recording.  dspark_timing_report
 * waits for the recorded events and writes one line per kernel name,
 * "name launches total_ms\n", into buf (NUL-terminated, truncated to cap),
 * then clears the record; with buf NULL it only returns the size and keeps
 * the record.  Returns the bytes needed (excluding the NUL) or a negative
 * dspark_status. */
int dspark_timing_enable(int on);
int dspark_timing_report(char* buf, size_t cap);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_H_ */

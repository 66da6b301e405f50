/*
 * domino_head.h -- C ABI of the MI355X (gfx950) Domino head drafting library.
 *
 * The Domino head (paper.oopus.info review of "Domino: Decoupling Causal
 * Modeling from Autoregressive Drafting in Speculative Decoding", section 二,
 * 第二步 Domino Head) turns the output of a parallel draft backbone -- hidden
 * states H and base logits L_base for a whole block, produced in one forward
 * pass (same section, 第一步; news.sig.ai article, section "Domino怎么做") --
 * into a causally consistent greedy draft.  For block positions p = 0..K-1:
 *
 *     u_p       = SiLU(W1 [H_p ; S_p])                    (rank r, no bias)
 *     L_final_p = L_base_p + W2 u_p                        (logit space)
 *     t_p       = argmax_v L_final_p[v]                    (greedy decoding)
 *     S_{p+1}   = GRU(E[x_p], S_p),  x_p = t_p or teacher[p]
 *
 * with S_0 = GRU(E[last_tok], S_init) (anchor step on the last confirmed
 * token; S_init = 0 when not given).  GRU is PyTorch's GRUCell: rows of
 * W_ih/W_hh/b_ih/b_hh in blocks (reset, update, new);
 *     r = sig(W_ir x + b_ir + W_hr s + b_hr), z = sig(W_iz x + b_iz + W_hz s + b_hz),
 *     n = tanh(W_in x + b_in + r * (W_hn s + b_hn)),  s' = (1 - z) * n + z * s.
 * SiLU(a) = a * sig(a).  Ties in the argmax go to the lowest index; a NaN
 * logit counts as larger than any number (the first NaN wins); -0 equals +0.
 * The head state S and all accumulation are float32.
 *
 * Every entry point returns 0 on success or a negative DOMINO_E* code; the
 * message of the last failure on the calling thread is domino_last_error().
 * Device work is asynchronous and ordered on the given HIP stream (NULL =
 * the null stream); nothing synchronizes except domino_head_check_error.
 * All tensors are row-major and contiguous, owned by the caller, and every
 * device pointer must be 16-byte aligned.
 */
#ifndef DOMINO_HEAD_H
#define DOMINO_HEAD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- error codes ---- */
#define DOMINO_OK 0
#define DOMINO_EINVAL (-1)      /* bad argument: NULL, misaligned, B out of range, K > 16 */
#define DOMINO_EUNSUPPORTED (-2) /* dimensions or dtype the kernels do not handle */
#define DOMINO_EWORKSPACE (-3)  /* workspace missing or smaller than domino_head_workspace_size */
#define DOMINO_EHIP (-4)        /* a HIP runtime call failed (message carries the HIP error) */
#define DOMINO_EDEVICE (-5)     /* domino_head_check_error found device-side flags */

/* ---- weight storage types ---- */
#define DOMINO_F32 0
#define DOMINO_BF16 1

/* ---- device-side flags reported by domino_head_check_error ---- */
#define DOMINO_FLAG_BAD_TOKEN 1u      /* a last_tok or used teacher id was outside [0, V) */
#define DOMINO_FLAG_SYNC_TIMEOUT 2u   /* a grid barrier spin limit ran out; outputs invalid */

/* ---- config.flags bits (execution strategy).  For B <= 8 every launch gives the same bits; for
 * B > 8 the launches round u to one bf16 matrix-core operand and agree with each other up to the
 * order of float32 sums (the logits move by at most about 1e-2 against the oracle either way) ---- */
#define DOMINO_EXEC_AUTO 0u        /* pick per call from B: the persistent launch for B <= 8, and for
                                      8 < B <= 256 where the batched persistent launch is available (see
                                      below); the step launches otherwise */
#define DOMINO_EXEC_PERSISTENT 1u  /* one cooperative launch covering all K positions: B <= 8, or (bf16
                                      weights, r = 256, DOMINO_FOLD_EMBED or DOMINO_MARKOV, h a multiple
                                      of 64, d of 32) B <= 256, where the GRU update and state products
                                      (for a Markov head, the table gather that forms u) are spread over
                                      the grid; either way each block keeps its W2 slice on chip */
#define DOMINO_EXEC_STEPWISE 2u    /* one launch per phase and position */
#define DOMINO_EXEC_STREAM_W2 8u   /* persistent launch: stream W2 from memory at every position instead of
                                      keeping the slice on chip (bf16, r = 256); for comparison */
#define DOMINO_FOLD_EMBED 4u       /* precompute P = E W_ih^T + b_ih ([V, 3h] float32, in the workspace) at
                                      create time, so each GRU step gathers one row of P instead of
                                      multiplying W_ih by the embedding row (same values up to rounding) */
#define DOMINO_EXEC_PLAIN_LAUNCH 16u /* persistent launch as an ordinary kernel launch instead of a
                                      cooperative one (about 17 us less dispatch time per call).  Its
                                      blocks (one per compute unit) wait for each other, so the caller
                                      guarantees that no other kernel that waits for other work (in
                                      particular no other persistent draft) runs on the device at the
                                      same time; otherwise the bounded waits time out and the call
                                      reports DOMINO_FLAG_SYNC_TIMEOUT.  A process that needs the
                                      persistent launch while another process that has made
                                      cooperative launches on the same GPU is alive sets this flag:
                                      the HIP runtime refuses that second process's cooperative
                                      launches (the draft returns DOMINO_EHIP, "the operation cannot
                                      be performed in the present state") */

#define DOMINO_EXEC_POSITION_BATCHED 32u /* with a teacher: take the step launches even for B <= 8.  With
                                      a teacher the states of all positions follow from the given
                                      tokens alone, so the step launches run the GRU chain first and
                                      then the W2 products of all K positions as one launch over B*K
                                      rows (W2 read once instead of K times); they always do this
                                      when a teacher is given.  Same values as the per-position
                                      launches, bit for bit */

#define DOMINO_LBASE_BF16 64u         /* domino_head_draft's L_base holds bfloat16 bit patterns instead of
                                      float32: half the bytes of the base-logit stream, which dominates
                                      at large B.  Every path widens each value exactly, so the draft
                                      equals a float32 call on the widened values bit for bit */

/* ---- config.flags bit that changes the model ---- */
#define DOMINO_MARKOV 128u            /* Markov head instead of the recurrent one.  The news.sig.ai
                                      article (section 从Domino看DSpark) names a Markov head, DSpark's
                                      default, beside an RNN head that corresponds to Domino's causal
                                      encoder, and gives no formula.  Reading taken: each position is
                                      conditioned on the token before it alone, S_p = GRU(E[x_p], 0)
                                      with x_0 = last_tok and x_p = t_{p-1} (or teacher[p-1]), so
                                      W1_S S_p is a row of the per-token table M = W1_S GRU(E[t], 0)
                                      ([V, r] float32 in the workspace, filled at create) and
                                      u_p = SiLU(W1_H H_p + M[x_p]).  The same weights serve both
                                      heads.  Not combinable with DOMINO_FOLD_EMBED or
                                      DOMINO_EXEC_STREAM_W2; domino_head_draft then takes no S_init
                                      and writes no S_out (both must be NULL) */

/*
 * Head configuration.  All weight pointers are DEVICE pointers, borrowed for
 * the lifetime of the handle (never copied, never written), stored in
 * `wdtype` (float32, or bfloat16 as raw 16-bit patterns):
 *   W1   [r, d+h]  columns 0..d-1 multiply H_p, columns d..d+h-1 multiply S_p
 *   W2   [V, r]
 *   W_ih [3h, d], W_hh [3h, h]   GRU weights, row blocks (reset, update, new)
 *   b_ih [3h], b_hh [3h]         GRU biases, NULL means zero
 *   E    [V, d]                  token embedding table (the GRU input rows)
 * Limits: 1 <= K <= 16; d, h multiples of 8, h <= 2048; r/8 (bf16) or r/4
 * (float32) a power of two, r <= 1024; 1 <= max_batch <= 1024; V >= 1.
 */
typedef struct domino_head_config {
    int32_t d, h, r, V, K, max_batch;
    int32_t wdtype;
    uint32_t flags;
    const void *W1, *W2, *W_ih, *W_hh, *b_ih, *b_hh, *E;
} domino_head_config;

typedef struct domino_head *domino_head_t;

/* Host only.  Bytes of device workspace a handle with this config needs. */
int domino_head_workspace_size(const domino_head_config *cfg, size_t *bytes);

/*
 * Validates cfg and binds the caller-allocated device `workspace` (>=
 * domino_head_workspace_size bytes, 256-byte aligned, not shared with another
 * handle).  No allocation.  Without DOMINO_FOLD_EMBED or DOMINO_MARKOV no
 * device work either; with one of them, kernels fill the folded table (or the
 * Markov table, in chunks of tokens through a create-time region of the
 * workspace) on the null stream and create
 * waits for it.  On success *out is a new handle; release it with
 * domino_head_destroy.  The workspace state is cleared by the first draft.
 */
int domino_head_create(const domino_head_config *cfg, void *workspace, size_t workspace_bytes,
                       domino_head_t *out);

/*
 * Draft one block for B rows (1 <= B <= max_batch).  Device pointers:
 *   H        [B, K, d]  wdtype     backbone hidden states of the block
 *   L_base   [B, K, V]  float32    backbone base logits of the block (bfloat16
 *                                  bit patterns with DOMINO_LBASE_BF16)
 *   last_tok [B]        int32      last confirmed token (anchor GRU input)
 *   teacher  [B, K]     int32      NULL = free running; else teacher forcing:
 *                                  teacher[b][p] replaces t_p as GRU input for
 *                                  p <= K-2 (teacher[b][K-1] is never read)
 *   S_init   [B, h]     float32    NULL = zero initial state
 * Outputs (device):
 *   tokens   [B, K]     int32      greedy draft t_0..t_{K-1}; -1 for every
 *                                  position of a row whose last_tok or used
 *                                  teacher id lies outside [0, V)
 *   L_final  [B, K, V]  float32    NULL = not stored
 *   S_out    [B, K, h]  float32    NULL = not stored; S_0..S_{K-1}
 *   u_out    [B, K, r]  float32    NULL = not stored; u_0..u_{K-1}
 * Outputs may not alias inputs.  One draft may be in flight per handle (the
 * workspace is reused); calls on one handle must be ordered on one stream.
 * Bad token ids and barrier timeouts never abort: they set device flags read
 * by domino_head_check_error.
 */
int domino_head_draft(domino_head_t hd, int32_t B, const void *H, const void *L_base, const int32_t *last_tok,
                      const int32_t *teacher, const float *S_init, int32_t *tokens, float *L_final, float *S_out,
                      float *u_out, void *stream);

/*
 * Verify-side accept length (paper.oopus.info review, section 一; the
 * researchpapers.dev summary, 关键结果: the verifier keeps the longest draft
 * prefix that equals its own tokens).  Device pointers: draft, target [B, K]
 * int32; out_len [B] int32 receives the first p with draft[b][p] !=
 * target[b][p], or K when the whole row matches.  0 <= B, 1 <= K <= 16;
 * B = 0 is a no-op.  Raw int32 comparison, asynchronous on `stream`.
 */
int domino_accept_len(int32_t B, int32_t K, const int32_t *draft, const int32_t *target, int32_t *out_len,
                      void *stream);

/*
 * Greedy verify step of speculative decoding (paper.oopus.info review, section
 * 一: the target model checks the whole drafted block in one parallel pass and
 * keeps what it would have produced itself; researchpapers.dev summary, 关键结果
 * and 常见问题: every accepted token is the target's own).  Device pointers:
 *   logits   [B, K+1, V] float32  target logits; row j scores the token after
 *                                 the context plus draft[b][0..j-1], row K
 *                                 follows the whole draft
 *   draft    [B, K] int32         the drafted block (e.g. domino_head_draft's
 *                                 tokens; -1 entries simply never match)
 *   workspace                     >= domino_verify_workspace_size(B, K, V) bytes,
 *                                 scratch for this call (contents need no
 *                                 initialisation and are not read afterwards)
 * Outputs (device):
 *   target   [B, K+1] int32       NULL = not stored; argmax of each row, with
 *                                 the draft's rules (lowest index on ties, a
 *                                 NaN above every number, -0 == +0)
 *   accept   [B] int32            first j < K with draft[b][j] != target[b][j],
 *                                 else K
 *   next     [B] int32            target[b][accept[b]]: the target's token after
 *                                 the accepted prefix; the step commits
 *                                 draft[b][0..accept-1] and then this token,
 *                                 which is the next block's last_tok
 * 0 <= B; 1 <= K <= 16; V >= 1.  B = 0 is a no-op.  All pointers 16-byte
 * aligned; outputs may not alias inputs or the workspace.  Two kernel launches,
 * asynchronous on `stream`; no allocation, no synchronization.
 */
int domino_verify_workspace_size(int32_t B, int32_t K, int32_t V, size_t *bytes);
int domino_verify(int32_t B, int32_t K, int32_t V, const float *logits, const int32_t *draft, void *workspace,
                  size_t workspace_bytes, int32_t *target, int32_t *accept, int32_t *next, void *stream);

/*
 * domino_verify without a workspace, for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc.  Same arguments, outputs and results as domino_verify
 * (same kernels), but the per-call scratch (one 8-byte key per (row, chunk))
 * lives in a 1 MiB static device array of the library, one per device, held
 * until the process ends.  Nothing is allocated and nothing needs clearing
 * (every scratch word a call reads it has written first).  Returns
 * DOMINO_EUNSUPPORTED, before any device work, when
 * domino_verify_workspace_size(B, K, V) exceeds 1 MiB (about B (K+1) + 2048 >
 * 131072).  All calls on one device share the array: calls that may overlap
 * on one device (different streams, or host threads) race and give wrong
 * results; order them on one stream.
 */
int domino_verify_noalloc(int32_t B, int32_t K, int32_t V, const float *logits, const int32_t *draft,
                          int32_t *target, int32_t *accept, int32_t *next, void *stream);

/*
 * ---- operators over vocabulary rows: top logits, beam selection, distillation ----
 *
 * Rows of logits [B, R, V] (R: the K+1 rows of a verified block, the K rows of a draft, the beams of a
 * search).  `data` is a device pointer of `dtype` (DOMINO_F32, or DOMINO_BF16 as raw 16-bit patterns) with
 * any element alignment; strides count elements, so that a slice of a larger tensor or a padded vocabulary
 * is passed as it is.  0 <= batch_stride, 0 <= row_stride; an output's rows may not overlap.  Every call takes
 * B R (V / 1024 + 1) < 2^24 (DOMINO_EUNSUPPORTED above).  A temperature is a double: one of 0.7 in float32 moves
 * z / temperature by 1.7e-8 of itself, which a loss of rows whose logits reach 20 shows.  An output that shares memory with an input, another
 * output or the workspace is refused (DOMINO_EINVAL), but for the gradient in the logits' own rows; rows that lie
 * between each other's in one buffer share none.
 */
typedef struct domino_logits {
    const void *data;
    int64_t batch_stride, row_stride;
    int32_t B, R, V, dtype;
} domino_logits;
typedef domino_logits domino_rows; /* the same for other operands: rows of V elements each */

/*
 * The k largest logits of every row, and the row's log-sum-exp: what a teacher leaves behind for
 * domino_distill, and what sampling from the head of the distribution needs.
 *   n_rows  [B] int32           NULL = all R; else rows r >= n_rows[b] are left out (not read)
 *   workspace                   >= domino_top_logits_workspace_size bytes; scratch of this call (where that is
 *                               0, NULL will do)
 * Outputs (device):
 *   ids     [B, R, k] int32     the k largest, largest first; ties go to the lowest id, a NaN counts as
 *                               larger than any number, -0 equals +0; -1 in rows left out
 *   values  [B, R, k] float32   their logits (-inf in rows left out)
 *   lse     [B, R]    float32   log sum_v exp(z_v / temperature): -inf where every logit is -inf and in rows
 *                               left out, +inf where one is +inf, NaN where one is NaN; infinite, too, where it
 *                               exceeds float32 (logits at the type's lowest value, temperatures below 1)
 * 0 <= B, 1 <= R, 1 <= k <= 128, k <= V <= 524288, 1e-4 <= temperature <= 1e4; B = 0 is a no-op.  ids
 * and values do not depend on how a row is split over the device (V, k and B R decide that); the last place
 * of lse may.  At most two launches, asynchronous on `stream`; no allocation, no synchronization.  Pointers
 * other than logits->data 16-byte aligned; outputs may not alias inputs or the workspace.
 */
int domino_top_logits_workspace_size(const domino_logits *logits, int32_t k, size_t *bytes);
int domino_top_logits(const domino_logits *logits, int32_t k, double temperature, const int32_t *n_rows,
                      void *workspace, size_t workspace_bytes, int32_t *ids, float *values, float *lse, void *stream);

/*
 * One step of beam search.  Row w of batch entry b holds the logits of beam w (W = logits->R beams).  The
 * candidates are all (w, v), with
 *     score(w, v) = scores[b][w] + z_wv - log sum_u exp(z_wu),
 * and the n_out best of them become the beams of the next step: higher scores first, equal ones by lowest
 * w, then lowest v (a beam's own candidates are ordered by their logits).  Scores are compared in 64 bits, and so are
 * the rows' sums of exponentials joined: exponentials, and the sums of the 64 at most that one thread takes, are
 * float32.
 *   - A beam whose score is -inf is dead: its candidates score -inf.  So do tokens whose logit is -inf, in a
 *     row of nothing but -inf too.
 *   - An ended beam (finished[b][w] != 0) has one candidate, (w, eos), with the score it has; the others
 *     score -inf.
 *   - A score of NaN or +inf, or a row with a NaN or +inf logit, makes a beam's candidates NaN, which counts
 *     as larger than any number: it shows in the result, from token 0 on.
 *   Rows of dead and ended beams are not read.  Candidates of -inf are taken, by their places, only when
 *   nothing else is left; parent and token are valid indices then, too.
 * Inputs (device): scores [B, W] float32; finished [B, W] bytes or NULL; state [B, W, state_bytes] or NULL
 * (any beam state, state_bytes a positive multiple of 4); history [B, W, T] int32 or NULL.
 * Outputs (device): out_scores [B, n_out] float32; out_parent, out_token [B, n_out] int32; out_finished
 * [B, n_out] bytes, NULL = not stored (the parent had ended, or the token is eos); out_state [B, n_out,
 * state_bytes]: the parent's state; out_history [B, n_out, T]: the parent's history with token at `step`.
 * eos: the end token, or -1 for none (then finished must be NULL).
 * Limits: 1 <= W <= 32, 1 <= n_out <= 128, n_out <= W V, V <= 524288, 0 <= step < T.  B = 0 is a no-op.  At
 * most two launches, asynchronous on `stream`; no allocation, no synchronization.  Pointers other than
 * logits->data 16-byte aligned; outputs may not alias inputs or the workspace.
 */
typedef struct domino_beam {
    int32_t n_out, eos, T, step;
    int64_t state_bytes;
    const float *scores;
    const uint8_t *finished;
    const void *state;
    const int32_t *history;
    float *out_scores;
    int32_t *out_parent, *out_token;
    uint8_t *out_finished;
    void *out_state;
    int32_t *out_history;
} domino_beam;

int domino_beam_step_workspace_size(const domino_logits *logits, int32_t n_out, size_t *bytes);
int domino_beam_step(const domino_logits *logits, const domino_beam *beam, void *workspace, size_t workspace_bytes,
                     void *stream);

/*
 * Distillation of a student's rows from a teacher's top logits.  With y = z / temperature, q = softmax(y),
 * the entries j of a row whose id lies in [0, V), t_j = values_j / temperature - L, p_j = exp(t_j):
 *     L = teacher_lse where given (domino_top_logits' lse at this temperature), else log sum_j exp(values_j /
 *         temperature): the teacher's distribution over its entries alone
 *     rest = max(0, 1 - sum_j p_j) where teacher_lse is given (the mass of all other ids, taken as one
 *         event), else 0;  Qr = the sum of q over the ids that no entry names
 *     loss = temperature^2 ( sum_j p_j (t_j - log q_j) + rest log(rest / Qr) )
 * teacher_lse is a float32, which leaves a relative error of |L| 2^-24 in every p_j and as much of a mass open: at a
 * logit of 20, 1e-6 at temperature 1 and 1e-5 at 0.1.  With
 *     noise = (|L| + 32) 2^-24
 * a row counts as given without teacher_lse (rest = 0, the p_j brought to a sum of 1) where | 1 - sum_j p_j | <= noise
 * and Qr <= noise^2: the teacher's mass of the other ids cannot be told from none there, and the student has none.  So
 * a student that equals its teacher has a loss of 0 where the entries hold all there is (k = V, or a mask that leaves
 * no more than k), and one of at most about temperature^2 noise log(1 / noise) elsewhere.  An L whose noise exceeds
 * 2^-6 (|L| near 2^18: temperatures near 1e-4; rows at the type's lowest value, an L of -inf beside values that are
 * not) says nothing of the other ids' mass: such a row counts as given without it, too.
 * An id outside [0, V) (-1 pads a row) is passed over; an id named twice has both masses.  A row without a
 * valid id, one whose entries' values are all -inf (with teacher_lse: and that is -inf too, as domino_top_logits
 * leaves a row of nothing but -inf), and rows r >= n_rows[b] are left out: loss 0, gradient 0, whatever their
 * logits hold.  A row of nothing but -inf has q = 0; a NaN or +inf among a row's logits makes its loss and
 * gradient NaN.
 *   ids        [B, R, k] int32, values [B, R, k] float32, teacher_lse [B, R] float32 or NULL
 *   n_rows     [B] int32 or NULL (all R)
 *   workspace  >= domino_distill_workspace_size bytes; scratch of this call (where that is 0, NULL will do)
 *   loss       [B, R] float32
 *   stats      [B, R, 4 + k] float32: what the backward pass needs of the forward pass; NULL = not stored
 *   grad_loss  [B, R] float32 or NULL.  Given, the call also writes the gradient grad_loss[b][r] *
 *              dloss/dz to `grad` (then not NULL), and stats must be NULL
 *   grad       same dtype, B, R and V as the logits; its rows may be the logits' own (same data, and strides
 *              where a dimension is longer than 1: the gradient takes their place) or lie apart from them
 * domino_distill_backward writes the gradient from the forward pass' stats, with the same logits, ids,
 * temperature and n_rows.  0 <= B, 1 <= R, 1 <= V, 1 <= k <= 128, 1e-4 <= temperature <= 1e4; B = 0 is a
 * no-op.  The sum over the ids that no entry names is float32 within a wave's elements and 64 bits across, the
 * entries' terms are in 64 bits, stats are float32; results do not change from call to call.  At most two launches for the loss and one for the gradient, asynchronous on `stream`; no
 * allocation, no synchronization.  Pointers other than the logits' and the gradient's data 16-byte aligned;
 * apart from what is said of grad, outputs may not alias inputs or the workspace.
 */
int domino_distill_workspace_size(const domino_logits *logits, int32_t k, size_t *bytes);
int domino_distill(const domino_logits *logits, int32_t k, const int32_t *ids, const float *values,
                   const float *teacher_lse, double temperature, const int32_t *n_rows, void *workspace,
                   size_t workspace_bytes, float *loss, float *stats, const float *grad_loss,
                   const domino_logits *grad, void *stream);
int domino_distill_backward(const domino_logits *logits, int32_t k, const int32_t *ids, const float *stats,
                            const float *grad_loss, double temperature, const int32_t *n_rows,
                            const domino_logits *grad, void *stream);

/*
 * Log-probabilities of given tokens, the entropies of their rows, and the likeliest alternatives.  With y = z /
 * temperature, p = softmax(y), w the row's token:
 *     logprob = log p_w       entropy = - sum_v p_v log p_v (0 log 0 = 0)
 *     alternatives: the k largest logits' ids, in the order of domino_top_logits, and log p of each
 *     dlogprob/dz_v = (1[v = w] - p_v) / temperature       dentropy/dz_v = - p_v (log p_v + entropy) / temperature
 * Rows r >= n_rows[b], and rows whose token lies outside [0, V) (-1 ignores a row), are left out: not read, logprob,
 * entropy and gradient 0, ids -1, their log-probabilities -inf.  A logit of -inf has probability 0; a row of nothing but
 * -inf has logprob -inf, entropy 0, alternatives of -inf and gradient 0.  A NaN or +inf among a row's logits makes its
 * logprob, entropy, alternatives' log-probabilities and gradient NaN (the ids stay those of domino_top_logits).  A
 * log-probability below float32's range (logits at the type's lowest value, temperatures below 1) is -inf.
 *   tokens        [B, R] int32
 *   k             alternatives, 0 for none; ids [B, R, k] int32 and logprobs [B, R, k] float32, NULL with k = 0
 *   n_rows        [B] int32 or NULL (all R)
 *   workspace     >= domino_token_logprobs_workspace_size bytes; scratch of this call (where that is 0, NULL will do)
 *   logprob, entropy  [B, R] float32
 *   stats         [B, R, 8] float32: what the backward pass needs of the forward pass; NULL = not stored
 *   grad_logprob, grad_entropy  [B, R] float32 or NULL (0).  One given, the call also writes grad_logprob dlogprob/dz +
 *                 grad_entropy dentropy/dz to `grad` (then not NULL); stats must be NULL and k 0
 *   grad          as for domino_distill: the logits' own rows, or apart from them
 * domino_token_logprobs_backward writes the gradient from the forward pass' stats, with the same logits, tokens,
 * temperature and n_rows.  0 <= B, 1 <= R, 1 <= V, 0 <= k <= 128, 1e-4 <= temperature <= 1e4; with alternatives k <= V <=
 * 524288.  B = 0 is a no-op.  A thread's sums are float32, all others 64 bits; the largest element of a row is taken
 * apart from its sums, so that rows that are nearly certain keep their digits.  Results do not change from call to
 * call.  At most two launches forward and one backward, asynchronous on `stream`; no allocation, no synchronization.
 * Pointers other than the logits' and the gradient's data 16-byte aligned; outputs may not alias inputs or the workspace.
 */
int domino_token_logprobs_workspace_size(const domino_logits *logits, int32_t k, size_t *bytes);
int domino_token_logprobs(const domino_logits *logits, const int32_t *tokens, int32_t k, double temperature,
                          const int32_t *n_rows, void *workspace, size_t workspace_bytes, float *logprob, float *entropy,
                          int32_t *ids, float *logprobs, float *stats, const float *grad_logprob,
                          const float *grad_entropy, const domino_logits *grad, void *stream);
int domino_token_logprobs_backward(const domino_logits *logits, const int32_t *tokens, const float *stats,
                                   const float *grad_logprob, const float *grad_entropy, double temperature,
                                   const int32_t *n_rows, const domino_logits *grad, void *stream);

/*
 * ---- layers: embedding, linear, and their gradients ----
 *
 * Operands are rows of V elements, [B, R, V] as for logits: any element alignment and strides, float32 or bfloat16 each
 * for itself, B R (V / 1024 + 1) < 2^24 for each of them (a table or weights among them).  A table or a weight matrix has B = 1.  An output that shares memory with an input, another output or
 * the workspace is refused (DOMINO_EINVAL) but where it says otherwise, as are outputs whose rows overlap.
 *
 * Embedding: out_i = scale * table[ids_i], 0 where ids_i is outside [0, rows of the table).  ids [B, R] int32.
 * Computed in float32 and rounded once.  One launch.
 *
 * domino_embed_backward: table[v] = scale * sum of grad_i over the i with ids_i = v, for every row v; with accumulate
 * != 0 that is added to the rows that ids name, and the others stay as they are.  Ids outside the table are passed
 * over.  Each token's rows are added in float32: up to 256 tokens in the order of their places; more are sorted, and a
 * token's are added in that order within tiles of up to 64, whose sums are added in theirs.  The result does not change
 * from call to call.  `table` is the gradient, of type and shape of its own ([1, rows, V]).  workspace >=
 * domino_embed_backward_workspace_size bytes, 16-byte aligned (where that is 0, NULL will do).  One launch for up to 256
 * tokens, three for up to 8192, above that two and three more for each 6 bits of the table's number of rows.
 * V <= 2^20, scale finite in float32.  B = 0: nothing to look up; the gradient is 0 (without accumulate).
 * Asynchronous on `stream`; no allocation, no synchronization.
 */
int domino_embed(const domino_rows *table, const int32_t *ids, double scale, const domino_rows *out, void *stream);
int domino_embed_backward_workspace_size(const domino_rows *grad, size_t *bytes);
int domino_embed_backward(const domino_rows *grad, const int32_t *ids, double scale, int32_t accumulate,
                          void *workspace, size_t workspace_bytes, const domino_rows *table, void *stream);

/*
 * Linear layer: y = act(x weight^T + bias) + residual.
 *   x [B, R, K], weight [1, N, K], bias [1, 1, N] or NULL, residual [B, R, N] or NULL, y [B, R, N], pre [B, R, N] or
 *   NULL: x weight^T + bias, which the backward pass of an activation takes
 *   activation: DOMINO_NO_ACT, DOMINO_SILU (a sigmoid(a)), DOMINO_GELU (a Phi(a), Phi the normal distribution's
 *   function), DOMINO_RELU
 * Gradient, from grad = dloss/dy: with dpre = grad act'(pre),
 *   grad_x [B, R, K] = dpre weight, grad_weight [1, N, K] = dpre^T x, grad_bias [1, 1, N] = sum of dpre over the rows;
 *   NULL: not wanted (not all three).  pre: NULL without an activation.  accumulate != 0: grad_weight and grad_bias
 *   are added to what is there (grad_x is not).  relu's slope at 0 is 0.  The residual's gradient is grad itself.
 * Operands are multiplied as they are: products of bfloat16 are exact, float32 operands go in three parts of 8 bits, so
 * that two of them multiply to 2^-24 of the product (below 2^-100 a part may fall under the type's range); sums are
 * float32, and each output is rounded once.  Infinities and NaN of the operands, and sums past float32, give what these
 * products and sums give: infinity times a number that is not 0 is infinite, times 0 NaN, infinities of both signs add up
 * to NaN (a float32 operand beside them makes such a tile take about three times as long).  silu and gelu of -inf, and their
 * slopes at infinities, are NaN, as their formulas give.
 * Results do not change from call to call; the last places of an element may depend on the other sizes of the call.
 * workspace >= domino_linear_workspace_size (x and weight: sizes and types alone) or domino_linear_backward_workspace_size (grad,
 * x, weight, and which gradients are wanted: likewise) bytes, 16-byte aligned (where that is 0, NULL will do).
 * y may be the residual (same data, and strides where a dimension is longer than 1).
 * B R, N and K below 2^24 each besides, with gelu B R N below 2^33.  B = 0: y has no rows; grad_weight and grad_bias are 0 (without accumulate).
 * At most two launches forward and six backward, asynchronous on `stream`; no allocation, no synchronization.
 */
#define DOMINO_NO_ACT 0
#define DOMINO_SILU 1
#define DOMINO_GELU 2
#define DOMINO_RELU 3

int domino_linear_workspace_size(const domino_rows *x, const domino_rows *weight, int32_t activation, size_t *bytes);
int domino_linear(const domino_rows *x, const domino_rows *weight, const domino_rows *bias, int32_t activation,
                  const domino_rows *residual, void *workspace, size_t workspace_bytes, const domino_rows *y,
                  const domino_rows *pre, void *stream);
int domino_linear_backward_workspace_size(const domino_rows *grad, const domino_rows *x, const domino_rows *weight,
                                          int32_t activation, int32_t want_x, int32_t want_weight, int32_t want_bias,
                                          size_t *bytes);
int domino_linear_backward(const domino_rows *grad, const domino_rows *x, const domino_rows *weight,
                           const domino_rows *pre, int32_t activation, int32_t accumulate, void *workspace,
                           size_t workspace_bytes, const domino_rows *grad_x, const domino_rows *grad_weight,
                           const domino_rows *grad_bias, void *stream);

/*
 * Synchronizes the device (every stream, so drafts replayed from a captured
 * HIP graph on any stream are included), reads and clears the device flags
 * (DOMINO_FLAG_*) into *device_flags (may be NULL) and resets the handle's
 * barrier state (the next draft clears it on the device before it runs).
 * Returns DOMINO_EDEVICE if any flag was set.
 */
int domino_head_check_error(domino_head_t hd, uint32_t *device_flags);

/*
 * Host only, no device work.  Which launch domino_head_draft takes for B rows
 * on this handle: *persistent = 1 for the single cooperative launch that runs
 * the whole drafting loop, 0 for one launch per step; *w2_resident = 1 when
 * that persistent launch keeps each block's share of W2 on chip across the K
 * positions instead of re-reading it; *grid = blocks of the persistent launch
 * (0 for the per-step launches).  Output pointers may be NULL.  Same errors as
 * domino_head_draft for B and for a forced persistent launch that cannot run.
 */
int domino_head_exec_info(domino_head_t hd, int32_t B, int32_t *persistent, int32_t *w2_resident, int32_t *grid);

/*
 * Host only.  Bound on every device-side wait of later drafts on this handle
 * (grid barriers, argmax and operand arrivals), in polling iterations of
 * roughly 0.1-1 us each.  A wait that runs out sets DOMINO_FLAG_SYNC_TIMEOUT
 * and its block leaves the launch, so every launch ends even if a block never
 * arrives.  The default is 2^22 (or DOMINO_BARRIER_SPIN_LIMIT from the
 * environment at create); 0 makes every wait give up at once, which forces
 * the timeout path from the host.
 */
int domino_head_set_spin_limit(domino_head_t hd, uint32_t limit);

/*
 * Host only.  Parameters of the head: r(d+h) + V r + 3h d + 3h h (+ 6h if GRU
 * biases are given); the embedding table E is the target's and not counted.
 * The paper.oopus.info review (section 二, 第二步 Domino Head) puts the head at
 * about 56 million parameters, 5.3% of the drafter: 55,934,976 (+6,144 biases)
 * at d = 4096, h = 1024, r = 256, V = 151936.
 */
int domino_head_param_count(const domino_head_config *cfg, int64_t *n);

/* Releases the handle (not the workspace or the weights).  NULL is a no-op. */
void domino_head_destroy(domino_head_t hd);

/* Message of the last failed call on this thread ("" if none). */
const char *domino_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* DOMINO_HEAD_H */

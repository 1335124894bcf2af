/*
 * spec_verify.h -- C ABI of the MI355X (gfx950) batched draft-verification
 * library.
 *
 * The operation. For every request b of a batch, a drafter has proposed
 * up to K tokens x_0..x_{K-1}; the target model has scored the whole block
 * in one pass, giving K+1 logit rows (one per drafted position plus the
 * position after the block). Of the K drafted tokens only the first k_b (the
 * request's verify budget) are checked. The library decides which drafted
 * tokens survive and draws the one token that follows them:
 *
 *   - Greedy verification (temperature == 0), as described in
 *     "Speculative decoding becomes standard: DSpark and multi-token
 *     drafters", section "Why draft-and-verify does not change the output",
 *     paragraph 1: keep drafted tokens while they equal the target's most
 *     likely token (lowest index among equal maxima), and at the first
 *     mismatch emit the target's own token; if all k_b agree, emit the
 *     target's token at position k_b.
 *   - Sampled verification (temperature T > 0), same section, paragraph 2
 *     (the rule of Leviathan, Kalman and Matias): with p_i = softmax(z_t/T)
 *     and q_i = softmax(z_d/T) over the full vocabulary, drafted token x_i
 *     survives when u < min(1, p_i(x_i)/q_i(x_i)); at the first rejection j
 *     the token is drawn from the renormalised residual max(0, p_j - q_j);
 *     if all k_b survive, a bonus token is drawn from p_{k_b}. Draws are
 *     inverse-CDF in vocabulary order.
 *   - Per-request budgets k_b (0 <= k_b <= K) model the confidence-driven
 *     scheduler of the same page, section "What DSpark adds", paragraph 2.
 *
 * Random numbers: Philox4x32-10 (Salmon et al., SC'11) with key = seed
 * (low word, high word) and counter = (b, i, 0, 0) for position i of request
 * b; output word 0 gives the acceptance uniform of position i, word 1 its
 * sampling uniform, each as (word >> 8) * 2^-24.
 *
 * Conventions shared by every entry point:
 *   - All tensors are caller-owned device memory; the library never frees
 *     or retains them past a call. The library owns only the context and its
 *     device workspace.
 *   - Work is enqueued on the caller's HIP stream (hipStream_t passed as
 *     void*, NULL = default stream) and the call returns without waiting.
 *   - Return values are sv_status codes; nothing is thrown across the ABI.
 *     Argument errors are detected on the host before anything is enqueued.
 *     Errors only visible on the device (a budget outside [0, K], a drafted
 *     token outside [0, V)) set bits of a device status word read by
 *     spec_verify_status; the kernels never read out of bounds because of
 *     them.
 *   - One context serves one stream at a time: calls that overlap in time
 *     on the same context race on its workspace.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct spec_verify_ctx spec_verify_ctx;

/* Storage type of the logit tensors. */
enum sv_dtype {
    SV_DTYPE_F32 = 0,   /* IEEE fp32 */
    SV_DTYPE_BF16 = 1   /* bfloat16: the upper 16 bits of an fp32 */
};

/* Return codes. */
enum sv_status {
    SV_OK = 0,
    SV_ERR_NULL = -1,    /* a required pointer is NULL */
    SV_ERR_ARG = -2,     /* a scalar argument is out of range */
    SV_ERR_DTYPE = -3,   /* unknown storage type */
    SV_ERR_ALIGN = -4,   /* a pointer is not aligned to its element size */
    SV_ERR_HIP = -5,     /* the HIP runtime reported an error */
    SV_ERR_NOMEM = -6,   /* device workspace allocation failed */
    SV_ERR_STATE = -7,   /* NULL or already freed context */
    SV_ERR_TOO_BIG = -8  /* spec_verify_run_noalloc: the call needs more
                            workspace than its static scratch holds */
};

/* Bits of the device status word (spec_verify_status). */
#define SV_FLAG_BAD_BUDGET 0x1u /* a budget was outside [0, K]; it was clamped */
#define SV_FLAG_BAD_TOKEN  0x2u /* a checked drafted token was outside [0, V);
                                   it was treated as rejected, its p and q as 0 */
#define SV_FLAG_SYNC_TIMEOUT 0x4u /* an internal consistency check failed (a
                                   wave's bounded wait for another wave of its
                                   own workgroup expired, or a decision was
                                   read before it was final); the outputs of
                                   that call are not valid. No wait depends on
                                   other workgroups being resident. */

#define SV_FLAG_BAD_LENGTH 0x8u /* a request's tokens do not fit its page table
                                   row (or an output); it was skipped */
#define SV_FLAG_BAD_PAGE 0x10u  /* a page number that a call needed was outside
                                   the pool; its tokens were skipped */
#define SV_FLAG_NO_PAGES 0x20u  /* too few free pages: some request got none */
#define SV_FLAG_BAD_PARENT 0x40u /* a parent outside the batch, or one that has a
                                   parent itself; treated as none */
#define SV_FLAG_NO_PREFIX 0x80u /* a page of a prefix was not in the parent's row;
                                   a new one, which holds nothing of it, took its
                                   place */

/* Library limits. */
#define SV_MAX_BATCH 16384
#define SV_MAX_K 32
#define SV_MAX_VOCAB (1 << 20)
#define SV_MAX_HEADS 256
#define SV_MAX_PAGE 4096
#define SV_MAX_CONTEXT (1 << 24)
#define SV_MAX_HIDDEN 65536
#define SV_MAX_STRIDE 2147483647
#define SV_MAX_GROUPS 512

/* Size of the static device scratch of spec_verify_run_noalloc (per GPU). */
#define SV_NOALLOC_SCRATCH_BYTES (16u << 20)

/*
 * spec_verify_init -- create a context for one device and one problem shape
 * (the batched verify step of "Speculative decoding becomes standard: DSpark
 * and multi-token drafters", section "Why draft-and-verify does not change
 * the output", with the per-request budgets of section "What DSpark adds",
 * paragraph 2).
 *   out        receives the context (set to NULL on failure).
 *   device     HIP device ordinal.
 *   max_batch  largest B a run will pass, 1..SV_MAX_BATCH.
 *   max_k      largest K a run will pass, 0..SV_MAX_K.
 *   vocab      V, the vocabulary size of every run, 1..SV_MAX_VOCAB.
 *   dtype      sv_dtype of the logits of every run.
 * Allocates and zeroes the device workspace (per-chunk partial statistics,
 * per-row argmax keys and per-request counters of greedy mode, status
 * word). The context owns it until spec_verify_free. Synchronous.
 * Errors: SV_ERR_NULL, SV_ERR_ARG, SV_ERR_DTYPE, SV_ERR_HIP, SV_ERR_NOMEM.
 */
int spec_verify_init(spec_verify_ctx** out, int device, int max_batch, int max_k,
                     int vocab, int dtype);

/*
 * spec_verify_run -- verify one batch (stream-ordered, no host sync): the
 * greedy rule ("Speculative decoding becomes standard: DSpark and
 * multi-token drafters", section "Why draft-and-verify does not change the
 * output", paragraph 1) when temperature == 0, else the rejection rule with
 * residual and bonus draws (same section, paragraph 2), over the budgeted
 * positions of each request (section "What DSpark adds", paragraph 2).
 *   target_logits     [B, K+1, V] row-major, storage ctx dtype (device).
 *   draft_logits      [B, K, V] row-major, same storage (device); may be
 *                     NULL when temperature == 0 (never read then).
 *   draft_tokens      int32 [B, K] drafted token ids (device); entries at
 *                     positions >= budgets[b] are never read.
 *   budgets           int32 [B] verify budgets k_b, 0 <= k_b <= K (device).
 *   B, K              batch size (0..max_batch; 0 is a no-op) and block
 *                     width (0..max_k).
 *   temperature       0 = greedy; > 0 = sampled; must be finite. Sampled
 *                     rows are reduced with c = log2(e) / T in fp32 and the
 *                     scaled maximum max(z) c, so |z| c must stay inside the
 *                     fp32 range (for logits below 1e4 in magnitude: T >= 1e-30).
 *   seed              Philox key of this call.
 *   out_tokens        int32 [B, K+1]: x_0..x_{j-1}, then the drawn token,
 *                     then -1 padding (device).
 *   out_num_accepted  int32 [B]: j, the number of drafted tokens kept.
 *   out_p_draft       float [B, K] or NULL: p_i(x_i) for i < k_b, NaN for
 *                     i >= k_b and in greedy mode (device).
 *   out_q_draft       float [B, K] or NULL: q_i(x_i), same layout.
 *   stream            hipStream_t or NULL.
 * The caller keeps ownership of every tensor. Request b uses Philox counter
 * (b, i, 0, 0); spec_verify_run_ex offsets b.
 * Pointers must be aligned to their element size; a 16-byte aligned logit
 * base with V * sizeof(element) a multiple of 16 takes the vector-load path
 * for every row. Rows b*(K+1)+i beyond i = k_b are never read.
 * Errors (host-detected, nothing enqueued): SV_ERR_STATE, SV_ERR_NULL,
 * SV_ERR_ARG, SV_ERR_ALIGN; SV_ERR_HIP if the launch fails.
 */
int spec_verify_run(spec_verify_ctx* ctx, const void* target_logits,
                    const void* draft_logits, const int32_t* draft_tokens,
                    const int32_t* budgets, int B, int K, float temperature,
                    uint64_t seed, int32_t* out_tokens, int32_t* out_num_accepted,
                    float* out_p_draft, float* out_q_draft, void* stream);

/*
 * spec_verify_run_ex -- spec_verify_run on a slice of a larger batch: row b
 * of the tensors is request request_base + b of the whole batch, and its
 * Philox counters are (request_base + b, i, 0, 0). Requests are independent,
 * so calls over disjoint slices with their own bases give the outputs of one
 * call over the whole batch, bit for bit (how the batch would be split across
 * GPUs, each taking a contiguous range of requests). Arguments as in
 * spec_verify_run; 0 <= request_base <= 2^32 - 1 - B, else SV_ERR_ARG.
 */
int spec_verify_run_ex(spec_verify_ctx* ctx, const void* target_logits,
                       const void* draft_logits, const int32_t* draft_tokens,
                       const int32_t* budgets, int B, int K, float temperature,
                       uint64_t seed, int64_t request_base, int32_t* out_tokens,
                       int32_t* out_num_accepted, float* out_p_draft,
                       float* out_q_draft, void* stream);

/*
 * spec_verify_run_noalloc -- spec_verify_run_ex without a context, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation). It calls no
 * hipMalloc or hipFree: its workspace is a static device array of
 * SV_NOALLOC_SCRATCH_BYTES that every GPU the library runs on holds until the
 * process ends. It runs on the current HIP device; vocab and dtype are given
 * per call. Every call on one GPU shares that GPU's array: calls that overlap
 * in time on one GPU (on different streams, or from different threads) race
 * and their outputs are undefined; calls in stream order are safe (each call
 * clears the counters it needs with a fill kernel, no memset).
 *   vocab, dtype  as in spec_verify_init.
 *   out_status    uint32 [1] (device) or NULL: this call's SV_FLAG_BAD_BUDGET
 *                 and SV_FLAG_BAD_TOKEN bits (written, not accumulated).
 *   other arguments as in spec_verify_run_ex.
 * Three launches: the fill kernel, the streaming pass and, in sampled mode,
 * the draw pass.
 * Errors (nothing enqueued): SV_ERR_NULL, SV_ERR_ARG, SV_ERR_DTYPE,
 * SV_ERR_ALIGN; SV_ERR_TOO_BIG when the call's workspace (it grows with
 * min(B, 8192) * (K + 1) and the vocabulary's chunk count) exceeds the
 * static array, e.g. B = 512, K = 8, V = 151936 in bf16 or fp32 fits;
 * SV_ERR_HIP if a launch fails.
 */
int spec_verify_run_noalloc(int vocab, int dtype, const void* target_logits,
                            const void* draft_logits, const int32_t* draft_tokens,
                            const int32_t* budgets, int B, int K, float temperature,
                            uint64_t seed, int64_t request_base, int32_t* out_tokens,
                            int32_t* out_num_accepted, float* out_p_draft,
                            float* out_q_draft, uint32_t* out_status, void* stream);

/*
 * spec_verify_check_args -- the host-side argument check of spec_verify_run
 * for a context created with (max_batch, max_k, vocab, dtype), without a
 * context or a device. Pointers are only tested for NULL and alignment,
 * never dereferenced. Returns SV_OK or the code spec_verify_run would return.
 */
int spec_verify_check_args(int max_batch, int max_k, int vocab, int dtype,
                           const void* target_logits, const void* draft_logits,
                           const void* draft_tokens, const void* budgets, int B,
                           int K, float temperature, const void* out_tokens,
                           const void* out_num_accepted, const void* out_p_draft,
                           const void* out_q_draft);

/*
 * spec_verify_status -- wait for the device, return and clear the status
 * word (SV_FLAG_* bits accumulated by runs since the last call).
 * Errors: SV_ERR_STATE, SV_ERR_NULL, SV_ERR_HIP.
 */
int spec_verify_status(spec_verify_ctx* ctx, uint32_t* flags);

/*
 * spec_verify_philox_words -- write the Philox4x32-10 blocks the verifier
 * uses: out_words[(b*P + i)*4 + w] = word w of the block with key = seed and
 * counter = (b, i, 0, 0), for b < B, i < P (device buffer of 4*B*P uint32).
 * Stream-ordered. For checking the device generator against other
 * implementations. Errors: SV_ERR_NULL, SV_ERR_ARG, SV_ERR_HIP.
 */
int spec_verify_philox_words(uint64_t seed, int B, int P, uint32_t* out_words,
                             void* stream);

/*
 * spec_verify_timing -- per-pass device timing of later runs (off by
 * default). enable != 0: every later spec_verify_run on this context records
 * a HIP event pair on its stream around each pass it launches -- pass 0 the
 * streaming pass (row statistics; the greedy decisions and outputs), pass 1
 * the draw pass of sampled mode (accept decisions, first rejection,
 * residual or bonus draw, outputs) -- up to
 * 65536 passes, then recording stops. enable == 0 waits for and discards
 * what is recorded. The events are the context's; recording adds event
 * markers between the launches and nothing else.
 * Errors: SV_ERR_STATE, SV_ERR_HIP.
 */
int spec_verify_timing(spec_verify_ctx* ctx, int enable);

/*
 * spec_verify_timing_read -- wait for the recorded passes, write per pass p
 * (0 streaming, 1 draw) the number of launches counts[p] and the sum of their
 * durations total_ms[p] in milliseconds (host arrays of 2), and clear the
 * record (timing stays as set).
 * Errors: SV_ERR_STATE, SV_ERR_NULL, SV_ERR_HIP.
 */
int spec_verify_timing_read(spec_verify_ctx* ctx, int* counts, double* total_ms);

/*
 * spec_budget_schedule -- per-request verify budgets from per-position
 * confidences ("Speculative decoding becomes standard: DSpark and
 * multi-token drafters", section "What DSpark adds", paragraph 2: each
 * drafted position has a confidence, read as its chance of acceptance once
 * every earlier position of the block was accepted, and verify windows are
 * sized jointly over the batch, shrinking as load grows; the Analytics
 * Vidhya DSpark page, section "Gotchas and Issues": the cut is set afresh
 * for every batch, and a position is verified only if it is expected to
 * pay off). Stream-ordered, no host sync, no context and no workspace.
 *   confidences  float [B, K] row-major (device): c[b, i] for drafted
 *                position i of request b. NaN and negatives read as 0,
 *                values above 1 as 1.
 *   B, K         requests (0..SV_MAX_BATCH; 0 is a no-op) and drafted
 *                positions per request (0..SV_MAX_K).
 *   n_total      the batch's verify budget N >= 0: drafted positions to
 *                verify over all requests (the load sets it).
 *   tau          >= 0, finite: a position is verified only if its gain
 *                exceeds tau.
 *   out_budgets  int32 [B] (device): k_b, ready for spec_verify_run.
 * The gain of position k of request b is g = c[b,0] * c[b,1] * ... * c[b,k]
 * (the expected accepted tokens it adds), multiplied left to right in fp32.
 * The N largest gains above tau are verified, equal gains by position, then
 * request; k_b counts those of request b, always a prefix of its block.
 * sum_b k_b = min(N, number of gains above tau).
 * Errors (nothing enqueued): SV_ERR_ARG, SV_ERR_NULL, SV_ERR_ALIGN (pointers
 * not 4-byte aligned); SV_ERR_HIP if the launch fails.
 */
int spec_budget_schedule(const float* confidences, int B, int K, int n_total, float tau,
                         int32_t* out_budgets, void* stream);

/*
 * spec_head_stats -- row statistics of the shared output head, computed on
 * the matrix cores without writing the logits ("Speculative decoding becomes
 * standard: DSpark and multi-token drafters", section "What DSpark adds",
 * paragraph 1: the drafter reuses the target's output projection unchanged;
 * section "Why draft-and-verify does not change the output", paragraphs 1
 * and 2: a verify step needs each scored row's most likely token, or p(x)
 * and q(x) of the drafted token). Stream-ordered, no host sync.
 *   hidden      bf16 [R, H] row-major (device, 16-byte aligned): hidden
 *               states, one row per scored position (target or drafter).
 *   weight      bf16 [V, H] row-major (device, 16-byte aligned): the head.
 *   R, H, V     rows (>= 0; 0 is a no-op), hidden size (>= 8, a multiple of
 *               8) and vocabulary (1..SV_MAX_VOCAB).
 *   tokens      int32 [R] or NULL: the token whose logit out_ztok reports.
 *   temperature > 0: sampled statistics; 0: greedy (max and argmax only).
 *   out_max     float [R]: m = max_v z[r, v], z = hidden weight^T (fp32
 *               accumulation of exact bf16 products).
 *   out_sumexp  float [R] or NULL: sum_v 2^((z[r, v] - m) log2(e) / T)
 *               (sampled; NaN in greedy mode). p(x) = 2^((z_x - m) log2(e)/T)
 *               / sum.
 *   out_ztok    float [R] or NULL: z[r, tokens[r]], NaN if out of range.
 *   out_argmax  int32 [R] or NULL: the first argmax (greedy; -1 when sampled).
 *   workspace   device scratch of at least spec_head_workspace_bytes(R, V)
 *               bytes (16-byte aligned), caller-owned; calls that share it
 *               must not overlap.
 * Errors (nothing enqueued): SV_ERR_ARG, SV_ERR_NULL, SV_ERR_ALIGN;
 * SV_ERR_HIP if a launch fails.
 */
int spec_head_stats(const void* hidden, const void* weight, int R, int H, int V,
                    const int32_t* tokens, float temperature, float* out_max,
                    float* out_sumexp, float* out_ztok, int32_t* out_argmax,
                    void* workspace, size_t workspace_bytes, void* stream);

/* spec_head_workspace_bytes -- scratch spec_head_stats needs for (R, V):
 * one 16-byte partial per row and vocabulary split (for 1,536 rows or more
 * and V of at least 10,240: 40 per row plus at most ceil(V / 256) / 16 + 4).
 * 0 on bad arguments. Host only. */
size_t spec_head_workspace_bytes(int R, int V);

/*
 * spec_verify_hidden -- one verify step from hidden states through the shared
 * output head: the outputs of spec_verify_run on the logits z = h W^T,
 * without writing the logits of the scored rows anywhere ("Speculative
 * decoding becomes standard: DSpark and multi-token drafters", section "What
 * DSpark adds", paragraph 1: the drafter reuses the target's output
 * projection unchanged; section "Why draft-and-verify does not change the output",
 * paragraphs 1 and 2: the greedy and sampled rules; section "What DSpark
 * adds", paragraph 2: per-request budgets). Logits are fp32 accumulations of
 * exact bf16 products; p and q, the accept test, the Philox counters and the
 * inverse-CDF draw are those of spec_verify_run. Stream-ordered, no host
 * sync; five launches (plan, head statistics, decide, and in sampled mode
 * the head product over each request's draw rows and the draw). With at
 * least 512 requests (when the head's many-row product takes the draw rows)
 * that product leaves per-block draw masses instead of logits, so no logit
 * reaches memory; with fewer it writes the draw rows' fp32 logits to the
 * workspace.
 *   target_hidden  bf16 [B, K+1, H] row-major (device, 16-byte aligned).
 *   draft_hidden   bf16 [B, K, H] (device, 16-byte aligned); may be NULL
 *                  when temperature == 0 or K == 0.
 *   head           bf16 [V, H] row-major (device, 16-byte aligned).
 *   draft_tokens   int32 [B, K] (device); may be NULL when K == 0.
 *   budgets        int32 [B] (device), 0 <= k_b <= K.
 *   B, K, H, V     requests (0..SV_MAX_BATCH; 0 is a no-op), drafted
 *                  positions (0..SV_MAX_K), hidden size (>= 8, a multiple
 *                  of 8), vocabulary (1..SV_MAX_VOCAB).
 *   temperature    > 0 sampled, 0 greedy (drafter states and seed unused).
 *   seed           Philox key; counter (b, i, 0, 0) as in spec_verify_run.
 *   out_tokens     int32 [B, K+1]: x_0..x_{j-1}, y, then -1.
 *   out_num_accepted int32 [B]: j_b.
 *   out_p_draft, out_q_draft  float [B, K] or NULL: p_i(x_i), q_i(x_i) for
 *                  i < k_b, NaN elsewhere and in greedy mode.
 *   out_status     int32 [1] (device) or NULL: this call's SV_FLAG_BAD_BUDGET
 *                  and SV_FLAG_BAD_TOKEN bits (written, not accumulated). A
 *                  flagged request's outputs are undefined.
 *   workspace      device scratch of at least
 *                  spec_verify_hidden_workspace_bytes(B, K, V) bytes,
 *                  256-byte aligned, caller-owned; calls sharing it must not
 *                  overlap. Most of it is the fp32 logits of two rows per
 *                  request (8 B V bytes).
 * Errors (nothing enqueued): SV_ERR_ARG, SV_ERR_NULL, SV_ERR_ALIGN;
 * SV_ERR_HIP if a launch fails.
 */
int spec_verify_hidden(const void* target_hidden, const void* draft_hidden, const void* head,
                       const int32_t* draft_tokens, const int32_t* budgets, int B, int K, int H,
                       int V, float temperature, uint64_t seed, int32_t* out_tokens,
                       int32_t* out_num_accepted, float* out_p_draft, float* out_q_draft,
                       int32_t* out_status, void* workspace, size_t workspace_bytes,
                       void* stream);

/* spec_verify_hidden_workspace_bytes -- scratch spec_verify_hidden needs for
 * (B, K, V); 0 on bad arguments. Host only. */
size_t spec_verify_hidden_workspace_bytes(int B, int K, int V);

/*
 * spec_markov_draft -- the drafter's low-rank Markov head over a block of K
 * drafted positions ("Speculative decoding becomes standard: DSpark and
 * multi-token drafters", section "What DSpark adds", paragraph 1: the block
 * comes from a parallel backbone and a factorised rank-256 Markov model over
 * consecutive positions corrects it; "DSpark" (finds page): the deployed
 * sequential structure conditions only on the preceding token, through a
 * low-rank matrix). For i = 0..K-1 in
 * order: z_i = base_i + A[x_{i-1}] Bm^T, the bias an fp32 sum of exact bf16
 * products, the sum formed in fp32 and rounded once to bf16 (to nearest,
 * ties to even) and stored; x_i = the first (lowest index) argmax of the
 * stored row; x_{-1} = prev_tokens. The stored rows are drafter logits a
 * verify step can read. Stream-ordered, no host sync; K + 2 launches when r
 * is a multiple of 16 up to 256 and V a multiple of 8, else 1 + 2K.
 *   base_logits  bf16 [B, K, V] row-major (device, 16-byte aligned): the
 *                backbone's logits.
 *   markov_a     bf16 [V, r] (device, 16-byte aligned): the previous token's
 *                factor.
 *   markov_b     bf16 [V, r] (device, 16-byte aligned): the vocabulary factor.
 *   prev_tokens  int32 [B] (device): the last token of each sequence.
 *   B, K, r, V   requests (0..SV_MAX_BATCH; 0 is a no-op), positions
 *                (0..SV_MAX_K; 0 is a no-op), rank (>= 8, a multiple of 8),
 *                vocabulary (1..SV_MAX_VOCAB).
 *   out_logits   bf16 [B, K, V] (device, 16-byte aligned, not base_logits).
 *   out_tokens   int32 [B, K] (device): the drafted tokens.
 *   out_status   int32 [1] (device) or NULL: SV_FLAG_BAD_TOKEN if a previous
 *                token is outside [0, V) (written, not accumulated); that
 *                request's outputs are undefined.
 *   workspace    device scratch of at least
 *                spec_markov_draft_workspace_bytes(B, V) bytes, 256-byte
 *                aligned, caller-owned; calls sharing it must not overlap.
 *                It holds two token maps of B entries, three arrays of one
 *                8-byte first-argmax key per request (positions in turn),
 *                and one 8-byte first-argmax entry per request and
 *                vocabulary split for the product of other shapes; the bias
 *                rows never reach memory, and of the stored rows only each
 *                request's best 32 columns per position are read back.
 * Errors (nothing enqueued): SV_ERR_ARG, SV_ERR_NULL, SV_ERR_ALIGN;
 * SV_ERR_HIP if a launch fails.
 */
int spec_markov_draft(const void* base_logits, const void* markov_a, const void* markov_b,
                      const int32_t* prev_tokens, int B, int K, int r, int V, void* out_logits,
                      int32_t* out_tokens, int32_t* out_status, void* workspace,
                      size_t workspace_bytes, void* stream);

/* spec_markov_draft_workspace_bytes -- scratch spec_markov_draft needs for
 * (B, V); 0 on bad arguments. Host only. */
size_t spec_markov_draft_workspace_bytes(int B, int V);

/*
 * The paged 4-bit key/value cache of the target model.
 *
 * A verify step scores a block in one pass of the target ("Speculative
 * decoding becomes standard: DSpark and multi-token drafters", section "Why
 * draft-and-verify does not change the output"): per layer, the k_b + 1 new
 * tokens' keys and values enter the cache and every row of the block attends
 * over it. The cache is one caller-owned buffer of
 * spec_verify_cache_bytes() bytes (device, 16-byte aligned):
 *   uint8 [num_pages][kv_heads][page_size / 32][34 * head_dim],
 * tiles of 32 consecutive tokens of one head. Keys and values are e2m1 codes
 * (a sign bit, then 0, 0.5, 1, 1.5, 2, 3, 4, 6), one scale byte per token,
 * head and 32 channels: 2^(byte - 127), 255 = not a number. The scale is the
 * smallest power of two, at least 2^-64, under which the group's largest
 * magnitude is at most 6 (at most 2^125: larger magnitudes saturate); codes
 * are rounded to nearest, ties to even. A group that holds a NaN or an
 * infinity reads as NaN. Tokens never share a scale, so rejected drafted
 * tokens are undone by the lengths alone.
 * Inside a tile, for token tok (0..31) with half = tok / 16, low = tok % 16,
 * quad = low / 4, and D = head_dim, U = min(16, D / 8), C = min(4, D / 32):
 *   key bytes    y = 0 .. D/2 - 1  at half 8 D + (y / U) 16 U + low U + y % U
 *   value bytes  y = 0 .. D/2 - 1, piece = y / C, at 16 D +
 *       (((piece / 16) 2 + half) 4 + quad) 64 C + (piece % 16) 4 C +
 *       (low % 4) C + y % C
 *   key scale of group g = channel / 32    at 32 D + 32 g + 2 low + half
 *   value scale of group g                 at 33 D + 32 g + 8 quad + 4 half + low % 4
 * Byte y holds channel 2 y in its low half and 2 y + 1 in its high half.
 * Shared arguments:
 *   kv_heads, head_dim   1..SV_MAX_HEADS; 64, 128 or 256.
 *   page_size    tokens of a page: a power of two, 32..SV_MAX_PAGE.
 *   page_table   int32 [B, max_pages] (device): the page of positions
 *                [i page_size, (i + 1) page_size) of request b. Entries that a
 *                call does not need are never read as pages; a needed entry
 *                outside [0, num_pages) sets SV_FLAG_BAD_PAGE and is never
 *                accessed: writes and reads skip its tokens, the attention's
 *                outputs of that request are undefined. max_pages *
 *                page_size is at most SV_MAX_CONTEXT.
 *   ctx_lens     int32 [B] (device): tokens of request b in the cache before
 *                this block; negative marks an empty slot, which is skipped
 *                (nothing read, nothing written).
 *   budgets      int32 [B] (device) or NULL: the block has budgets[b] + 1
 *                tokens, at positions ctx_lens[b] onwards (clamped into the
 *                block's width, with SV_FLAG_BAD_BUDGET); NULL: all of them.
 *   out_status   int32 [1] (device) or NULL: SV_FLAG_* bits are OR-ed into it
 *                (the caller clears it; one word can collect a whole step).
 *                Outputs of a flagged request are undefined, apart from what
 *                is said to be skipped.
 * A block that does not fit its page table row sets SV_FLAG_BAD_LENGTH and is
 * skipped. Requests may share pages that are only read; what two tokens written
 * to the same place at once leave there is undefined.
 */

/* spec_verify_cache_bytes -- bytes of a cache of num_pages pages; 0 on bad
 * arguments. Host only. */
size_t spec_verify_cache_bytes(int num_pages, int kv_heads, int head_dim, int page_size);

/*
 * spec_verify_cache_write -- quantise the keys and values of every request's
 * block (or prompt) into the cache. Stream-ordered, one launch.
 *   keys, values   [B, T, kv_heads, head_dim] of type dtype (device, 16-byte
 *                  aligned): token t of request b starts at element (b T + t)
 *                  stride, its heads contiguous. Tokens at t > budgets[b] are
 *                  never read.
 *   key_stride, value_stride  elements between tokens: at least kv_heads *
 *                  head_dim, a multiple of 16 bytes (a slice of a fused
 *                  projection's rows is taken as it is).
 *   B, T           requests (0..SV_MAX_BATCH; 0 is a no-op), tokens per
 *                  request (0..SV_MAX_CONTEXT; 0 is a no-op); T * kv_heads *
 *                  head_dim at most 2^33.
 * Other bytes of the cache keep their values.
 * Errors (nothing enqueued): SV_ERR_ARG, SV_ERR_DTYPE, SV_ERR_NULL,
 * SV_ERR_ALIGN; SV_ERR_HIP if the launch fails.
 */
int spec_verify_cache_write(const void* keys, const void* values, int dtype, int64_t key_stride,
                            int64_t value_stride, const int32_t* page_table,
                            const int32_t* ctx_lens, const int32_t* budgets, int B, int T,
                            int kv_heads, int head_dim, int page_size, int max_pages,
                            int num_pages, void* cache, int32_t* out_status, void* stream);

/*
 * spec_verify_pages_plan -- one step of the page tables: from the requests'
 * lengths, which pages every request holds, and where its new tokens go. The
 * caller keeps two arrays, which the call changes: the page table, and for every
 * page of the pool the number of table entries that hold it (0: free).
 * Page i of request b is needed if it holds a position of [0, ctx_lens[b] +
 * budgets[b] + 1) that, with window > 0, is below `sinks` or at or behind
 * ctx_lens[b] - window + 1 (what spec_verify_attention_sinks reads in this and
 * later steps). Pages held and not needed are given back: an empty slot (a
 * negative length) gives back all, and a slot is emptied by one call before
 * another request takes it. Needed pages not held come from the parent's row, or
 * are the lowest-numbered free ones, dealt out in the order of requests and of
 * positions in each. A request whose new pages, with those of all requests
 * before it, are more than there are free gets none of them
 * (SV_FLAG_NO_PAGES). A function of the arguments alone. Stream-ordered, no
 * host sync.
 *   page_table   int32 [B, max_pages] (device), changed: entries in [0,
 *                num_pages) are held; others are none and become -1 (those
 *                >= num_pages with SV_FLAG_BAD_PAGE). At first: all -1.
 *   page_refs    int32 [num_pages] (device), changed. At first: all 0. 0 or
 *                less is free. num_pages * page_size is at most 2^31 - 1.
 *   parents, prefix_lens  int32 [B] (device) or NULL: request b takes the
 *                pages of its parent's first prefix_lens[b] tokens (a length
 *                of 0 or less: none) where it holds none itself, as the
 *                parent's row was before the call; only whole pages, and only
 *                in front of ctx_lens[b], so that its own slots lie in pages of
 *                its own. Tokens behind the last whole page are the request's
 *                to write: one that starts behind a prefix starts at a multiple
 *                of page_size (a prompt matched in full runs its last page
 *                again). Negative: no parent. A parent has none itself
 *                (SV_FLAG_BAD_PARENT) and has written the prefix before: its
 *                own length is not below prefix_lens[b], and lengths do not go
 *                back into shared pages. Where its row lacks a page that would
 *                have been taken (it was given back behind a window, refused,
 *                or the parent never held it), the request gets a new page and
 *                SV_FLAG_NO_PREFIX: it runs, but what that page holds in front
 *                of ctx_lens[b] is for the caller to write before any attention
 *                reads it.
 *   T            the block's width, 1..SV_MAX_CONTEXT; B 0..SV_MAX_BATCH.
 *   out_starts   int32 [B] (device): ctx_lens[b] where the request's pages are
 *                all there, else -1 (an empty slot, no pages, or a block that
 *                does not fit its row, which then stays as it is, with
 *                SV_FLAG_BAD_LENGTH). Serves as ctx_lens of the other calls.
 *   out_slots    int32 [B, T] (device): page * page_size + position in the
 *                page of token t, or -1 for t > budgets[b] and where
 *                out_starts is -1.
 *   out_positions  int32 [B, T] (device): out_starts[b] + t, or -1 likewise.
 *   workspace    device scratch of at least
 *                spec_verify_pages_plan_workspace_bytes() bytes (256-byte
 *                aligned), caller-owned, its contents of no account; calls
 *                that share it must not overlap.
 * Errors (nothing enqueued): SV_ERR_ARG, SV_ERR_NULL, SV_ERR_ALIGN;
 * SV_ERR_HIP if a launch fails.
 */
int spec_verify_pages_plan(int32_t* page_table, int32_t* page_refs, const int32_t* ctx_lens,
                           const int32_t* budgets, const int32_t* parents,
                           const int32_t* prefix_lens, int B, int T, int page_size, int max_pages,
                           int num_pages, int window, int sinks, int32_t* out_starts,
                           int32_t* out_slots, int32_t* out_positions, int32_t* out_status,
                           void* workspace, size_t workspace_bytes, void* stream);

/* spec_verify_pages_plan_workspace_bytes -- scratch spec_verify_pages_plan
 * needs; 0 on bad arguments. Host only. */
size_t spec_verify_pages_plan_workspace_bytes(int B, int max_pages, int num_pages);

/*
 * spec_verify_cache_write_rotated -- a step's projections on their way into the
 * attention: queries and keys normalised per head and rotated to their
 * positions, queries stored, keys and values quantised into the cache. Token n
 * goes to slots[n]; a negative slot skips it (nothing read, nothing written).
 * Per query or key head of D channels:
 *   y = x / sqrt(mean(x^2) + eps) * w   (y = x where the weights are NULL)
 * and its first `rot` channels are turned in pairs by a = positions[n] *
 * inv_freq[i]: (y_i, y_j) -> factor (y_i cos a - y_j sin a, y_j cos a + y_i
 * sin a), with j = i + rot / 2, or, interleaved, channels 2 i and 2 i + 1.
 * Sums and products are fp32; angles, sine and cosine are formed in fp64 (right
 * to 2^-29 of a turn for |position| <= 2^24 and frequencies up to 1) and rounded
 * to fp32; magnitudes whose squares' sum leaves fp32's range are not normalised
 * rightly. Queries
 * are rounded to bf16 once; keys are rounded to bf16 and then quantised, so
 * that the cache's bytes are those of spec_verify_cache_write on out_keys.
 * Stream-ordered, one launch.
 *   queries, keys, values  of type dtype: [tokens, q_heads (kv_heads),
 *                head_dim] (device, 16-byte aligned), the heads contiguous,
 *                `*_stride` elements between tokens (a multiple of 16 bytes; a
 *                slice of a fused projection's rows is taken as it is).
 *   slots, positions  int32 [tokens] (device), as spec_verify_pages_plan gives
 *                them. A slot outside the pool is skipped with SV_FLAG_BAD_PAGE.
 *   tokens       0 (a no-op) .. 2^31 - 1.
 *   inv_freq     float [rot / 2] (device; NULL if rot is 0).
 *   rot          0..head_dim, a multiple of 16.
 *   factor       finite; usually 1.
 *   q_norm, k_norm  [head_dim] of type norm_dtype (device, 16-byte aligned) or
 *                NULL; eps finite, at least 0.
 *   out_queries  bf16 [tokens, q_heads, head_dim]; out_keys bf16 [tokens,
 *                kv_heads, head_dim] or NULL (device, 16-byte aligned). Rows of
 *                skipped tokens keep their values. They may not overlap any
 *                other argument.
 * kv_heads, head_dim, page_size, num_pages, cache, out_status as above;
 * num_pages * page_size is at most 2^31 - 1.
 * Errors (nothing enqueued): SV_ERR_ARG, SV_ERR_DTYPE, SV_ERR_NULL,
 * SV_ERR_ALIGN; SV_ERR_HIP if the launch fails.
 */
int spec_verify_cache_write_rotated(const void* queries, const void* keys, const void* values,
                                    int dtype, int64_t query_stride, int64_t key_stride,
                                    int64_t value_stride, const int32_t* slots,
                                    const int32_t* positions, int64_t tokens,
                                    const float* inv_freq, int rot, int interleaved, float factor,
                                    const void* q_norm, const void* k_norm, int norm_dtype,
                                    float eps, int q_heads, int kv_heads, int head_dim,
                                    int page_size, int num_pages, void* cache, void* out_queries,
                                    void* out_keys, int32_t* out_status, void* stream);

/*
 * spec_verify_cache_read -- read tokens back as the values their codes stand
 * for (exact in both types). Stream-ordered, one launch.
 *   starts       int32 [B] (device) or NULL (all 0): first position; negative
 *                marks an empty slot.
 *   lens         int32 [B] (device): tokens to read, at most T (more, or past
 *                the page table row: SV_FLAG_BAD_LENGTH, request skipped);
 *                0 or less: none.
 *   B, T, dtype  as above; out_keys, out_values [B, T, kv_heads, head_dim] of
 *                type dtype (device, 16-byte aligned). Tokens at t >= lens[b]
 *                keep their values.
 * Errors as spec_verify_cache_write.
 */
int spec_verify_cache_read(const void* cache, const int32_t* page_table, const int32_t* starts,
                           const int32_t* lens, int B, int T, int kv_heads, int head_dim,
                           int page_size, int max_pages, int num_pages, int dtype, void* out_keys,
                           void* out_values, int32_t* out_status, void* stream);

/*
 * spec_verify_attention -- attention of every row of the drafted blocks over
 * the cache, which already holds the blocks' own tokens
 * (spec_verify_cache_write on the same stream). Row t of request b, t <=
 * budgets[b], stands at position p = ctx_lens[b] + t and sees the positions
 * [max(0, p - window + 1), p] (window 0: [0, p]); query head i reads kv head
 * i / (q_heads / kv_heads):
 *   out = sum_j softmax_j(scale q . k_j) v_j.
 * Products accumulate in fp32, the softmax's statistics are fp32. The weights,
 * up to 2^8 under a reference that lags behind the maximum, are rounded to bf16
 * for the product with the values, not for their sum (so equal values come back
 * within that rounding); weighted sums past fp32's range give infinities or NaN.
 * A NaN group of a key or value reaches exactly the rows that see its token.
 * K = 0 is the single-token form. Stream-ordered, no host sync, one launch, or
 * two when the contexts may be split over workgroups (a choice by the shapes alone; how they
 * are split is decided on the device by all requests' lengths and budgets, so
 * the order of a request's sums may depend on what else is in the batch).
 *   queries      bf16 [B, K+1, q_heads, head_dim] (device, 16-byte aligned),
 *                query_stride elements between tokens (at least q_heads *
 *                head_dim, a multiple of 8). Rows t > budgets[b] are never read.
 *   B, K         requests (0..SV_MAX_BATCH; 0 is a no-op), drafted tokens
 *                (0..SV_MAX_K).
 *   q_heads      a multiple of kv_heads, up to SV_MAX_HEADS.
 *   scale        finite; usually 1 / sqrt(head_dim). |scale| log2(e) is held
 *                within fp32's normal numbers. A score scale log2(e) q . k above
 *                fp32's range gives NaN; positions whose score is below it have
 *                no weight (NaN where a row sees no other).
 *   window       0, or the number of positions a row sees, its own included.
 *                Pages wholly before every row's window are not needed, and
 *                positions before it need never have been written.
 *   out          bf16 [B, K+1, q_heads, head_dim] (device, 16-byte aligned).
 *                Rows t > budgets[b] and empty slots keep their values. It may
 *                not overlap any other argument.
 *   workspace    device scratch of at least
 *                spec_verify_attention_workspace_bytes() bytes (256-byte
 *                aligned), caller-owned, its contents of no account; calls
 *                that share it must not overlap.
 * Errors (nothing enqueued): SV_ERR_ARG, SV_ERR_NULL, SV_ERR_ALIGN;
 * SV_ERR_HIP if a launch fails.
 */
int spec_verify_attention(const void* queries, int64_t query_stride, const void* cache,
                          const int32_t* page_table, const int32_t* ctx_lens,
                          const int32_t* budgets, int B, int K, int q_heads, int kv_heads,
                          int head_dim, int page_size, int max_pages, int num_pages, float scale,
                          int window, void* out, int32_t* out_status, void* workspace,
                          size_t workspace_bytes, void* stream);

/* spec_verify_attention_workspace_bytes -- scratch spec_verify_attention
 * needs; 0 on bad arguments. Host only. */
size_t spec_verify_attention_workspace_bytes(int B, int K, int q_heads, int kv_heads,
                                             int head_dim, int page_size, int max_pages,
                                             int window);

/*
 * spec_verify_attention_sinks -- spec_verify_attention under a window with
 * sinks: a row at position p also sees the positions [0, min(sinks, p + 1)) in
 * front of its window, each position once. Everything else, errors included, as
 * there; with window 0 or sinks 0 it is that call.
 *   sinks        0 or more. Pages between the sinks and every row's window are
 *                not needed.
 */
int spec_verify_attention_sinks(const void* queries, int64_t query_stride, const void* cache,
                                const int32_t* page_table, const int32_t* ctx_lens,
                                const int32_t* budgets, int B, int K, int q_heads, int kv_heads,
                                int head_dim, int page_size, int max_pages, int num_pages,
                                float scale, int window, int sinks, void* out,
                                int32_t* out_status, void* workspace, size_t workspace_bytes,
                                void* stream);

/* spec_verify_attention_sinks_workspace_bytes -- scratch
 * spec_verify_attention_sinks needs; 0 on bad arguments. Host only. */
size_t spec_verify_attention_sinks_workspace_bytes(int B, int K, int q_heads, int kv_heads,
                                                   int head_dim, int page_size, int max_pages,
                                                   int window, int sinks);

/*
 * spec_verify_attention_shared -- spec_verify_attention (without a window) for
 * requests that share a prefix: what the requests of a group have in common is
 * read and computed once for all their rows. The result is that call's but for
 * the order of its sums. Three launches (with G = 0 it is that call), which pay
 * where many rows stand behind a long prefix: from about 64 requests behind 2,000
 * tokens or 32 blocks behind 8,000 on (8 kv heads of 128); spec_verify_attention
 * is the faster one below.
 *   groups       int32 [B] (device): the group of request b; a number outside
 *                [0, G): none.
 *   shared_lens  int32 [G] (device): tokens from position 0 on that all
 *                requests of the group have in common: the page table rows
 *                agree on the pages that lie wholly in front of it or the
 *                tokens are the same. Read through the row of the group's
 *                first request that holds any (a bad page there leaves the
 *                whole group's outputs undefined). Whole tiles of 32 tokens up
 *                to the shortest context of the group are shared; groups of
 *                fewer than two requests, and lengths below 32, share nothing.
 *   G            0 (nothing is shared) .. SV_MAX_GROUPS.
 *   workspace    at least spec_verify_attention_shared_workspace_bytes() bytes;
 *                it holds fp32 partial results of all rows.
 * Everything else as in spec_verify_attention.
 */
int spec_verify_attention_shared(const void* queries, int64_t query_stride, const void* cache,
                                 const int32_t* page_table, const int32_t* ctx_lens,
                                 const int32_t* budgets, const int32_t* groups,
                                 const int32_t* shared_lens, int B, int K, int G, int q_heads,
                                 int kv_heads, int head_dim, int page_size, int max_pages,
                                 int num_pages, float scale, void* out, int32_t* out_status,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* spec_verify_attention_shared_workspace_bytes -- scratch
 * spec_verify_attention_shared needs; 0 on bad arguments. Host only. */
size_t spec_verify_attention_shared_workspace_bytes(int B, int K, int G, int q_heads,
                                                    int kv_heads, int head_dim, int page_size,
                                                    int max_pages);

/*
 * The output head in 8-bit floating point (the shared projection of "What
 * DSpark adds", paragraph 1, held in half of bf16's bytes).
 *
 * Codes are e4m3 (largest 448), rows padded with zeros to Hp = H rounded up
 * to a multiple of 128; scales are bytes 2^(byte - 127), 255 = not a number,
 * one per block: a row's 128 channels, or 128 x 128 of a head. The scale is
 * the smallest power of two, at least 2^-64, under which the block's largest
 * magnitude is at most 448 (at most 2^119: larger magnitudes saturate); codes
 * are rounded to nearest, ties to even. A block that holds a NaN or an
 * infinity has NaN codes and scale.
 */

/*
 * spec_head_quantize -- quantise hidden states or a head. Stream-ordered, one
 * launch (several for states of more than 2^31 / 16 blocks).
 *   src         [rows, H] of type dtype (sv_dtype), row-major (device,
 *               16-byte aligned); rows 0..SV_MAX_VOCAB (0 is a no-op), H a
 *               multiple of 8, 8..SV_MAX_HIDDEN.
 *   block_rows  1 (states) or 128 (a head).
 *   out_codes   uint8 [rows, Hp] (device, 16-byte aligned).
 *   out_scales  uint8 [ceil(rows / block_rows), Hp / 128] (device).
 * Errors (nothing enqueued): SV_ERR_ARG, SV_ERR_DTYPE, SV_ERR_NULL,
 * SV_ERR_ALIGN; SV_ERR_HIP if the launch fails.
 */
int spec_head_quantize(const void* src, int dtype, int rows, int H, int block_rows,
                       void* out_codes, void* out_scales, void* stream);

/*
 * spec_head_logits -- logits of quantised states under a quantised head,
 *   out[r, v] = sum_i (h[r, i] s_h) (w[v, i] s_w),
 * the rows that spec_verify_run reads. Stream-ordered, one launch.
 *   h_codes, h_scales  R states quantised with block_rows = 1.
 *   w_codes, w_scales  the head, V rows quantised with block_rows = 128.
 *   R, H, V    rows (0..SV_MAX_VOCAB; 0 is a no-op), hidden size
 *              (1..SV_MAX_HIDDEN; codes have Hp channels), vocabulary
 *              (1..SV_MAX_VOCAB).
 *   dtype      type of out (sv_dtype). fp32 logits are fp32 accumulations of
 *              exact products. bf16 logits may come from the 8-bit matrix
 *              instructions, whose sums keep about 16 bits (1e-5 relative to
 *              the row, measured), before they are rounded to 8.
 *   out        [R, V] row-major (device, aligned to its element size).
 * Codes are 16-byte aligned.
 * Errors (nothing enqueued): SV_ERR_ARG, SV_ERR_DTYPE, SV_ERR_NULL,
 * SV_ERR_ALIGN; SV_ERR_HIP if the launch fails.
 */
int spec_head_logits(const void* h_codes, const void* h_scales, const void* w_codes,
                     const void* w_scales, int R, int H, int V, int dtype, void* out,
                     void* stream);

/* spec_verify_free -- release the context (NULL-safe, idempotent on NULL).
 * Waits for the device before freeing the workspace. */
void spec_verify_free(spec_verify_ctx* ctx);

/* spec_verify_strerror -- static text for an sv_status code. */
const char* spec_verify_strerror(int code);

/* spec_verify_chunks -- number of vocabulary chunks a row is split into for
 * (vocab, dtype) in sampled mode (the unit of the workspace's per-chunk
 * records; greedy calls use chunks twice as long), or a negative sv_status
 * on bad arguments. Host only. */
int spec_verify_chunks(int vocab, int dtype);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */

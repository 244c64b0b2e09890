/*
 * spec_verify.h -- C interface of the batched speculative-decoding verify step
 * (accept/reject of draft tokens plus the corrected or bonus draw) on an
 * AMD Instinct MI355X (gfx950).
 *
 * What one call computes, for every sequence s of a batch (K = K_s proposed
 * tokens x_0..x_{K-1}, target logits at K+1 positions, draft logits at K):
 *
 *   p_i = softmax(target_i / T),  q_i = softmax(draft_i / T)
 *       Both logit rows are divided by the temperature before the softmax
 *       (gitcode.csdn.net tutorial, section 4.3).
 *   scan i = 0..K-1: accept x_i iff u_i < min(1, p_i(x_i) / q_i(x_i)),
 *       stop at the first rejection
 *       ("Draft Model（草稿模型）", compassingai.com, section 2
 *       接受-拒绝准则 and the one-step algorithm box under 技术原理).
 *   on a rejection at A: draw from norm(max(0, p_A - q_A))
 *       (same page, section 2; tutorial section 3.2);
 *   if all K are accepted: draw one bonus token from p_K
 *       (same page, the one-step algorithm box).
 *   One round therefore emits between 1 and K+1 tokens.
 *
 * Modes per sequence:
 *   SV_SAMPLE  the rule above.
 *   SV_ONEHOT  deterministic proposal (N-gram / prompt lookup): q is the
 *              one-hot distribution on the proposed token, so x_i is accepted
 *              iff u_i < p_i(x_i), and a rejection draws from p_A with x_A
 *              removed ("5.2 Draft 模型与无模型方案", AIInfraGuide, section 4.3).
 *              No draft logits are read.
 *   SV_GREEDY  strict greedy: accept iff x_i is the argmax of the raw target
 *              logits (lowest index on ties); emit that argmax on a mismatch
 *              and as the bonus.  The temperature is ignored.
 *   SV_STRICT  sample match ("Speculative Decoding在分布式推理中的应用",
 *              wmrh.cn, sections 二 and 三): the target draws its own token
 *              y_i ~ p_i by the inverse CDF with u_i; x_i is accepted iff
 *              y_i = x_i, and on a mismatch y_A is emitted (it is the draw
 *              from p_A with x_A removed, at the point u_A*S minus x_A's mass
 *              when u_A lies above x_A's interval).  All K accepted: bonus
 *              from p_K as above.  Lossless; the acceptance probability is
 *              p_i(x_i).  No draft logits are read.
 *
 * Randomness: u_i and the final draw's uniform come from Philox4x32-10
 * (Salmon et al., SC'11) with key = seed and counter = (position, purpose,
 * seq_id, 0); purpose 0 for u_i at positions 0..K-1, purpose 1 for the final
 * draw at position A (SV_STRICT draws its correction with u_A, purpose 0,
 * and only its bonus with purpose 1); u = (word0 >> 8) * 2^-24.  Results are a pure function
 * of (inputs, seed, seq_ids): any call can be replayed exactly, and a batch
 * split across calls (with global seq_ids) gives the same outputs.
 *
 * Filters (top_k / top_p, optional): top-k and nucleus rejection sampling
 * keep the target's distribution ("Draft Model（草稿模型）", compassingai.com,
 * 常见误读纠偏 误读 4; gitcode.csdn.net tutorial, section 5.4): each used row
 * of a filtered SAMPLE, ONEHOT or STRICT sequence (target and draft alike)
 * keeps the tokens with logit >= tau and is renormalised before the rule
 * above; GREEDY ignores the filter.  top-k: tau is the k-th largest logit
 * (ties at it all kept).  top-p, after top-k: a token is kept iff the mass of
 * the strictly larger tokens is below p (the largest logit always kept).
 * The output then follows the filtered target distribution.  A filtered
 * call runs one more kernel (one block per used row of a filtered sequence)
 * that reads those rows again: whole, or only the parts whose maximum can
 * reach the row's threshold.
 *
 * Final draw: inverse CDF over the unnormalised weights w (residual, one-hot
 * residual or p_K): t = u * sum(w), emit the first token k whose inclusive
 * prefix sum exceeds t; tokens with w = 0 are never emitted.
 *
 * Packed ragged layout (no padding between sequences):
 *   off_d[s] = sum_{j<s} K_j            draft rows / draft_tokens / p,q at proposal
 *   off_t[s] = off_d[s] + s             target rows / emitted_tokens
 *   target row off_t[s]+i judges draft token i; row off_t[s]+K_s is the bonus row.
 *   Logit rows are ld elements apart (ld >= vocab); columns >= vocab are never read.
 *   Logits pointers are aligned to their element size (4 bytes fp32, 2 bf16).
 *
 * Arithmetic: float32 (logits are read as float32 or bfloat16 and widened
 * exactly); exp2-based online max/sum; fixed-order reductions, no float
 * atomics, so repeated calls are bitwise identical.
 *
 * Threading: a context owns device scratch memory; calls that share a context
 * must be ordered on one stream.  Use one context per concurrent stream.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct spec_verify_ctx spec_verify_ctx;

/* element types: logits are SV_F32 or SV_BF16, cached keys and values SV_BF16 or SV_F16 */
enum { SV_F32 = 0, SV_BF16 = 1, SV_F16 = 2 };

/* per-sequence verify mode (values of args->mode[s]) */
enum { SV_SAMPLE = 0, SV_GREEDY = 1, SV_ONEHOT = 2, SV_STRICT = 3 };

/* return codes */
enum {
  SV_OK = 0,
  SV_ERR_INVALID = -1,   /* bad argument; nothing was enqueued */
  SV_ERR_NOMEM = -2,     /* device allocation failed (create / timing_enable only) */
  SV_ERR_HIP = -3,       /* a HIP call failed; see spec_verify_last_error() */
  SV_ERR_CAPACITY = -4   /* the call exceeds the sizes given to spec_verify_create */
};

/* per-sequence status bits (args->status[s]).  Any bit in 1..64 means the
 * sequence was not verified: accepted_len = -1, its emitted slots are -1 and
 * its p/q at proposal are NaN.  Bit 128 is informational. */
enum {
  SV_ST_BAD_LAYOUT = 1,        /* num_draft has a negative entry or does not sum to total_draft (set for every sequence; every output slot is cleared) */
  SV_ST_K_TOO_LARGE = 2,       /* K_s > max_k of the context */
  SV_ST_BAD_MODE = 4,          /* mode[s] not one of SV_SAMPLE, SV_GREEDY, SV_ONEHOT, SV_STRICT */
  SV_ST_BAD_TEMPERATURE = 8,   /* SAMPLE/ONEHOT/STRICT with temperature not finite or below SV_MIN_TEMPERATURE */
  SV_ST_NO_DRAFT_LOGITS = 16,  /* SAMPLE sequence with K_s > 0 but draft_logits == NULL */
  SV_ST_BAD_TOKEN = 32,        /* a proposed token outside [0, vocab) */
  SV_ST_NONFINITE = 64,        /* a used logit row holds NaN or +inf, or is entirely -inf */
  SV_ST_ZERO_RESIDUAL = 128,   /* the residual had no mass (rounding only); the token was drawn from p_A instead */
  /* the paged cache's operators only */
  SV_ST_BAD_SEQ = 256,         /* a sequence slot outside the cache, or named twice where it may be named once */
  SV_ST_BAD_LENGTH = 512,      /* a length or token count that is negative or does not fit */
  SV_ST_BAD_PAGE = 1024,       /* a page outside the pool */
  SV_ST_CACHE_FULL = 2048      /* the pool has too few free pages */
};

/* smallest accepted temperature for SAMPLE/ONEHOT/STRICT (float32 1e-6) */
#define SV_MIN_TEMPERATURE 1e-6f

typedef struct spec_verify_args {
  int32_t batch;               /* B >= 0 (host value); 0 is a no-op */
  int64_t vocab;               /* V >= 1 (host value) */
  int64_t total_draft;         /* sum_s K_s (host value): sizes the grids, must match num_draft */
  int32_t target_dtype;        /* SV_F32 or SV_BF16 */
  int32_t draft_dtype;         /* SV_F32 or SV_BF16 (ignored when draft_logits == NULL) */
  const void* target_logits;   /* device, [total_draft + B][ld_target] */
  int64_t ld_target;           /* elements between target rows, >= vocab */
  const void* draft_logits;    /* device, [total_draft][ld_draft], or NULL if no SV_SAMPLE sequence has K_s > 0 */
  int64_t ld_draft;            /* elements between draft rows, >= vocab */
  const int32_t* draft_tokens; /* device, [total_draft]; may be NULL iff total_draft == 0 */
  const int32_t* num_draft;    /* device, [B], K_s */
  const float* temperature;    /* device, [B], or NULL (= 1.0 for every sequence) */
  const uint8_t* mode;         /* device, [B], or NULL (= SV_SAMPLE for every sequence) */
  const uint32_t* seq_ids;     /* device, [B], or NULL (= s): Philox counter word 2 */
  uint64_t seed;               /* Philox key */
  int32_t* accepted_len;       /* device out, [B]: accepted draft tokens A_s (0..K_s), -1 if not verified */
  int32_t* emitted_tokens;     /* device out, [total_draft + B]: seq s at off_t[s]: x_0..x_{A-1}, y, then -1 */
  float* p_at_proposal;        /* device out, [total_draft] or NULL: p_i(x_i) for every i < K_s (T = 1 for GREEDY) */
  float* q_at_proposal;        /* device out, [total_draft] or NULL: q_i(x_i); 1.0 for ONEHOT and GREEDY */
  int32_t* status;             /* device out, [B] or NULL: SV_ST_* bits */
  const int32_t* top_k;        /* device, [B], or NULL: top-k filter per sequence (<= 0 or >= vocab: off) */
  const float* top_p;          /* device, [B], or NULL: top-p filter per sequence (>= 1 or NaN: off) */
} spec_verify_args;

/* Create a context on HIP device `device` for batches of at most max_batch
 * sequences, K_s <= max_k (1..128) and vocab <= max_vocab.  Allocates the
 * context's device scratch (per-chunk partial row statistics and, for the
 * filters, 32 segment maxima per chunk; per-sequence final-draw records
 * and tile sums; defaults for NULL optional inputs): about 144 bytes per 8192
 * vocabulary entries per row slot, max_batch * (2 * max_k + 1) slots, plus
 * small per-slot and per-sequence arrays (among them the filter's list of
 * rows).  The caller owns every input and output
 * buffer.  Returns SV_OK and sets *out, or an error code (then *out = NULL). */
int spec_verify_create(spec_verify_ctx** out, int device, int32_t max_batch, int32_t max_k, int64_t max_vocab);

/* Enqueue one verify step on `hip_stream` (a hipStream_t; NULL = the null
 * stream).  Validates the host-side arguments first (SV_ERR_INVALID /
 * SV_ERR_CAPACITY: nothing is enqueued); problems that only the device can
 * see are reported per sequence through `status`.  Does not allocate, does
 * not synchronise; outputs are valid once the stream has reached this point.
 * Launches two kernels (three with top_k / top_p): row statistics (one
 * block per 32 KB of every logit row); final (per sequence: the acceptance
 * test, then the sums of the final weights over 8192-element tiles of the
 * row(s) at the stop position and the inverse-CDF search; for batches below
 * 128 a sequence's tiles are spread over several blocks, and the last of
 * them to store its tile sums does the search).  The timing slot "select"
 * is kept for the interface and reads 0. */
int spec_verify_run(spec_verify_ctx* ctx, const spec_verify_args* args, void* hip_stream);

/* ---- allocation-free call --------------------------------------------------
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * step as spec_verify_run, without a context.  Its scratch is one array of
 * SV_NOALLOC_SCRATCH_BYTES bytes in the library's device data, which every
 * GPU the library runs on holds until the process ends; it is laid out per
 * call for exactly the call's sizes (about 16 bytes per 32 KB chunk of each
 * of batch * (2 * max_k + 1) row slots, eight times that more with top_k /
 * top_p, plus small per-sequence arrays).  max_k (1..128) plays the part of
 * the context's max_k (K_s > max_k: status SV_ST_K_TOO_LARGE); batch <= 4096.
 * A call that would need more scratch returns SV_ERR_CAPACITY with the
 * needed size in the message; other checks and errors as spec_verify_run.
 * Runs on the calling thread's current device (hip_stream must belong to
 * it).  Allocates nothing; the first call on a device looks up the array's
 * address and writes the defaults for NULL temperature / mode / seq_ids with
 * synchronous copies, so make one call on each device before capturing a
 * graph.  All calls on one GPU share its array and it keeps the last call's
 * contents: calls that overlap on one GPU (concurrent streams or threads)
 * race and give undefined results.  No timing hooks. */
#define SV_NOALLOC_SCRATCH_BYTES 67108864
int spec_verify_run_noalloc(const spec_verify_args* args, int32_t max_k, void* hip_stream);

/* Free the context and its device memory.  NULL is accepted. */
void spec_verify_destroy(spec_verify_ctx* ctx);

/* Message of the last failing call on this thread (static storage). */
const char* spec_verify_last_error(void);

/* ---- measurement hooks ---------------------------------------------------
 * spec_verify_timing_enable(ctx, n) makes the next n calls of
 * spec_verify_run time each of its kernel slots with a pair of HIP events
 * that the dispatch itself records (hipExtLaunchKernel), so a slot's time is
 * its kernel's execution, without event gaps (n = 0 turns it off; events are
 * created here, never inside run).  spec_verify_timing_read waits for those events and
 * returns the number of recorded calls and, per slot, the summed elapsed
 * milliseconds (ms_per_kernel has SV_NUM_KERNELS entries: row statistics,
 * filter, final, select; a slot whose kernel was not launched reads 0),
 * then resets the record. */
#define SV_NUM_KERNELS 4
int spec_verify_timing_enable(spec_verify_ctx* ctx, int32_t max_calls);
int spec_verify_timing_read(spec_verify_ctx* ctx, int32_t* calls, double* ms_per_kernel);

/* ---- N-gram (prompt-lookup) proposer -------------------------------------
 * "5.2 Draft 模型与无模型方案" (AIInfraGuide), sections 4.1-4.3 and the lookup
 * experiment of section 6: for each sequence, the last n token ids of its
 * history are looked up earlier in the same history and the tokens that
 * followed become a deterministic proposal, which the target then verifies
 * as a one-hot draft (spec_verify_run with mode SV_ONEHOT).
 *
 * With history h of length L and window n, a start s is an occurrence when
 * h[s .. s+n-1] equals h[L-n .. L-1] and s + n < L - n (the occurrence ends
 * before the tail and at least one token follows it outside the tail).  The
 * chosen occurrence has the largest n in [min_n, max_n], then the largest s;
 * the proposal is h[s+n .. min(s+n+max_tokens, L-n) - 1] (never copied from
 * the tail).  No occurrence: an empty proposal.
 *
 * All pointers are device pointers owned by the caller.
 *   history        [total_len] int32 token ids; sequence b is
 *                  history[hist_offsets[b] .. hist_offsets[b+1] - 1]
 *   hist_offsets   [batch + 1] int64
 *   total_len      host value: the length of `history`; bounds every read
 *   min_n, max_n   1 <= min_n <= max_n <= SV_NGRAM_MAX_N
 *   max_tokens     1 .. SV_NGRAM_MAX_TOKENS
 *   draft_tokens   out [batch * max_tokens] int32: sequence b's proposal at
 *                  b * max_tokens, -1 after it
 *   num_draft      out [batch] int32: proposal length (0: none)
 *   match_n        out [batch] int32 or NULL: the window that matched (0:
 *                  none; -1: sequence b's offsets are out of order or outside
 *                  total_len, and nothing of it was read)
 * spec_verify_ngram_propose checks the host-side values (SV_ERR_INVALID:
 * nothing is enqueued), enqueues one kernel on `hip_stream` (one block per
 * sequence), allocates nothing and does not synchronise.  It needs no
 * context. */
#define SV_NGRAM_MAX_N 16
#define SV_NGRAM_MAX_TOKENS 128
typedef struct spec_verify_ngram_args {
  int32_t batch;
  const int32_t* history;
  const int64_t* hist_offsets;
  int64_t total_len;
  int32_t min_n;
  int32_t max_n;
  int32_t max_tokens;
  int32_t* draft_tokens;
  int32_t* num_draft;
  int32_t* match_n;
} spec_verify_ngram_args;
int spec_verify_ngram_propose(const spec_verify_ngram_args* args, void* hip_stream);

/* sizeof(spec_verify_ngram_args) as compiled into the library. */
int64_t spec_verify_ngram_args_size(void);

/* ---- acceptance statistics ------------------------------------------------
 * "5.2 Draft 模型与无模型方案" (AIInfraGuide), section 7: over R verify rounds
 * that proposed D draft tokens of which C were accepted, the draft acceptance
 * rate is C / D and the mean acceptance length 1 + C / R (a complete round
 * also commits its corrected or bonus token); candidate coverage is the
 * share of rounds that had any candidate; per position, the conditional
 * acceptance rate (among rounds that reached the position) differs from the
 * rate of being accepted all the way through it.
 *
 * A round is one sequence of one verify call: K = num_draft[s], A =
 * accepted_len[s].  spec_verify_stats_accumulate ADDS one call's rounds to
 * `stats`, device uint64 [SV_STATS_WORDS(max_k)], owned by the caller, who
 * zeroes it to start an observation window (with a fill kernel or a copy;
 * the library never clears it):
 *   [0] R rounds counted             [4] rounds with K > 0 and A = K
 *   [1] D = sum K                    [5] rounds not counted: A < 0 (not
 *   [2] C = sum A                        verified), K outside 0..max_k, A > K
 *   [3] rounds with K > 0            [6] emitted tokens sum (A + 1)   [7] 0
 *   [8 + i]            rounds with K > i                 (proposed at i)
 *   [8 + max_k + i]    rounds with K > i and A >= i      (reached i)
 *   [8 + 2 max_k + i]  rounds with A > i                 (accepted at i)
 * Counts are exact (integer sums, no atomics).  num_draft and accepted_len
 * are device int32 [batch] (for instance the verify call's own arrays, on
 * the same stream).  One block of the kernel walks the batch: meant for the
 * batch of one decode step.
 *
 * spec_verify_stats_summary writes device float64 [SV_STATS_SUMMARY_WORDS]:
 *   [0] C / D   [1] 1 + C / R   [2] [3] / R (coverage)   [3] [4] / [3]
 *   [4 + i]          conditional acceptance at i: accepted_i / reached_i
 *   [4 + max_k + i]  accepted through i:          accepted_i / proposed_i
 * NaN where the denominator is 0; each value is one correctly rounded
 * float64 division of the counts (plus 1.0 for [1]).
 * Both enqueue one kernel on `hip_stream`, allocate nothing and do not
 * synchronise; SV_ERR_INVALID (nothing enqueued) for max_k outside
 * 1..SV_STATS_MAX_K, batch < 0 or a missing buffer. */
#define SV_STATS_MAX_K 128
#define SV_STATS_WORDS(max_k) (8 + 3 * (max_k))
#define SV_STATS_SUMMARY_WORDS(max_k) (4 + 2 * (max_k))
int spec_verify_stats_accumulate(int32_t batch, int32_t max_k, const int32_t* num_draft,
                                 const int32_t* accepted_len, uint64_t* stats, void* hip_stream);
int spec_verify_stats_summary(int32_t max_k, const uint64_t* stats, double* summary, void* hip_stream);

/* ---- draft-length controllers ---------------------------------------------
 * One controller per sequence slot, fed after each round with (K, A) and
 * giving the proposal length of the next round; a round with A < 0 changes
 * nothing.  The ratio a controller sees depends on `count`:
 *   SV_ADAPT_COUNT_EMITTED (0, the pages' count)  min(A + 1, K) / K, and 0
 *       when K = 0: the tutorial's verifier returns the accepted draft
 *       tokens plus the token drawn after a rejection, without a bonus token
 *       (gitcode.csdn.net tutorial, section 4.3 验证器实现), and its decoder
 *       feeds len(accepted_tokens) / draft_len (section 4.4 完整的解码器);
 *       "Speculative Decoding在分布式推理中的应用" (wmrh.cn), section 三,
 *       counts the resampled token the same way.
 *   SV_ADAPT_COUNT_DRAFT_ONLY (1)  A / max(K, 1): accepted draft tokens only.
 * Decisions are taken in float64.
 *   SV_ADAPT_WINDOW          keep the last `window` ratios; once at least
 *       `min_samples` are held, their mean (summed oldest first) above
 *       target + 0.1 lengthens by one, below target - 0.1 shortens by one,
 *       within [min_k, max_k] (tutorial, section 5.2 动态草稿长度策略; the
 *       page's defaults are window 100, min_samples 10, target 0.7,
 *       length 5 in 1..10).
 *   SV_ADAPT_MULTIPLICATIVE  above target + 0.1 the length L becomes
 *       min(max_k, int(L (1 + rate))), below target - 0.1
 *       max(min_k, int(L (1 - rate))); int truncates (tutorial, section
 *       4.4; defaults target 0.7, rate 0.1, lengths 1..5).
 *   SV_ADAPT_OPTIMAL_K       a = max(ratio, 0.01), k* = floor(ln(1/(1-a))/a)
 *       (unbounded at a = 1), L becomes min(clamp(k*, 2, 16), max(L, 2));
 *       min_k, max_k, window and rate are not used (wmrh.cn, section 三,
 *       adapt_draft_length).
 *
 * state: device memory owned by the caller, SV_ADAPT_STATE_BYTES(batch,
 * window) bytes, 16-byte aligned: int32 [batch][4] {length, count, head, 0},
 * then float64 [batch][window] ratio rings.  spec_verify_adapt_reset sets
 * every length to init_k and empties the rings (call it first, and again
 * after changing kind, window or count); spec_verify_adapt reads num_draft and
 * accepted_len (device int32 [batch]), updates the state and writes next_k
 * (device int32 [batch]; also for unchanged lengths).  Sequence b always
 * uses slot b.  Each call enqueues one kernel on `hip_stream`, allocates
 * nothing and does not synchronise; SV_ERR_INVALID (nothing enqueued) for a
 * bad kind or count, bounds outside 1 <= min_k <= max_k <= SV_ADAPT_MAX_LENGTH,
 * window outside 1..SV_ADAPT_MAX_WINDOW or min_samples < 1 (window kind),
 * target or rate outside [0, 1], init_k outside 1..SV_ADAPT_MAX_LENGTH, or a
 * missing or misaligned buffer. */
enum { SV_ADAPT_WINDOW = 0, SV_ADAPT_MULTIPLICATIVE = 1, SV_ADAPT_OPTIMAL_K = 2 };
enum { SV_ADAPT_COUNT_EMITTED = 0, SV_ADAPT_COUNT_DRAFT_ONLY = 1 };
#define SV_ADAPT_MAX_WINDOW 256
#define SV_ADAPT_MAX_LENGTH 4096
#define SV_ADAPT_STATE_BYTES(batch, window) ((int64_t)(batch) * (16 + 8 * (int64_t)(window)))
typedef struct spec_verify_adapt_args {
  int32_t batch;
  int32_t kind;
  int32_t min_k;
  int32_t max_k;
  int32_t window;
  int32_t min_samples;
  int32_t count;               /* SV_ADAPT_COUNT_EMITTED or SV_ADAPT_COUNT_DRAFT_ONLY */
  double target;
  double rate;
  const int32_t* num_draft;
  const int32_t* accepted_len;
  void* state;
  int32_t* next_k;
} spec_verify_adapt_args;
int spec_verify_adapt_reset(const spec_verify_adapt_args* args, int32_t init_k, void* hip_stream);
int spec_verify_adapt(const spec_verify_adapt_args* args, void* hip_stream);

/* sizeof(spec_verify_adapt_args) as compiled into the library. */
int64_t spec_verify_adapt_args_size(void);

/* ---- log probabilities of given tokens -------------------------------------
 * For each of `rows` rows of logits (a verify call's target rows, for
 * instance: its emitted_tokens has one entry per target row, so the two go
 * together as they are) and one token per row:
 *   logprob  log softmax(x / T)[token], natural logarithm
 *   entropy  -sum p log p of softmax(x / T), in nats
 *   rank     1 + the number of logits strictly above the token's
 *   top_*    the `top` largest logits' tokens, best first (the lower index
 *            first on ties), and their log probabilities
 * A row whose token is negative (the -1 behind a round's emitted tokens) is
 * not read: logprob 0, entropy 0, rank 0, top tokens -1 with -inf.  With
 * tokens == NULL every row is read, for entropy and top alone.
 * All pointers are device pointers owned by the caller.
 *   logits         [rows][ld], SV_F32 or SV_BF16, ld >= vocab, aligned to
 *                  the element size; columns >= vocab are never read
 *   tokens         [rows] int32 or NULL (then logprob and rank are NULL too)
 *   temperature    [rows] float or NULL (= 1.0)
 *   top            0 .. SV_LOGPROBS_MAX_TOP, at most vocab
 *   logprob, entropy, rank, top_logprobs, status   each may be NULL
 *   top_tokens     [rows * top] int32, required for top > 0
 *   status         SV_ST_BAD_TOKEN (token >= vocab), SV_ST_BAD_TEMPERATURE
 *                  (as for a verify call) or SV_ST_NONFINITE (the row holds
 *                  NaN or +inf, or is entirely -inf): the row's values are
 *                  then NaN, its rank 0 and its top tokens -1
 *   workspace      16-byte aligned, at least
 *                  spec_verify_logprobs_workspace(...) bytes; its contents
 *                  need not survive the call, and calls that may overlap
 *                  each need their own
 * Sums are float32 in a fixed order: repeated calls are bitwise identical.
 * Enqueues two kernels on `hip_stream`, which belongs to the calling
 * thread's current device; allocates nothing, does not synchronise.
 * SV_ERR_INVALID: nothing was enqueued.  rows == 0 is a no-op. */
#define SV_LOGPROBS_MAX_TOP 64
typedef struct spec_verify_logprobs_args {
  int64_t rows;
  int64_t vocab;               /* 1 .. 2097152 */
  int32_t dtype;
  int32_t top;
  const void* logits;
  int64_t ld;
  const int32_t* tokens;
  const float* temperature;
  float* logprob;
  float* entropy;
  int32_t* rank;
  int32_t* top_tokens;
  float* top_logprobs;
  int32_t* status;
  void* workspace;
  int64_t workspace_bytes;
} spec_verify_logprobs_args;
int spec_verify_token_logprobs(const spec_verify_logprobs_args* args, void* hip_stream);

/* Bytes of workspace for these sizes, or SV_ERR_INVALID. */
int64_t spec_verify_logprobs_workspace(int64_t rows, int64_t vocab, int32_t dtype, int32_t top);

/* sizeof(spec_verify_logprobs_args) as compiled into the library. */
int64_t spec_verify_logprobs_args_size(void);

/* ---- attention over a paged key-value cache ---------------------------------
 * The attention of the target's verification pass: sequence b brings n =
 * num_draft[b] + 1 new tokens (its last emitted one and its drafts; n = 1 is
 * plain decoding), whose query rows are packed like a verify call's target
 * rows.  Its keys and values lie in pages and are in the cache already:
 * seq_len tokens, the n new ones last.  Query row i sees the positions
 * j <= seq_len - n + i, with window > 0 only the last `window` of them:
 *   out = sum_j softmax_j(scale * q . k_j) v_j,  lse = ln sum_j exp(scale * q . k_j)
 * `heads` query heads share `kv_heads` key heads in groups of neighbours
 * (query head h reads key head h / (heads / kv_heads)).  A row that sees
 * nothing gets out = 0 and lse = -inf.  Keys and values that a row does not
 * see have no effect on it, whatever they hold; a row that sees one that is
 * not finite is not finite itself (where its weight is not 0).
 * All pointers are device pointers owned by the caller.
 *   q              [total_rows][heads][head_dim], dtype SV_BF16 or SV_F16
 *   k, v           [num_pages][kv_heads][page_size][head_dim] of the same
 *                  type, in any order of the first three: strides in elements
 *                  for page, head and token; head_dim is contiguous
 *   page_table     [slots][page_table_stride] int32: entry j of a row holds
 *                  tokens j * page_size ..; max_pages entries may be used
 *   seq_len        [slots] int32
 *   seqs           [batch] int32: sequence b is row seqs[b] of page_table and
 *                  seq_len (a slot may be named more than once); NULL: row b
 *   num_draft      [batch] int32, sum of (num_draft + 1) = total_rows
 *   start          [batch] int32 or NULL: what spec_verify_cache_reserve gave
 *                  for the n new tokens; a sequence that it refused (-1), or
 *                  whose seq_len is not start + n, has none and is refused
 *   out            [total_rows][heads][head_dim], contiguous
 *   lse            [total_rows][heads] float or NULL
 *   status         [batch] int32 or NULL
 *   workspace      16-byte aligned, at least spec_verify_attention_workspace()
 *                  bytes; its contents need not survive the call, and calls
 *                  that may overlap each need their own
 * head_dim 64, 128 or 256; page_size a power of two from 16 to 1024; q, k, v
 * and out 16-byte aligned with strides in multiples of 8 elements; batch <=
 * 4096, total_rows <= 524288, heads / kv_heads <= 256.
 * Scores, softmax and sums are float32, the softmax's weights enter the
 * second product as the sum of two 16-bit values (held to 2^-16 of themselves
 * for SV_BF16; to 2^-22, or 2^-39 of a row's largest, for SV_F16), the result
 * is rounded once.
 * Repeated calls are bitwise identical.
 * What only the device can see: num_draft that does not add up sets
 * SV_ST_BAD_LAYOUT for every sequence and every output is NaN; a sequence
 * with SV_ST_BAD_SEQ (slot outside 0..slots-1), SV_ST_BAD_LENGTH (seq_len
 * negative, above max_pages * page_size or not what start says) or
 * SV_ST_BAD_PAGE (a page that holds visible tokens is outside the pool) gets
 * NaN, and no such page is read.
 * Enqueues two kernels on `hip_stream`, which belongs to the calling
 * thread's current device; allocates nothing, does not synchronise.
 * SV_ERR_INVALID: nothing was enqueued.  batch == 0 (without rows) is a no-op. */
typedef struct spec_verify_attention_args {
  int32_t batch;
  int32_t total_rows;
  int32_t heads;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t dtype;
  int32_t page_size;
  int32_t window;              /* 0: every earlier position */
  int64_t num_pages;
  int32_t slots;
  int32_t max_pages;
  int64_t page_table_stride;   /* >= max_pages */
  const void* q;
  int64_t q_row_stride;
  int64_t q_head_stride;
  const void* k;
  int64_t k_page_stride;
  int64_t k_head_stride;
  int64_t k_token_stride;
  const void* v;
  int64_t v_page_stride;
  int64_t v_head_stride;
  int64_t v_token_stride;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* seqs;
  const int32_t* num_draft;
  double scale;                /* |scale| < 2.3e38; head_dim^-0.5 for the usual attention */
  void* out;
  float* lse;
  int32_t* status;
  void* workspace;
  int64_t workspace_bytes;
  const int32_t* start;
} spec_verify_attention_args;
int spec_verify_paged_attention(const spec_verify_attention_args* args, void* hip_stream);

/* Bytes of workspace for a call with these sizes (the pointers, strides and
 * tables of args are not looked at), or SV_ERR_INVALID. */
int64_t spec_verify_attention_workspace(const spec_verify_attention_args* args);

/* sizeof(spec_verify_attention_args) as compiled into the library. */
int64_t spec_verify_attention_args_size(void);

/* ---- the paged cache ---------------------------------------------------------
 * The pages that spec_verify_paged_attention reads, and what a decode loop
 * does with them around a verify call: reserve places for the K_s + 1 new
 * tokens of each sequence, write their keys and values (per layer), and after
 * the verify call commit what it accepted; fork a sequence into branches that
 * share its pages, release one, compact the pool.
 *
 * State, device memory owned by the caller, who starts it with page_table -1,
 * seq_len 0 and refcount 0:
 *   page_table  [slots][max_pages] int32: the sequence's pages in order, -1 behind them
 *   seq_len     [slots] int32: cached tokens
 *   refcount    [num_pages] int32, 16-byte aligned: sequences that use the page; 0: free
 *   k, v        [layers][num_pages][kv_heads][page_size][head_dim] of a 16-bit
 *               type, 16-byte aligned
 *   workspace   16-byte aligned, spec_verify_cache_workspace() bytes
 * slots <= SV_CACHE_MAX_SLOTS, max_pages <= 131072, page_size a power of two
 * from 16 to 1024, head_dim a multiple of 8, kv_heads * head_dim <= 65536,
 * num_pages < 2^30, layers <= 4096.
 *
 * Calls on one cache must be ordered on one stream (they change its state and
 * share its workspace).  Each names its sequences with seqs, int32 [batch]
 * (NULL: slots 0 .. batch - 1); a slot outside the cache, or named by an
 * earlier entry of the same call, gets SV_ST_BAD_SEQ.  A refused entry
 * changes nothing; status (int32 [batch] or NULL) says why, 0 where the entry
 * was carried out.  What a call does depends on the state and the arguments
 * alone: the lowest free pages are taken first, entry by entry.
 *
 * spec_verify_cache_reserve: entry b grows by num_new[b] >= 0 tokens, packed
 * total_new = sum num_new <= 524288 (otherwise SV_ST_BAD_LAYOUT for every
 * entry, nothing changes).  start[b] is its old length (-1: refused), slots
 * (int64 [total_new]) the place of each new token, page * page_size + offset
 * (-1: refused).  A partly filled last page that other sequences use too is
 * first copied to a page of its own, in every layer.  Users and free pages are
 * counted as they were before the call: where all users of such a page append
 * in one call, each gets a copy, one page more than they need, and the old page
 * is free afterwards.  SV_ST_BAD_LENGTH: the table row would be too short;
 * SV_ST_CACHE_FULL: too few free pages (so are the entries behind it that need
 * any).
 * spec_verify_cache_truncate: entry b loses its last drop[b] tokens, or all
 * of them with drop == NULL; pages that hold none of its tokens any more
 * lose it as a user.  SV_ST_BAD_LENGTH: drop outside 0 .. length.
 * spec_verify_cache_commit: entry b, which reserved num_draft[b] + 1 tokens,
 * keeps accepted_len[b] + 1 of them (its last emitted token and the accepted
 * drafts; the token the verify call drew is the next round's first), or none
 * for accepted_len[b] = -1 (not verified).  It takes the entry's word that
 * these tokens are there: an entry whose reserve was refused has grown by
 * none, and would lose older ones.
 * spec_verify_cache_commit_reserved: the same with reserve's start, [batch];
 * an entry that reserve refused (-1), or whose length is not start[b] +
 * num_draft[b] + 1, keeps what it has: SV_ST_BAD_LENGTH.
 * spec_verify_cache_fork: slot children[b], of length 0, gets the length and
 * pages of slot parents[b] (which may be named more than once), as they were
 * before the call.  SV_ST_BAD_LENGTH: the child is not empty.
 * spec_verify_cache_compact: the pages in use move, in order, to the front of
 * the pool: afterwards pages 0 .. live - 1 are in use and the others free;
 * live is int32 [1] or NULL.  Places handed out before are void.
 * spec_verify_cache_write: row r of k_new and v_new, [rows][kv_heads]
 * [head_dim] with strides in elements (multiples of 8, 16-byte aligned), goes
 * to slots[r] of a layer; places outside the pool (-1) are left out, and no
 * place may be named twice.
 *
 * All enqueue one or two kernels on `hip_stream`, which belongs to the
 * calling thread's current device, allocate nothing and do not synchronise;
 * SV_ERR_INVALID (nothing enqueued) for sizes outside their range or a
 * missing or misaligned buffer; batch 0 and rows 0 are no-ops. */
#define SV_CACHE_MAX_SLOTS 4096
typedef struct spec_verify_cache {
  int32_t slots;
  int32_t max_pages;
  int32_t page_size;
  int32_t num_pages;
  int32_t layers;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t* page_table;
  int32_t* seq_len;
  int32_t* refcount;
  void* k;
  void* v;
  void* workspace;
  int64_t workspace_bytes;
} spec_verify_cache;
int spec_verify_cache_reserve(const spec_verify_cache* cache, int32_t batch, const int32_t* seqs, const int32_t* num_new,
                              int64_t total_new, int32_t* start, int64_t* slots, int32_t* status, void* hip_stream);
int spec_verify_cache_truncate(const spec_verify_cache* cache, int32_t batch, const int32_t* seqs, const int32_t* drop,
                               int32_t* status, void* hip_stream);
int spec_verify_cache_commit(const spec_verify_cache* cache, int32_t batch, const int32_t* seqs, const int32_t* num_draft,
                             const int32_t* accepted_len, int32_t* status, void* hip_stream);
int spec_verify_cache_commit_reserved(const spec_verify_cache* cache, int32_t batch, const int32_t* seqs,
                                      const int32_t* num_draft, const int32_t* accepted_len, const int32_t* start,
                                      int32_t* status, void* hip_stream);
int spec_verify_cache_fork(const spec_verify_cache* cache, int32_t batch, const int32_t* parents, const int32_t* children,
                           int32_t* status, void* hip_stream);
int spec_verify_cache_compact(const spec_verify_cache* cache, int32_t* live, void* hip_stream);
int spec_verify_cache_write(const spec_verify_cache* cache, int32_t layer, int64_t rows, const void* k_new,
                            int64_t k_row_stride, int64_t k_head_stride, const void* v_new, int64_t v_row_stride,
                            int64_t v_head_stride, const int64_t* slots, void* hip_stream);

/* Bytes of workspace for a cache with these sizes (its pointers are not
 * looked at), or SV_ERR_INVALID. */
int64_t spec_verify_cache_workspace(const spec_verify_cache* cache);

/* sizeof(spec_verify_cache) as compiled into the library. */
int64_t spec_verify_cache_size(void);

/* ---- a cache held in 8 bits ----------------------------------------------------
 * The same paged cache with k and v as 8-bit codes, half the bytes to keep and
 * to read.  A vector (one token's key or value of one head) is head_dim codes
 * and one float32 scale, x ~ scale * code:
 *   SV_CODES_E4M3  8-bit floating point (4 exponent, 3 mantissa bits, largest
 *                  448); the scale is the smallest power of two under which no
 *                  element is above 448, the code x / scale to nearest even
 *   SV_CODES_INT8  scale = max |x| / 127, code = round(x * (127 / max |x|))
 * both in float32.  A vector whose largest magnitude is below 2^-100 is held as
 * 0, one that is not finite as NaN.
 *   k, v of spec_verify_cache  [layers][num_pages][kv_heads][page_size][head_dim] codes
 *   k_scale, v_scale           [layers][num_pages][kv_heads][page_size] float, 16-byte aligned
 *   dtype                      SV_BF16 or SV_F16: what is written and read back
 * head_dim is a multiple of 16, at most 512.  spec_verify_cache_truncate,
 * _commit, _commit_reserved and _fork touch no page and serve both kinds; the
 * calls that do take the codes as well, with codes = NULL for a 16-bit cache:
 *
 * spec_verify_coded_cache_reserve, _compact: as without; reserve also gives
 * positions, int32 [total_new] or NULL: each new token's place in its sequence
 * (-1: refused).
 * spec_verify_coded_cache_write: as spec_verify_cache_write, rows of the 16-bit
 * type, held as codes (codes is required).
 * spec_verify_cache_read: tokens first[b] .. first[b] + count[b] - 1 of each
 * sequence's keys and values in a layer, packed [total][kv_heads][head_dim] of
 * the 16-bit type `dtype` (codes times scale, rounded, at most its largest
 * finite value), k_out and v_out 16-byte aligned.  total = sum count <= 524288,
 * batch <= 4096, seqs (or NULL) may name a slot twice.  status (int32 [batch]
 * or NULL): SV_ST_BAD_LAYOUT (counts that do not add up: for every entry, all
 * rows are NaN), SV_ST_BAD_SEQ, SV_ST_BAD_LENGTH (tokens the sequence does not
 * have): the entry's rows are NaN; SV_ST_BAD_PAGE: those of the page are.
 *
 * Streams, errors and no-ops as for the paged cache. */
enum { SV_CODES_NONE = 0, SV_CODES_E4M3 = 1, SV_CODES_INT8 = 2 };
typedef struct spec_verify_codes {
  int32_t codes;               /* SV_CODES_E4M3 or SV_CODES_INT8 */
  int32_t dtype;
  float* k_scale;
  float* v_scale;
} spec_verify_codes;
int spec_verify_coded_cache_reserve(const spec_verify_cache* cache, const spec_verify_codes* codes, int32_t batch,
                                    const int32_t* seqs, const int32_t* num_new, int64_t total_new, int32_t* start,
                                    int64_t* slots, int32_t* positions, int32_t* status, void* hip_stream);
int spec_verify_coded_cache_compact(const spec_verify_cache* cache, const spec_verify_codes* codes, int32_t* live,
                                    void* hip_stream);
int spec_verify_coded_cache_write(const spec_verify_cache* cache, const spec_verify_codes* codes, int32_t layer, int64_t rows,
                                  const void* k_new, int64_t k_row_stride, int64_t k_head_stride, const void* v_new,
                                  int64_t v_row_stride, int64_t v_head_stride, const int64_t* slots, void* hip_stream);
int spec_verify_cache_read(const spec_verify_cache* cache, const spec_verify_codes* codes, int32_t dtype, int32_t layer,
                           int32_t batch, const int32_t* seqs, const int32_t* first, const int32_t* count, int64_t total,
                           void* k_out, void* v_out, int32_t* status, void* hip_stream);

/* sizeof(spec_verify_codes) as compiled into the library. */
int64_t spec_verify_codes_size(void);

/* ---- attention over a cache held in 8 bits, and over shared prefixes --------------
 * spec_verify_paged_attention with more than its own arguments say: options
 * (NULL, or all zero: the call as it is).
 *   codes     SV_CODES_E4M3 or SV_CODES_INT8: k and v of args are codes, their
 *             strides count codes (multiples of 16); dtype is that of q and out
 *   k_scale, v_scale   float, strides in elements for page and head (multiples
 *             of 4), neighbouring tokens side by side, 16-byte aligned
 * Scores are products of q and the codes, times the key's scale; the weights
 * take the value's scale on before they are split in two bfloat16 (also for
 * SV_F16: held to 2^-16 of themselves).  A scale or code that is not a number,
 * or an infinite scale of a value, makes the rows that see it NaN whatever its
 * weight, and no others; an infinite scale of a key makes its scores infinite.
 *   num_groups   0, or the number (at most batch) of groups of neighbouring sequences
 *             whose first tokens are the same (forks of one sequence, for instance)
 *   groups    [num_groups + 1] int32: group g is the sequences groups[g] ..
 *             groups[g + 1] - 1, together 0 .. batch - 1 (a group may be empty)
 *   prefix_len   [num_groups] int32: how many tokens its sequences share (0:
 *             none); the new tokens are behind them
 * The keys of a prefix are read once for all rows of its group, from the pages
 * of the group's first sequence.  The result is that of the call without groups
 * up to float32 roundings.  Pages that a prefix fills have to be the same pages in
 * every page table of the group (a partly filled last one may be a copy): other
 * ones set SV_ST_BAD_PAGE.  A prefix that a sequence does not have in front of
 * its new tokens sets SV_ST_BAD_LENGTH for it; one that the group's first
 * sequence does not have refuses the group.  Groups that do not add up set
 * SV_ST_BAD_LAYOUT for every sequence.  Refused sequences' rows are NaN.  With
 * groups window is 0, and up to four kernels are enqueued instead of two.
 * workspace: spec_verify_attention_options_workspace() bytes. */
typedef struct spec_verify_attention_options {
  int32_t codes;
  const float* k_scale;
  int64_t k_scale_page_stride;
  int64_t k_scale_head_stride;
  const float* v_scale;
  int64_t v_scale_page_stride;
  int64_t v_scale_head_stride;
  int32_t num_groups;
  const int32_t* groups;
  const int32_t* prefix_len;
} spec_verify_attention_options;
int spec_verify_paged_attention_options(const spec_verify_attention_args* args, const spec_verify_attention_options* options,
                                        void* hip_stream);

/* Bytes of workspace for a call with these sizes (pointers, strides and tables
 * are not looked at), or SV_ERR_INVALID. */
int64_t spec_verify_attention_options_workspace(const spec_verify_attention_args* args,
                                                const spec_verify_attention_options* options);

/* sizeof(spec_verify_attention_options) as compiled into the library. */
int64_t spec_verify_attention_options_size(void);

/* ---- norms and position rotation of queries and keys ---------------------------
 * What a layer does to its projections' rows before it attends, in one pass.
 * For each head's vector x of row r, a token at positions[r]:
 *   y = x / sqrt(mean(x^2) + eps) * weight      (y = x where the weight is NULL)
 *   pair i of rotary / 2: (a, b) -> (a cos t - b sin t, b cos t + a sin t)
 *   with t = positions[r] * inv_freq[i], the pair (y_i, y_{i + rotary/2}) or,
 *   interleaved, (y_2i, y_2i+1); numbers from rotary on stay y
 * in float32 (angles in float64), rounded once.
 *   q, k           [rows][heads], [rows][kv_heads][head_dim] of dtype SV_BF16 or
 *                  SV_F16, strides in elements for row and head
 *   positions      [rows] int32; a row with a negative one is left out: NaN in
 *                  q_out and k_out, nothing in the cache
 *   inv_freq       [rotary / 2] double, radians for each position
 *   q_weight, k_weight   [head_dim] of weight_dtype (dtype, or SV_F32), each
 *                  may be NULL
 *   q_out          [rows][heads][head_dim], contiguous
 * Without a cache, k_out is [rows][kv_heads][head_dim], contiguous, and v and
 * slots are NULL.  With one, the keys go to the places slots[r] (int64, from
 * reserve) of `layer` instead, with them v ([rows][kv_heads][head_dim], as it
 * is), and k_out is NULL; codes as for spec_verify_coded_cache_write (keys are
 * held straight from float32); places outside the pool are left out, none may
 * be named twice.
 * head_dim a multiple of 16, at most 512; rotary a multiple of 16 from 0 to
 * head_dim; rows <= 524288; heads >= 1, kv_heads >= 1, together at most 4096;
 * eps >= 0; q, k, v, weights and outputs 16-byte aligned, strides in multiples
 * of 8 elements.  Outputs must not overlap inputs.
 * Enqueues one kernel on `hip_stream`, which belongs to the calling thread's
 * current device; allocates nothing, does not synchronise.  SV_ERR_INVALID:
 * nothing was enqueued.  rows == 0 is a no-op. */
typedef struct spec_verify_rope_args {
  int64_t rows;
  int32_t heads;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t rotary;
  int32_t interleaved;
  int32_t dtype;
  int32_t weight_dtype;
  int32_t layer;
  double eps;
  const void* q;
  int64_t q_row_stride;
  int64_t q_head_stride;
  const void* k;
  int64_t k_row_stride;
  int64_t k_head_stride;
  const void* v;
  int64_t v_row_stride;
  int64_t v_head_stride;
  const int32_t* positions;
  const double* inv_freq;
  const void* q_weight;
  const void* k_weight;
  void* q_out;
  void* k_out;
  const int64_t* slots;
} spec_verify_rope_args;
int spec_verify_qk_norm_rope(const spec_verify_rope_args* args, const spec_verify_cache* cache,
                             const spec_verify_codes* codes, void* hip_stream);

/* sizeof(spec_verify_rope_args) as compiled into the library. */
int64_t spec_verify_rope_args_size(void);

/* Library version string. */
const char* spec_verify_version(void);

/* sizeof(spec_verify_args) as compiled into the library, so that a binding
 * can check its own copy of the struct layout. */
int64_t spec_verify_args_size(void);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */

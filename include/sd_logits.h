/*
 * sd_logits.h — C ABI of the logit operators around the verify step.
 *
 * Before a round is verified, a serving loop changes the target's and the
 * drafter's logit rows: penalties for tokens that the text already holds,
 * per-request biases, a grammar's mask (sd_process_logits, with the counts
 * that sd_token_counts and sd_token_counts_add keep).  After it, the
 * target's rows are what the drafter learns from: their top logits
 * (sd_top_logits), the distillation loss over them and its gradient
 * (sd_distill).
 *
 * Conventions are those of sd_verify.h: every call is stream-ordered and
 * asynchronous, checks its arguments on the host, allocates nothing and keeps
 * no pointer; pointers are device pointers owned by the caller unless marked
 * "host"; data errors set bits in the optional *status word.  Row strides are
 * in elements; rows need no alignment beyond their element's.
 */
#ifndef SD_LOGITS_H_
#define SD_LOGITS_H_

#include "sd_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bit of *status. */
#define SD_STATUS_BAD_PENALTY 0x8u /* a repetition penalty that is not positive
                                      and finite, or a presence or frequency
                                      penalty that is not finite             */

#define SD_MAX_TOP 128  /* top logits kept per row                           */
#define SD_MAX_BIAS 1024 /* bias entries per sequence                        */

/*
 * Token counts of each sequence, the state that the penalties read:
 * counts [B][V], 16 bits per token id.  Bits 0..14: how often the id occurs
 * in history[b][prompt_lengths[b] .. lengths[b]), at most 32767; bit 15: it
 * occurs in history[b][0 .. prompt_lengths[b]).  history [B][L] int32 and
 * lengths [B] as in sd_ngram_draft (lengths clamped to [0, L]);
 * prompt_lengths [B] optional (null: no prompt), clamped to [0, length].
 * Every count is written.  Tokens outside [0, V) are not counted and set
 * SD_STATUS_BAD_TOKEN.
 */
sd_status_t sd_token_counts(int32_t B, int32_t L, int32_t V, const int32_t *history,
                            const int32_t *lengths, const int32_t *prompt_lengths,
                            uint16_t *counts, int32_t *status, void *stream);

/*
 * Adds a round's tokens to the counts: tokens[b][0 .. n[b]) of tokens [B][M]
 * (out_tokens and tau of sd_verify: M = K + 1; n clamped to [0, M]).  Counts
 * stay at most 32767; bit 15 is left as it is.  Tokens outside [0, V) are
 * not counted and set SD_STATUS_BAD_TOKEN.
 */
sd_status_t sd_token_counts_add(int32_t B, int32_t M, int32_t V, const int32_t *tokens,
                                const int32_t *n, uint16_t *counts, int32_t *status,
                                void *stream);

/*
 * Penalties, biases and masks on logits.  For row r of sequence b and token
 * v with logit x:
 *   c    = count of v in counts[b] + #{ i < base + r : prev[b][i] = v }
 *   seen = c > 0 or v's prompt bit is set
 *   x1   = seen ? (x > 0 ? x / repetition[b] : x * repetition[b]) : x
 *   x2   = x1 - frequency[b] c - presence[b] [c > 0]
 *   x3   = x2 + the sum of the bias_vals[b][i] with bias_ids[b][i] = v (in list order)
 *   y    = v allowed by the mask ? x3 : -inf
 * A logit of -inf stays -inf.  All in fp32, rounded once to the logits' type.
 * prev are the tokens drafted in this round: row r of the target's rows
 * [B][K+1][V] (base = 0) must count the drafts before position r, as the
 * drafter did when it drew draft r.  Null arrays are neutral (no counts, a
 * repetition penalty of 1, others of 0, no bias, every token allowed).
 * bias_ids: -1 marks an empty slot.  mask: bit v % 32 of word v / 32 of a
 * row of ceil(V / 32) words is set where v is allowed; bits from V on are
 * ignored; a mask stride may be 0 (rows share a mask).  A row whose mask
 * allows nothing comes out as only -inf.  A bad penalty of a sequence
 * (SD_STATUS_BAD_PENALTY) makes all of its rows NaN.  Ids outside [0, V) in
 * prev or bias_ids (other than -1 there) are ignored and set
 * SD_STATUS_BAD_TOKEN.  out may be logits itself (the same pointer and
 * strides: places that do not change are then not written); otherwise the
 * two must not overlap.
 */
typedef struct sd_process_args {
  int32_t B, R, V;            /* sequences, rows of each, vocabulary size     */
  int32_t dtype;              /* sd_dtype_t                                   */
  const void *logits;         /* [B][R][V]                                    */
  int64_t logits_sb, logits_sr; /* strides of a sequence and of a row         */
  void *out;                  /* [B][R][V]                                    */
  int64_t out_sb, out_sr;
  const uint16_t *counts;     /* [B][V] or null                               */
  const int32_t *prev;        /* [B][P] or null                               */
  int32_t P, base;            /* 0 <= base, base + R - 1 <= P <= SD_MAX_K where
                                 prev is given                                */
  const float *repetition;    /* [B] or null                                  */
  const float *presence;      /* [B] or null                                  */
  const float *frequency;     /* [B] or null                                  */
  const int32_t *bias_ids;    /* [B][n_bias] or null                          */
  const float *bias_vals;     /* [B][n_bias]                                  */
  int32_t n_bias;             /* at most SD_MAX_BIAS                          */
  const int32_t *mask;        /* [B][R][ceil(V / 32)] or null                 */
  int64_t mask_sb, mask_sr;   /* strides in words, may be 0                   */
  int32_t *status;            /* one int32 or null                            */
} sd_process_args;

sd_status_t sd_process_logits(const sd_process_args *args, void *stream);

/*
 * The top logits of each row of logits [N][V] (row stride `stride`): ids
 * [N][k] and vals [N][k] are the k largest, larger first, ties to the lowest
 * index; -inf and NaN are never chosen, and slots left over hold -1 and
 * -inf.  rest [N] (optional) is log sum exp(x / T) over the places not
 * chosen (-inf where that sum is zero, NaN where one of them is NaN or
 * +inf): the teacher's mass beside its top logits, as sd_distill takes it.
 * 1 <= k <= SD_MAX_TOP; T (host) positive and finite.
 */
sd_status_t sd_top_logits(int32_t N, int32_t V, int32_t dtype, const void *logits,
                          int64_t stride, int32_t k, float T, float *vals, int32_t *ids,
                          float *rest, void *stream);

/*
 * Distillation from a teacher's top logits, over the k named tokens of a row
 * and one bucket that holds all others:
 *   p_i  = exp(t_i / T) / Zt, p_r = exp(rest) / Zt,
 *          Zt = sum_i exp(t_i / T) + exp(rest)   (rest null: p_r = 0)
 *   q    = softmax(s / T), q_r = the sum of q over the others
 *   loss = w [ sum_i p_i log(p_i / q_i) + p_r log(p_r / q_r) ]
 *   grad = w / T (q_j - p_j)                 for a named token j
 *          w / T (q_j - p_r q_j / q_r)       for the others
 * student [N][V] (row stride student_s), ids [N][k] distinct (-1 marks an
 * empty slot), vals [N][k] and rest [N] as sd_top_logits writes them, weight
 * [N] optional (the gradient that reaches each row's loss; 1 without it).
 * loss [N] and grad [N][V] are optional, one of them is required; grad may
 * be student itself (same pointer and stride), otherwise they must not
 * overlap.  A row of weight 0 is not read: its loss and gradient are 0.  So
 * are those of a row whose teacher names nothing and has no rest (a teacher
 * row of only -inf), and of a row with an id outside [0, V) (other than -1)
 * or named twice, which also sets SD_STATUS_BAD_TOKEN.  Sums and the
 * softmax are in fp32; the gradient is rounded once to the student's type.
 * 0 <= k <= SD_MAX_TOP; T (host) positive and finite.
 */
typedef struct sd_distill_args {
  int32_t N, V, k;
  int32_t dtype;              /* sd_dtype_t of student and grad               */
  const void *student;        /* [N][V]                                       */
  int64_t student_s;
  const int32_t *ids;         /* [N][k]                                       */
  const float *vals;          /* [N][k]                                       */
  const float *rest;          /* [N] or null                                  */
  const float *weight;        /* [N] or null                                  */
  float T;
  float *loss;                /* [N] or null                                  */
  void *grad;                 /* [N][V] or null                               */
  int64_t grad_s;
  int32_t *status;            /* one int32 or null                            */
} sd_distill_args;

sd_status_t sd_distill(const sd_distill_args *args, void *stream);

/* Sizes of the argument structs as compiled into the library. */
size_t sd_process_args_size(void);
size_t sd_distill_args_size(void);

#ifdef __cplusplus
}
#endif

#endif /* SD_LOGITS_H_ */

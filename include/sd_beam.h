/*
 * sd_beam.h — C ABI of beam search's step on the GPU: the selection of the
 * next beams over beams and vocabulary, and the reordering of what a loop
 * keeps per beam (texts, token counts, contiguous caches).  Paged caches
 * follow the same parents: sd_kv_fork of sd_kv.h.
 *
 * Conventions are those of sd_verify.h and sd_logits.h: every call is
 * stream-ordered and asynchronous, checks its arguments on the host,
 * allocates nothing and keeps no pointer; pointers are device pointers owned
 * by the caller unless marked "host"; data errors set bits in the optional
 * *status word.
 */
#ifndef SD_BEAM_H_
#define SD_BEAM_H_

#include "sd_kv.h"
#include "sd_logits.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SD_MAX_BEAMS 32   /* beams per sequence                               */
#define SD_MAX_STATES 16  /* tensors of one sd_beam_reorder call              */

/*
 * The k best continuations of each sequence's W beams.  A live beam w with
 * logits x and score s offers every token v of finite logit:
 *   c(w, v) = s + x[v] / T - log sum_u exp(x[u] / T)
 * a finished beam (finished[b][w] != 0) offers itself as (w, eos) with c = s,
 * and its logits are not read.  Candidates are ranked by c / norm[b][w]
 * (c without norm), larger first, ties to the lowest w V + v.  Outputs, all
 * [B][k]: scores = c (fp32; not divided), parents = w, tokens = v, ended = 1
 * where the beam was finished or v == eos (eos = -1: no token ends a beam).
 * Slots left over hold -inf, -1, -1, 0.  Scores, their differences and the
 * ranking are in 64 bits, the sums of exponentials in fp32 per piece of a row
 * (up to 4 KB) and in whole units of 2^-31 above that.
 *   A beam offers nothing where its score is -inf (a dead beam), where its
 * row holds only -inf, where its row holds a NaN or +inf or its score is NaN
 * or +inf (SD_STATUS_NONFINITE), or where its norm is not positive and finite
 * (SD_STATUS_BAD_PENALTY).
 * 1 <= W <= SD_MAX_BEAMS, 1 <= k <= SD_MAX_TOP; T (host) positive, normal and
 * finite.
 * workspace: at least sd_beam_select_workspace_size bytes, 16-byte aligned;
 * nothing in it needs clearing, and calls that share it must not overlap on
 * the GPU.
 */
typedef struct sd_beam_select_args {
  int32_t B, W, V, k;
  int32_t dtype;              /* sd_dtype_t                                   */
  const void *logits;         /* [B][W][V]                                    */
  int64_t logits_sb, logits_sw; /* strides of a sequence and of a beam, elements */
  const float *scores;        /* [B][W]                                       */
  const uint8_t *finished;    /* [B][W] or null                               */
  const float *norm;          /* [B][W] or null                               */
  int32_t eos;                /* -1: none; required where finished is given   */
  float T;
  float *out_scores;          /* [B][k]                                       */
  int32_t *parents;           /* [B][k]                                       */
  int32_t *tokens;            /* [B][k]                                       */
  uint8_t *ended;             /* [B][k] or null                               */
  int32_t *status;            /* one int32 or null                            */
  void *workspace;
  size_t workspace_bytes;
} sd_beam_select_args;

/* 0 for arguments out of range. */
size_t sd_beam_select_workspace_size(int32_t B, int32_t W, int32_t V, int32_t dtype);

sd_status_t sd_beam_select(const sd_beam_select_args *args, void *stream);

/*
 * Rows reordered by their parents, for up to SD_MAX_STATES states at once:
 *   out[b][i] = in[b][parents[b][i]]   for i < k
 * parents [B][k] as sd_beam_select writes them; -1 (and, with
 * SD_STATUS_BAD_PARENT, anything outside [0, W)) stands for i itself, which
 * must then be a row (a slot i >= W is left as it is).  Rows are row_bytes
 * contiguous bytes of any type, at any strides (in bytes).  out may be in
 * itself with the same strides and k = W; rows whose parent they are
 * themselves are then not touched.  Otherwise the two must not overlap.
 */
typedef struct sd_beam_state {
  const void *in;             /* [B][W] rows                                  */
  int64_t in_sb, in_sw;
  void *out;                  /* [B][k] rows                                  */
  int64_t out_sb, out_sw;
  int64_t row_bytes;
} sd_beam_state;

sd_status_t sd_beam_reorder(int32_t B, int32_t W, int32_t k, const int32_t *parents,
                            int32_t n_states, const sd_beam_state *states /* host */,
                            int32_t *status, void *stream);

/* Sizes of the argument structs as compiled into the library. */
size_t sd_beam_select_args_size(void);
size_t sd_beam_state_size(void);

#ifdef __cplusplus
}
#endif

#endif /* SD_BEAM_H_ */

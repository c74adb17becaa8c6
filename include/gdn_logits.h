/*
 * gdn_logits.h -- C ABI of the rules between the target's logits and the acceptance of a
 * draft, on MI355X (gfx950): penalties for repeated tokens, biases, grammar masks, and the
 * probabilities at a temperature.
 *
 * The target gives one row of logits after every node of a draft.  gdn_adjust_logits applies
 * a slot's rules to every row, each with the tokens on its own path counted in, and gives
 * the logits (what greedy acceptance takes) or the probabilities (what sampled acceptance
 * takes as `target` in gdn_draft_accept).  The row of the committed prefix (`root`) is the
 * same call with one node per lane and no tokens, as is a plain decode step.
 *
 * Conventions are those of gdn_round.h; lanes may share a slot.  Notation: C lanes, N nodes
 * per lane, P slots, V tokens of vocabulary, s = slot_ids[c], path(i) = node i and its
 * ancestors.
 */
#ifndef GDN_LOGITS_H
#define GDN_LOGITS_H

#include "gdn_round.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A device status bit, next to those of gdn_verify.h and gdn_round.h. */
#define GDN_STATUS_RULE 512 /* repetition outside [2^-126, 2^126] (it and its reciprocal are
                               normal numbers there), a presence, frequency or temperature
                               that is not finite, or a temperature below 0                 */

/* Shape errors (GDN_ERR_SHAPE): a non-positive n_seqs, n_nodes, n_slots or vocab, a negative
   max_history or max_bias, an unknown dtype.  GDN_ERR_UNSUPPORTED: C > GDN_MAX_SEQS,
   N > GDN_MAX_NODES, V > 2^24, max_history > 2^20, max_bias > 1024, P * max_history or
   P * max_bias above 2^30, out_dtype neither dtype nor GDN_DTYPE_F32. */
typedef struct gdn_logits_shape {
    int32_t n_seqs;      /* C                                                   */
    int32_t n_nodes;     /* N rows per lane                                     */
    int32_t n_slots;     /* P                                                   */
    int32_t vocab;       /* V                                                   */
    int32_t max_history; /* entries of a slot's history                         */
    int32_t max_bias;    /* entries of a slot's bias list                       */
    int32_t dtype;       /* GDN_DTYPE_* of logits                               */
    int32_t out_dtype;   /* of out: dtype, or GDN_DTYPE_F32                     */
} gdn_logits_shape;

/* The rules of every slot; any pointer may be NULL. */
typedef struct gdn_logit_rules {
    const int32_t *history;     /* [P][max_history] token ids; those outside [0, V) count nowhere */
    const int32_t *history_len; /* [P] entries in use; needed with history (GDN_ERR_NULL)         */
    const int32_t *prompt_len;  /* [P] the first entries that are the prompt's; NULL: none        */
    const float *repetition;    /* [P] r in [2^-126, 2^126]; NULL: 1 */
    const float *presence;      /* [P] p; NULL: 0 */
    const float *frequency;     /* [P] f; NULL: 0 */
    const int32_t *bias_tokens; /* [P][max_bias] token ids; those outside [0, V) are skipped      */
    const float *bias;          /* [P][max_bias]; both or neither (GDN_ERR_NULL)                  */
    const float *temperature;   /* [P] T >= 0; NULL: out is the logits                            */
} gdn_logit_rules;

/*
 * For every present node i of a valid lane and every token x, in float32:
 *   z = logits[c][i][x] + the sum of s's biases of x, in the list's order
 *   z = z > 0 ? z * (1 / r) : z * r  where x is in s's history or on path(i)
 *   z = z - f n - p [n > 0]        n = occurrences of x in the history behind the prompt, and
 *                                  on path(i)
 *   z = -infinity                  where the mask's bit of x is 0, whatever the rest is
 * with 1 / r rounded to float32: such a z may be one step beside z / r, and equal to another
 * token's, or not, where that would be otherwise.
 * Without a temperature out[c][i][x] = z.  With T = temperature[s] > 0
 *   out[c][i][x] = e^{(z(x) - max z) / T} / sum_y e^{(z(y) - max z) / T}
 * (a z of +infinity counts e^0, a NaN makes its row NaN), and with T = 0 it is 1 at the
 * largest z (the lowest index of equal ones; NaN below all) and 0 elsewhere.  A row without
 * any z above -infinity gives zeros.
 *
 *   logits      row of node (c, i) at logits + (c*N + i) * row_stride, V values  (read)
 *   row_stride  >= V, in values (GDN_ERR_SHAPE)
 *   mask        [C][N][ceil(V / 32)] int32: bit x % 32 of word x / 32 is 1 where x is
 *               allowed; NULL: all are                                         (read)
 *   tokens      [C][N] the nodes' tokens; NULL: no token is on any path  (read)
 *   parents     [C][N], or NULL: a chain    lane_nodes [C], or NULL      (read)
 *   slot_ids    [C], -1 = padding lane      (read)
 *   out         [C][N][V] of out_dtype, written for present nodes of valid lanes
 *   workspace   at least gdn_adjust_logits_workspace_size(sh) bytes, 16-byte aligned, with a
 *               temperature; contents on entry do not matter; calls that overlap in time must
 *               not share it
 *   status      may be NULL; SLOT_RANGE / NODES / PARENT / TOKEN / RULE, and LENGTH: a
 *               history_len outside [0, max_history] or a prompt_len outside [0, history_len]
 * logits and out need the alignment of their type only, so V may be odd; every other buffer
 * 4 bytes.
 */
int gdn_adjust_logits(const gdn_logits_shape *sh, const void *logits, int64_t row_stride, const gdn_logit_rules *rules,
                      const int32_t *mask, const int32_t *tokens, const int32_t *parents, const int32_t *lane_nodes,
                      const int32_t *slot_ids, void *out, void *workspace, size_t workspace_bytes, int32_t *status,
                      hipStream_t stream);

/* Bytes of workspace gdn_adjust_logits needs for this shape where there is a temperature; 0
   for an invalid shape. */
size_t gdn_adjust_logits_workspace_size(const gdn_logits_shape *sh);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LOGITS_H */

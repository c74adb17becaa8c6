/*
 * gdn_round.h -- C ABI of what surrounds the recurrence in a speculative round on MI355X
 * (gfx950): the attention layers of a hybrid model and the acceptance of the draft.
 *
 * A hybrid model alternates gated delta rule layers (gdn_verify.h) with softmax attention
 * layers over a paged key/value cache.  One round of an attention layer, on the caller's
 * stream, is
 *
 *   gdn_rope_kv_write    rotary positions (with an optional norm) of the round's q and k; k
 *                        and v written into the slot's pages behind its committed rows;
 *   gdn_paged_attention  attention of the round's tokens over the committed rows and over
 *                        their own ancestors in the draft tree (a prompt chunk or plain
 *                        decode: over the chain so far), with an optional output gate;
 *
 * and once per round, after the last layer,
 *
 *   gdn_draft_accept     tests the drafted tokens against the target's probabilities with
 *                        given random numbers (or greedily): the accepted node of every
 *                        lane, which gdn_replay_commit_layers takes, and the next token;
 *   gdn_kv_commit_layers moves the accepted path's cache rows together in every attention
 *                        layer and gives the new lengths.
 *
 * A plain decode step is the same calls with one token per lane and no tree, a prompt chunk
 * with up to GDN_MAX_CHAIN tokens per lane; gdn_kv_commit_layers then only advances lengths.
 *
 * Conventions are those of gdn_verify.h (host validation before anything is enqueued, error
 * codes, padding lanes with slot -1, ragged lanes through lane_nodes, device status bits,
 * caller-owned memory, no allocation, no state between calls), and
 *   - values are float32, bfloat16 or float16 by gdn_attn_shape.dtype (GDN_DTYPE_*); dense
 *     value buffers are 16-byte aligned, int32 buffers 4-byte, inv_freq 8-byte aligned;
 *   - softmax statistics, norms and products are held in 32 bits, angles and the acceptance
 *     tests in 64; a 16-bit path rounds the softmax weights to its type before the product
 *     with v (half a step each; in float16 at least 2^-34 of a row's largest weight), and every
 *     output once;
 *   - lanes of one call use different slots (SLOT_DUP in the calls that write a cache);
 *   - pages that hold rows at or behind a slot's committed length belong to that slot alone
 *     (full pages in front of it may be shared between slots).
 *
 * Notation: C lanes, N new tokens (nodes) per lane, N_c the present ones of lane c, P slots,
 * s = slot_ids[c], L = seq_len[s] committed rows, G = H_q / H_kv query heads per kv head
 * (query head h reads kv head h / G), D = head_dim.  Node i's key and value are row L + i of
 * the slot's cache; row t of slot s lies in page page_table[s][t / page_size] at place
 * t % page_size.
 */
#ifndef GDN_ROUND_H
#define GDN_ROUND_H

#include "gdn_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_DTYPE_F32 0
#define GDN_DTYPE_BF16 1
#define GDN_DTYPE_F16 2

/* Device status bits, next to those of gdn_verify.h. */
#define GDN_STATUS_LENGTH 32 /* seq_len[s] < 0, or L + N_c above max_pages * page_size        */
#define GDN_STATUS_PAGE 64   /* a page id outside [0, n_pages) at a row that the call uses    */
#define GDN_STATUS_TOKEN 128 /* a drafted token outside [0, vocab)                            */
#define GDN_STATUS_AXIS 256  /* pair_axis outside [0, n_axes)                                 */

/* Shape errors (GDN_ERR_SHAPE): a non-positive dimension, H_q % H_kv != 0, an unknown dtype.
   GDN_ERR_UNSUPPORTED: head_dim not 64, 128 or 256; C > GDN_MAX_SEQS; N > GDN_MAX_CHAIN, or
   > GDN_MAX_NODES with parents; H_q > 1024; page_size > 65536; n_pages * H_kv * page_size
   or max_pages * page_size or P * max_pages above 2^30; C * N * H_q above 2^28. */
typedef struct gdn_attn_shape {
    int32_t n_seqs;     /* C                                                      */
    int32_t n_nodes;    /* N new tokens per lane                                  */
    int32_t n_slots;    /* P                                                      */
    int32_t n_q_heads;  /* H_q, a multiple of H_kv                                */
    int32_t n_kv_heads; /* H_kv                                                   */
    int32_t head_dim;   /* D: 64, 128 or 256                                      */
    int32_t page_size;  /* cache rows per page, any number from 1 to 65536        */
    int32_t n_pages;    /* pages of the pool                                      */
    int32_t max_pages;  /* page_table entries per slot                            */
    int32_t dtype;      /* GDN_DTYPE_* of q_out / q, the caches, gate and out     */
} gdn_attn_shape;

/* A [C][N][heads][D] view: value (c, i, h, e) at p[(c*N + i)*token_stride + h*head_stride + e].
   Both strides are non-negative multiples of 16 bytes (GDN_ERR_ALIGN), as is the pointer. */
typedef struct gdn_heads_view {
    const void *p;
    int64_t token_stride; /* in values */
    int64_t head_stride;  /* in values */
} gdn_heads_view;

/* Rotary positions.  Pair j of the first rot_dim values of a head turns by the angle
   positions[c][i][pair_axis[j]] * inv_freq[j] (64-bit); the values behind them are kept. */
typedef struct gdn_rope {
    const double *inv_freq;    /* [rot_dim / 2], device                                       */
    const int32_t *positions;  /* [C][N][n_axes], device; NULL: L + the node's depth (text)   */
    const int32_t *pair_axis;  /* [rot_dim / 2], device; NULL: axis 0                         */
    int32_t n_axes;            /* 1..16 (time, height, width, ...); 1 without positions       */
    int32_t rot_dim;           /* a multiple of 16, 16..D                                     */
    int32_t interleaved;       /* 0: pair j is values (j, j + rot_dim/2); 1: (2j, 2j + 1)     */
    const float *q_norm;       /* [D] weight of an RMS norm of each q head first, or NULL     */
    const float *k_norm;       /* [D] the same for k, or NULL                                 */
    float eps;                 /* x * rsqrt(mean(x^2) + eps) * weight; eps >= 0               */
} gdn_rope;

/*
 * Rotary positions and the cache write.  For every present node i of a valid lane:
 *   q_out[c][i][h] = rot(norm(q[c][i][h]))                     every query head
 *   K row L + i    = rot(norm(k[c][i][h])),  V row L + i = v[c][i][h]   every kv head
 * Rows of the cache behind L are scratch of the round until gdn_kv_commit_layers: the write
 * is not a transaction.  Nothing is written for an offending lane; a row whose page id is
 * outside the pool is left out (PAGE).
 *
 *   x_dtype     GDN_DTYPE_* of q, k, v: that of the shape, or GDN_DTYPE_F32
 *   q, k, v     views with H_q, H_kv, H_kv heads (e.g. of the stacked projection)    (read)
 *   k_cache, v_cache  [n_pages][H_kv][page_size][D]   rows L .. L + N_c - 1 written
 *   slot_ids    [C]              (read)    page_table [P][max_pages]  (read)
 *   seq_len     [P]              (read)    parents [C][N], or NULL: a chain (read)
 *   lane_nodes  [C], or NULL     (read)
 *   q_out       [C][N][H_q][D]   written for present nodes of valid lanes
 *   status      may be NULL; SLOT_RANGE / SLOT_DUP / PARENT / NODES / LENGTH / PAGE / AXIS
 */
int gdn_rope_kv_write(const gdn_attn_shape *sh, int32_t x_dtype, const gdn_heads_view *q, const gdn_heads_view *k,
                      const gdn_heads_view *v, const gdn_rope *rope, void *k_cache, void *v_cache,
                      const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                      const int32_t *parents, const int32_t *lane_nodes, void *q_out, int32_t *status,
                      hipStream_t stream);

/*
 * Attention of the round's tokens over the paged cache.  Node i of lane c attends to the rows
 *   t < L                       the committed rows, and
 *   t = L + j, j an ancestor of i or i itself (parents), or j <= i (parents NULL: a chain):
 *   out[c][i][h] = sum_t softmax_t(scale * q[c][i][h] . K[t][h / G]) V[t][h / G]  (* act(gate))
 * with act = silu (gate_mode 0) or sigmoid (gate_mode 1) as in gdn_prefill.  A row that a
 * node does not attend to contributes nothing, whatever it holds (NaN and infinities
 * included); an infinite or NaN value of an attended row, of a weight above 2^-34 of the
 * largest, makes its column of the output infinite or NaN.  A row in a page outside the pool
 * counts as not attended (PAGE); a node without any attended row of a score above -infinity
 * gets zeros, whatever its gate holds.
 *
 *   q           [C][N][H_q][D]   (read)
 *   k_cache, v_cache  [n_pages][H_kv][page_size][D]   (read); the round's rows are there
 *   slot_ids, page_table, seq_len, parents, lane_nodes   as above (lanes may share a slot)
 *   scale       > 0, and scale * log2(e) finite (GDN_ERR_SHAPE)
 *   gate        view with H_q heads of the shape's dtype, or NULL   (read)
 *   gate_mode   0 or 1 (GDN_ERR_SHAPE)
 *   out         [C][N][H_q][D]   written for present nodes of valid lanes
 *   workspace   at least gdn_paged_attention_workspace_size(sh) bytes, 16-byte aligned (may
 *               be NULL if that is 0); contents on entry do not matter.  Calls that overlap
 *               in time must not share it.
 *   status      may be NULL; SLOT_RANGE / PARENT / NODES / LENGTH / PAGE
 */
int gdn_paged_attention(const gdn_attn_shape *sh, const void *q, const void *k_cache, const void *v_cache,
                        const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                        const int32_t *parents, const int32_t *lane_nodes, float scale, const gdn_heads_view *gate,
                        int32_t gate_mode, void *out, void *workspace, size_t workspace_bytes, int32_t *status,
                        hipStream_t stream);

/* Bytes of workspace gdn_paged_attention needs for this shape: the partial results where the
   cache is split over workgroups (few rows); 0 where it is not, or for an invalid shape. */
size_t gdn_paged_attention_workspace_size(const gdn_attn_shape *sh);

typedef struct gdn_accept_shape {
    int32_t n_seqs;  /* C, 1..GDN_MAX_SEQS                        */
    int32_t n_nodes; /* N drafted nodes per lane, 1..GDN_MAX_NODES */
    int32_t vocab;   /* V, 1..2^24                                */
    int32_t dtype;   /* GDN_DTYPE_* of target, root and draft     */
} gdn_accept_shape;

/*
 * Acceptance of the draft.  p_i = target[c][i] are the target's probabilities after node i,
 * p_-1 = root[c] those after the committed prefix; node i's token tokens[c][i] is tested
 * against the row of its parent.  The walk starts at the prefix; at each place its children
 * are tested in index order, and the first accepted one is entered:
 *   accepted  if  u_accept[c][i] * q * left < p(token)      (evaluated in 64 bits)
 * with q = draft[c][i][token] (the probability that the drafter drew it with) or 1 without
 * draft (candidates), and left = 1 - the sum of p over the refused earlier siblings' tokens;
 * a token that an earlier sibling had is refused.  Without root the lowest child of the
 * prefix is a token already drawn: it is accepted without a test and its siblings refused.
 * Where no child is accepted (or there is none), next_token is drawn by u_next[c]: with
 *   w(x) = max(p(x) - draft[c][i](x), 0)  after node i of a draft was refused,
 *   w(x) = p(x), and 0 at the refused candidates' tokens, otherwise
 * (w = p where that leaves no weight) it is the lowest x whose running sum of w exceeds
 * u_next[c] times the whole sum (never an x of weight 0; -1 if all of p is 0).  Rows are
 * taken as they are given, not renormalised; negative and NaN probabilities count as 0.
 * With u_accept NULL the walk is greedy: a child is accepted if its token is the one of
 * largest p (the lowest of equal ones; NaN below all), and next_token is the largest at the
 * end; p may then be logits.
 *
 *   target     [C][N][V]            rows of present nodes (read)
 *   root       [C][V], or NULL      (read)
 *   draft      [C][N][V], or NULL   the distribution node i's token was drawn from; needs
 *                                   u_accept and a chain (parents NULL): GDN_ERR_UNSUPPORTED
 *   tokens     [C][N]               (read)
 *   parents    [C][N], or NULL: a chain;  lane_nodes [C], or NULL  (read)
 *   slot_ids   [C], or NULL         only a padding lane's -1 is looked at (read)
 *   u_accept   [C][N] in [0, 1), or NULL: greedy;  u_next [C] in [0, 1), with u_accept
 *   accept_node [C]  deepest accepted node, -1 = none     written for valid lanes
 *   n_accept    [C]  accepted nodes                       written for valid lanes
 *   next_token  [C]  -1 where there is no row to draw from (no root, no node)
 *   workspace  at least gdn_draft_accept_workspace_size(sh) bytes, 16-byte aligned; contents
 *              on entry do not matter; calls that overlap in time must not share it
 *   status     may be NULL; PARENT / NODES / TOKEN
 * target, root and draft need the alignment of their type only, so V may be odd.
 */
int gdn_draft_accept(const gdn_accept_shape *sh, const void *target, const void *root, const void *draft,
                     const int32_t *tokens, const int32_t *parents, const int32_t *lane_nodes,
                     const int32_t *slot_ids, const float *u_accept, const float *u_next, int32_t *accept_node,
                     int32_t *n_accept, int32_t *next_token, void *workspace, size_t workspace_bytes,
                     int32_t *status, hipStream_t stream);

/* Bytes of workspace gdn_draft_accept needs for this shape; 0 for an invalid one. */
size_t gdn_draft_accept_workspace_size(const gdn_accept_shape *sh);

/*
 * Commit of the paged caches.  For every lane with e = accept_node[c] >= 0 and the root path
 * a_0 < ... < a_m = e, in every layer and kv head, row L + j <- row L + a_j (j = 0..m, exact
 * copies), and new_len[s] = L + m + 1; every other slot's new_len is its seq_len.  Without
 * parents (a chain) no row moves.  A transaction like gdn_replay_commit: with a bit in
 * *status on entry or from the preflight over all lanes no cache row moves and new_len is
 * seq_len throughout.
 *
 *   n_layers   1..GDN_MAX_LAYERS attention layers; they share the page table
 *   k_caches, v_caches  host arrays of n_layers device pointers, updated in place
 *   slot_ids, page_table, seq_len, parents, lane_nodes, accept_node   (read)
 *   new_len    [P], overlapping nothing else (the caller passes it as seq_len next round)
 *   status     REQUIRED; SLOT_RANGE / SLOT_DUP / PARENT / NODES / ACCEPT / LENGTH / PAGE
 */
int gdn_kv_commit_layers(const gdn_attn_shape *sh, int32_t n_layers, void *const *k_caches, void *const *v_caches,
                         const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                         const int32_t *parents, const int32_t *lane_nodes, const int32_t *accept_node,
                         int32_t *new_len, int32_t *status, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ROUND_H */

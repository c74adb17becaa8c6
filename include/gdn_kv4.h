/*
 * gdn_kv4.h -- C ABI of the attention layers' part of a round over a key/value cache held in
 * 4 bits, on MI355X (gfx950).
 *
 * The calls are those of gdn_round.h for a paged cache whose rows are 4-bit floating point
 * numbers with one power of two for every 32 values: 4.25 bits a value, 0.27 of a 16-bit
 * cache's memory and bytes.  A round over it is
 *
 *   gdn_rope_kv4_write       rotary positions; k and v quantised into the slot's pages;
 *   gdn_paged_attention_kv4  attention of the round's tokens over the cache;
 *   gdn_kv4_commit_layers    the accepted path's rows moved together, every layer;
 *
 * and gdn_kv4_read_layers gives rows of the cache as values (to hand a sequence to a holder
 * of another cache, or to look at it).
 *
 * Format.  Value e of a row is a number of one sign bit, two exponent bits and one fraction
 * bit (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives: codes 0..7, and 8 more) times
 * 2^(scale - 127) with the scale byte of its block e / 32; a block of scale 255 is NaN
 * throughout.  Its code is the nibble e % 2 (0: the lower one) of byte e / 2 of the row.
 *
 * Quantising a block of 32 values x (float32, after norm and rotation): with a the largest
 * |x| and 2^E the power of two of a rounded to one fraction bit (1.75 and above round up to
 * 2, so that no value is off by more than half a step), the scale is 2^e with e = E - 2
 * within [-125, 125], or [-125, 13] in float16 (whose range then holds every value); a code
 * is x / 2^e rounded to nearest, ties to even, and at most 6 in magnitude.  A block of zeros
 * has e = -125.  A block that holds a NaN or an infinity gets scale 255.
 *
 * Conventions and notation are those of gdn_round.h.  gdn_attn_shape.dtype is the type of
 * q, gate, out and of the values that a cache's rows stand for in a call: exact in float32
 * and bfloat16 (scales of up to 252), rounded to it in float16 (exact for scales of
 * 104..140, which are the written ones but for blocks below 2^-21).
 */
#ifndef GDN_KV4_H
#define GDN_KV4_H

#include "gdn_round.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One layer's cache.  Codes are 16-byte aligned, scales D / 32 bytes; no array overlaps another. */
typedef struct gdn_kv4_cache {
    void *k_codes;  /* [n_pages][H_kv][page_size][D / 2]  bytes */
    void *k_scales; /* [n_pages][H_kv][page_size][D / 32] bytes */
    void *v_codes;  /* as k_codes  */
    void *v_scales; /* as k_scales */
} gdn_kv4_cache;

/*
 * Rotary positions and the quantised cache write: gdn_rope_kv_write with K row L + i and
 * V row L + i quantised; q_out is the same.
 *
 *   cache   rows L .. L + N_c - 1 written
 *   every other argument, the errors and the status bits as in gdn_rope_kv_write
 */
int gdn_rope_kv4_write(const gdn_attn_shape *sh, int32_t x_dtype, const gdn_heads_view *q, const gdn_heads_view *k,
                       const gdn_heads_view *v, const gdn_rope *rope, const gdn_kv4_cache *cache,
                       const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                       const int32_t *parents, const int32_t *lane_nodes, void *q_out, int32_t *status,
                       hipStream_t stream);

/*
 * Attention of the round's tokens over the 4-bit cache: gdn_paged_attention over the values
 * that the cache's rows stand for, with the same treatment of rows that are not attended, of
 * NaN blocks, of absent pages and of nodes without a row.
 *
 *   cache      (read); the round's rows are there
 *   workspace  at least gdn_paged_attention_kv4_workspace_size(sh) bytes
 *   every other argument, the errors and the status bits as in gdn_paged_attention
 */
int gdn_paged_attention_kv4(const gdn_attn_shape *sh, const void *q, const gdn_kv4_cache *cache,
                            const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                            const int32_t *parents, const int32_t *lane_nodes, float scale,
                            const gdn_heads_view *gate, int32_t gate_mode, void *out, void *workspace,
                            size_t workspace_bytes, int32_t *status, hipStream_t stream);

/* Bytes of workspace gdn_paged_attention_kv4 needs for this shape; 0 where the cache is not
   split over workgroups, or for an invalid shape. */
size_t gdn_paged_attention_kv4_workspace_size(const gdn_attn_shape *sh);

/*
 * Commit of the 4-bit caches: gdn_kv_commit_layers with codes and scales moved byte for byte.
 *
 *   caches  host array of n_layers caches, updated in place; all arrays disjoint
 *   every other argument, the errors and the status bits as in gdn_kv_commit_layers
 */
int gdn_kv4_commit_layers(const gdn_attn_shape *sh, int32_t n_layers, const gdn_kv4_cache *caches,
                          const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                          const int32_t *parents, const int32_t *lane_nodes, const int32_t *accept_node,
                          int32_t *new_len, int32_t *status, hipStream_t stream);

/*
 * Rows of the 4-bit caches as values: for every layer l, every present i of a valid lane and
 * every kv head h,
 *   k_out[l][c][i][h], v_out[l][c][i][h] = the values of row first_row[c] + i of slot s
 * in sh->dtype.  Lanes may share a slot; rows are read whether committed or not.  Nothing is
 * written for an offending lane, nor for a row in a page outside the pool (PAGE).
 *
 *   n_layers   1..GDN_MAX_LAYERS
 *   caches     host array of n_layers caches (read); layers may share arrays
 *   slot_ids, page_table, lane_nodes  as in gdn_rope_kv_write
 *   first_row  [C], >= 0, and first_row + N_c at most max_pages * page_size (LENGTH)  (read)
 *   k_out, v_out  [n_layers][C][N][H_kv][D]; either may be NULL (not both): not asked for
 *   status     may be NULL; SLOT_RANGE / NODES / LENGTH / PAGE
 * sh->n_q_heads is not used but has to be valid.
 */
int gdn_kv4_read_layers(const gdn_attn_shape *sh, int32_t n_layers, const gdn_kv4_cache *caches,
                        const int32_t *slot_ids, const int32_t *page_table, const int32_t *first_row,
                        const int32_t *lane_nodes, void *k_out, void *v_out, int32_t *status, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_KV4_H */

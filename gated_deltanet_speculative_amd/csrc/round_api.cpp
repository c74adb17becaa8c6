// Host entry points of gdn_round.h: argument validation, byte-range alias checks and kernel
// dispatch on the caller's stream.  Every check runs before anything is enqueued; no entry
// point allocates, synchronises or keeps state between calls.
#include "round_checks.h"

extern "C" {

int gdn_rope_kv_write(const gdn_attn_shape *sh, int32_t x_dtype, const gdn_heads_view *q, const gdn_heads_view *k,
                      const gdn_heads_view *v, const gdn_rope *rope, void *k_cache, void *v_cache,
                      const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                      const int32_t *parents, const int32_t *lane_nodes, void *q_out, int32_t *status,
                      hipStream_t stream) {
    gdn::RopeArgs a{};
    const CacheArrays cache{k_cache, v_cache, nullptr, nullptr};
    if (int r = check_rope(sh, x_dtype, q, k, v, rope, cache, slot_ids, page_table, seq_len, parents, lane_nodes, q_out, status, &a))
        return r;
    return gdn::launch_rope_kv_write(a, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_paged_attention_workspace_size(const gdn_attn_shape *sh) {
    gdn::AttnDims d;
    if (check_attn(sh, false, &d)) return 0;
    return gdn::attn_workspace_floats(d, gdn::attn_plan(d)) * F;
}

int gdn_paged_attention(const gdn_attn_shape *sh, const void *q, const void *k_cache, const void *v_cache,
                        const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                        const int32_t *parents, const int32_t *lane_nodes, float scale, const gdn_heads_view *gate,
                        int32_t gate_mode, void *out, void *workspace, size_t workspace_bytes, int32_t *status,
                        hipStream_t stream) {
    gdn::AttnArgs a{};
    const CacheArrays cache{const_cast<void *>(k_cache), const_cast<void *>(v_cache), nullptr, nullptr};
    if (int r = check_attention(sh, q, cache, slot_ids, page_table, seq_len, parents, lane_nodes, scale, gate, gate_mode, out,
                                workspace, workspace_bytes, gdn::attn_plan, status, &a))
        return r;
    return gdn::launch_paged_attention(a, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

static int check_accept(const gdn_accept_shape *sh) {
    if (!sh) return GDN_ERR_NULL;
    if (sh->n_seqs <= 0 || sh->n_nodes <= 0 || sh->vocab <= 0 || !known_dtype(sh->dtype)) return GDN_ERR_SHAPE;
    if (sh->n_seqs > GDN_MAX_SEQS || sh->n_nodes > GDN_MAX_NODES || sh->vocab > (1 << 24)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

size_t gdn_draft_accept_workspace_size(const gdn_accept_shape *sh) {
    if (check_accept(sh)) return 0;
    return gdn::accept_workspace_bytes(sh->n_seqs, sh->n_nodes, sh->vocab);
}

int gdn_draft_accept(const gdn_accept_shape *sh, const void *target, const void *root, const void *draft,
                     const int32_t *tokens, const int32_t *parents, const int32_t *lane_nodes,
                     const int32_t *slot_ids, const float *u_accept, const float *u_next, int32_t *accept_node,
                     int32_t *n_accept, int32_t *next_token, void *workspace, size_t workspace_bytes,
                     int32_t *status, hipStream_t stream) {
    if (int r = check_accept(sh)) return r;
    if (!target || !tokens || !accept_node || !n_accept || !next_token || !workspace || (!u_accept) != (!u_next))
        return GDN_ERR_NULL;
    if (draft && (parents || !u_accept)) return GDN_ERR_UNSUPPORTED;
    const int C = sh->n_seqs, N = sh->n_nodes, V = sh->vocab;
    const size_t es = value_bytes(sh->dtype), ws_b = gdn::accept_workspace_bytes(C, N, V);
    if (workspace_bytes < ws_b) return GDN_ERR_WORKSPACE;
    if (!aligned({target, root, draft}, es) || !aligned({workspace}, 16) ||
        !aligned({tokens, parents, lane_nodes, slot_ids, u_accept, u_next, accept_node, n_accept, next_token, status}, 4))
        return GDN_ERR_ALIGN;
    const size_t rows = (size_t)C * N, cb = (size_t)C * I, tb = rows * V * es;
    if (any_alias({{accept_node, cb}, {n_accept, cb}, {next_token, cb}, {workspace, ws_b}, {status, I}},
                  {{target, tb}, {root, (size_t)C * V * es}, {draft, tb}, {tokens, rows * I}, {parents, rows * I},
                   {lane_nodes, cb}, {slot_ids, cb}, {u_accept, rows * F}, {u_next, (size_t)C * F}}))
        return GDN_ERR_ALIAS;
    gdn::AcceptArgs a{C, N, V, sh->dtype, target, root, draft, tokens, parents, lane_nodes, slot_ids, u_accept, u_next,
                      accept_node, n_accept, next_token, workspace, status};
    return gdn::launch_draft_accept(a, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

int gdn_kv_commit_layers(const gdn_attn_shape *sh, int32_t n_layers, void *const *k_caches, void *const *v_caches,
                         const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                         const int32_t *parents, const int32_t *lane_nodes, const int32_t *accept_node,
                         int32_t *new_len, int32_t *status, hipStream_t stream) {
    gdn::AttnDims d;
    if (int r = check_attn(sh, parents != nullptr, &d)) return r;
    if (n_layers < 1 || n_layers > GDN_MAX_LAYERS) return GDN_ERR_UNSUPPORTED;
    if (!k_caches || !v_caches || !slot_ids || !page_table || !seq_len || !accept_node || !new_len || !status)
        return GDN_ERR_NULL;
    const size_t cb = cache_bytes(d), rows = (size_t)d.C * d.N;
    gdn::CacheLayers cl{};
    for (int l = 0; l < n_layers; ++l) {
        if (!k_caches[l] || !v_caches[l]) return GDN_ERR_NULL;
        if (!aligned({k_caches[l], v_caches[l]}, 16)) return GDN_ERR_ALIGN;
        cl.k[l] = k_caches[l];
        cl.v[l] = v_caches[l];
    }
    if (!aligned({slot_ids, page_table, seq_len, parents, lane_nodes, accept_node, new_len, status}, 4))
        return GDN_ERR_ALIGN;
    const std::initializer_list<Range> ins = {{slot_ids, (size_t)d.C * I}, {page_table, (size_t)d.P * d.max_pages * I},
                                              {seq_len, (size_t)d.P * I}, {parents, rows * I},
                                              {lane_nodes, (size_t)d.C * I}, {accept_node, (size_t)d.C * I}};
    if (any_alias({{new_len, (size_t)d.P * I}, {status, I}}, ins)) return GDN_ERR_ALIAS;
    // every cache against every input, the other outputs and every other cache
    for (int l = 0; l < 2 * n_layers; ++l) {
        const Range o{l % 2 ? cl.v[l / 2] : cl.k[l / 2], cb};
        if (any_alias({o, {new_len, (size_t)d.P * I}, {status, I}}, ins)) return GDN_ERR_ALIAS;
        for (int m = 0; m < l; ++m)
            if (overlap(o, {m % 2 ? cl.v[m / 2] : cl.k[m / 2], cb})) return GDN_ERR_ALIAS;
    }
    return gdn::launch_kv_commit(d, n_layers, cl,
                                 gdn::PagedLanes{slot_ids, page_table, seq_len, parents, lane_nodes, status},
                                 accept_node, new_len, stream) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

}  // extern "C"

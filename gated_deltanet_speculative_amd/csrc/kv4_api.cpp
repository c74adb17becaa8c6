// Host entry points of gdn_kv4.h: argument validation, byte-range alias checks and kernel dispatch on the caller's stream.
// Every check runs before anything is enqueued; no entry point allocates, synchronises or keeps state between calls.
#include <algorithm>

#include "gdn_kv4.h"
#include "round_checks.h"

namespace {

bool whole(const gdn_kv4_cache *c) { return c && c->k_codes && c->k_scales && c->v_codes && c->v_scales; }

CacheArrays arrays_of(const gdn_kv4_cache &c) { return CacheArrays{c.k_codes, c.v_codes, c.k_scales, c.v_scales}; }

// The caches of a call's layers: all there and aligned
int check_layers(const gdn::AttnDims &d, int32_t n_layers, const gdn_kv4_cache *caches, gdn::Cache4Layers *cl) {
    for (int l = 0; l < n_layers; ++l) {
        const gdn_kv4_cache &c = caches[l];
        if (!whole(&c)) return GDN_ERR_NULL;
        if (!aligned({c.k_codes, c.v_codes}, 16) || !aligned({c.k_scales, c.v_scales}, d.D / 32)) return GDN_ERR_ALIGN;
        cl->codes.k[l] = c.k_codes;
        cl->codes.v[l] = c.v_codes;
        cl->scales.k[l] = c.k_scales;
        cl->scales.v[l] = c.v_scales;
    }
    return GDN_OK;
}
// Array j of a layer: codes and scales of K, then of V
Range array_of(const gdn::AttnDims &d, const gdn_kv4_cache &c, int j) {
    const CacheArrays a = arrays_of(c);
    return j & 1 ? a.scales(d, j >> 1) : a.codes(d, j >> 1);
}

bool overlap_any(const Range &o, std::initializer_list<Range> others) {
    for (const Range &r : others)
        if (overlap(o, r)) return true;
    return false;
}
// Whether two of the ranges (none of them empty) overlap: in the order of their addresses, some neighbours then do
bool any_overlap(const Range *r, int n) {
    Range by[4 * GDN_MAX_LAYERS];
    std::copy(r, r + n, by);
    std::sort(by, by + n, [](const Range &a, const Range &b) { return a.p < b.p; });
    for (int k = 1; k < n; ++k)
        if (overlap(by[k - 1], by[k])) return true;
    return false;
}

}  // namespace

extern "C" {

int gdn_rope_kv4_write(const gdn_attn_shape *sh, int32_t x_dtype, const gdn_heads_view *q, const gdn_heads_view *k,
                       const gdn_heads_view *v, const gdn_rope *rope, const gdn_kv4_cache *cache,
                       const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                       const int32_t *parents, const int32_t *lane_nodes, void *q_out, int32_t *status,
                       hipStream_t stream) {
    if (!sh || !whole(cache)) return GDN_ERR_NULL;
    gdn::RopeArgs a{};
    if (int r = check_rope(sh, x_dtype, q, k, v, rope, arrays_of(*cache), slot_ids, page_table, seq_len, parents, lane_nodes,
                           q_out, status, &a))
        return r;
    return gdn::launch_rope_kv_write(a, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_paged_attention_kv4_workspace_size(const gdn_attn_shape *sh) {
    gdn::AttnDims d;
    if (check_attn(sh, false, &d)) return 0;
    return gdn::attn_workspace_floats(d, gdn::attn_plan_kv4(d)) * F;
}

int gdn_paged_attention_kv4(const gdn_attn_shape *sh, const void *q, const gdn_kv4_cache *cache,
                            const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                            const int32_t *parents, const int32_t *lane_nodes, float scale,
                            const gdn_heads_view *gate, int32_t gate_mode, void *out, void *workspace,
                            size_t workspace_bytes, int32_t *status, hipStream_t stream) {
    if (!sh || !whole(cache)) return GDN_ERR_NULL;
    gdn::AttnArgs a{};
    if (int r = check_attention(sh, q, arrays_of(*cache), slot_ids, page_table, seq_len, parents, lane_nodes, scale, gate,
                                gate_mode, out, workspace, workspace_bytes, gdn::attn_plan_kv4, status, &a))
        return r;
    return gdn::launch_paged_attention_kv4(a, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

int gdn_kv4_commit_layers(const gdn_attn_shape *sh, int32_t n_layers, const gdn_kv4_cache *caches,
                          const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                          const int32_t *parents, const int32_t *lane_nodes, const int32_t *accept_node,
                          int32_t *new_len, int32_t *status, hipStream_t stream) {
    gdn::AttnDims d;
    if (int r = check_attn(sh, parents != nullptr, &d)) return r;
    if (n_layers < 1 || n_layers > GDN_MAX_LAYERS) return GDN_ERR_UNSUPPORTED;
    if (!caches || !slot_ids || !page_table || !seq_len || !accept_node || !new_len || !status) return GDN_ERR_NULL;
    gdn::Cache4Layers cl{};
    if (int r = check_layers(d, n_layers, caches, &cl)) return r;
    if (!aligned({slot_ids, page_table, seq_len, parents, lane_nodes, accept_node, new_len, status}, 4))
        return GDN_ERR_ALIGN;
    const size_t rows = (size_t)d.C * d.N;
    const std::initializer_list<Range> ins = {{slot_ids, (size_t)d.C * I}, {page_table, (size_t)d.P * d.max_pages * I},
                                              {seq_len, (size_t)d.P * I}, {parents, rows * I},
                                              {lane_nodes, (size_t)d.C * I}, {accept_node, (size_t)d.C * I}};
    if (any_alias({{new_len, (size_t)d.P * I}, {status, I}}, ins)) return GDN_ERR_ALIAS;
    // every array against every input, the other outputs and every other array
    Range arrays[4 * GDN_MAX_LAYERS];
    for (int l = 0; l < 4 * n_layers; ++l) arrays[l] = array_of(d, caches[l / 4], l % 4);
    if (any_overlap(arrays, 4 * n_layers)) return GDN_ERR_ALIAS;
    for (int l = 0; l < 4 * n_layers; ++l)
        if (overlap_any(arrays[l], ins) || overlap(arrays[l], {new_len, (size_t)d.P * I}) || overlap(arrays[l], {status, I}))
            return GDN_ERR_ALIAS;
    return gdn::launch_kv4_commit(d, n_layers, cl,
                                  gdn::PagedLanes{slot_ids, page_table, seq_len, parents, lane_nodes, status},
                                  accept_node, new_len, stream) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

int gdn_kv4_read_layers(const gdn_attn_shape *sh, int32_t n_layers, const gdn_kv4_cache *caches,
                        const int32_t *slot_ids, const int32_t *page_table, const int32_t *first_row,
                        const int32_t *lane_nodes, void *k_out, void *v_out, int32_t *status, hipStream_t stream) {
    gdn::AttnDims d;
    if (int r = check_attn(sh, false, &d)) return r;
    if (n_layers < 1 || n_layers > GDN_MAX_LAYERS) return GDN_ERR_UNSUPPORTED;
    if (!caches || !slot_ids || !page_table || !first_row || (!k_out && !v_out)) return GDN_ERR_NULL;
    gdn::Cache4Layers cl{};
    if (int r = check_layers(d, n_layers, caches, &cl)) return r;
    if (!aligned({k_out, v_out}, 16) || !aligned({slot_ids, page_table, first_row, lane_nodes, status}, 4)) return GDN_ERR_ALIGN;
    const size_t cb = (size_t)d.C * I, ob = (size_t)n_layers * d.C * d.N * d.Hkv * d.D * value_bytes(d.dtype);
    const Range outs[3] = {{k_out, ob}, {v_out, ob}, {status, I}};
    if (any_alias({outs[0], outs[1], outs[2]}, {{slot_ids, cb}, {page_table, (size_t)d.P * d.max_pages * I}, {first_row, cb}, {lane_nodes, cb}}))
        return GDN_ERR_ALIAS;
    for (int l = 0; l < 4 * n_layers; ++l)
        for (const Range &o : outs)
            if (overlap(o, array_of(d, caches[l / 4], l % 4))) return GDN_ERR_ALIAS;
    return gdn::launch_kv4_read(d, n_layers, cl, gdn::PagedLanes{slot_ids, page_table, nullptr, nullptr, lane_nodes, status},
                                first_row, k_out, v_out, stream) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

}  // extern "C"

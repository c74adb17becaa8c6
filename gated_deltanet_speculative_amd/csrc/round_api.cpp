// Host entry points of gdn_round.h: argument validation, byte-range alias checks and kernel
// dispatch on the caller's stream.  Every check runs before anything is enqueued; no entry
// point allocates, synchronises or keeps state between calls.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "round_internal.h"

namespace {

struct Range {
    const void *p;
    size_t bytes;
};

bool overlap(const Range &a, const Range &b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const char *a0 = static_cast<const char *>(a.p), *b0 = static_cast<const char *>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// every output range against every input and every other output
bool any_alias(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Range &i : ins)
            if (overlap(*o, i)) return true;
        for (auto o2 = o + 1; o2 != outs.end(); ++o2)
            if (overlap(*o, *o2)) return true;
    }
    return false;
}

bool aligned(std::initializer_list<const void *> ps, uintptr_t a) {
    for (const void *p : ps)
        if (reinterpret_cast<uintptr_t>(p) % a) return false;
    return true;
}

constexpr size_t F = sizeof(float), I = sizeof(int32_t);
size_t value_bytes(int dtype) { return dtype == GDN_DTYPE_F32 ? 4 : 2; }
bool known_dtype(int dtype) { return dtype >= GDN_DTYPE_F32 && dtype <= GDN_DTYPE_F16; }

int check_attn(const gdn_attn_shape *sh, bool tree, gdn::AttnDims *d) {
    if (!sh) return GDN_ERR_NULL;
    if (sh->n_seqs <= 0 || sh->n_nodes <= 0 || sh->n_slots <= 0 || sh->n_q_heads <= 0 || sh->n_kv_heads <= 0 ||
        sh->head_dim <= 0 || sh->page_size <= 0 || sh->n_pages <= 0 || sh->max_pages <= 0 || !known_dtype(sh->dtype))
        return GDN_ERR_SHAPE;
    if (sh->n_q_heads % sh->n_kv_heads != 0) return GDN_ERR_SHAPE;
    constexpr int64_t kRows = 1 << 30;
    if ((sh->head_dim != 64 && sh->head_dim != 128 && sh->head_dim != 256) || sh->n_seqs > GDN_MAX_SEQS ||
        sh->n_nodes > (tree ? GDN_MAX_NODES : GDN_MAX_CHAIN) || sh->n_q_heads > 1024 || sh->page_size > 65536)
        return GDN_ERR_UNSUPPORTED;
    if ((int64_t)sh->n_kv_heads * sh->page_size > kRows / sh->n_pages ||
        (int64_t)sh->max_pages * sh->page_size > kRows || (int64_t)sh->n_slots * sh->max_pages > kRows ||
        (int64_t)sh->n_seqs * sh->n_nodes * sh->n_q_heads > (1 << 28))
        return GDN_ERR_UNSUPPORTED;
    *d = gdn::AttnDims{sh->n_seqs, sh->n_nodes, sh->n_slots, sh->n_q_heads, sh->n_kv_heads,
                       sh->n_q_heads / sh->n_kv_heads, sh->head_dim, sh->n_pages, sh->max_pages, sh->dtype,
                       gdn::Divisor::of((uint32_t)sh->page_size)};
    return GDN_OK;
}

size_t cache_bytes(const gdn::AttnDims &d) {
    return (size_t)d.n_pages * d.Hkv * d.page.d * d.D * value_bytes(d.dtype);
}

// A view's strides; its extent in bytes where they are sound.
int check_view(const gdn_heads_view &v, const gdn::AttnDims &d, int heads, int dtype, size_t *bytes) {
    const size_t es = value_bytes(dtype);
    constexpr int64_t kMost = 1ll << 40;
    if (v.token_stride < 0 || v.head_stride < 0 || v.token_stride > kMost || v.head_stride > kMost) return GDN_ERR_SHAPE;
    if (!aligned({v.p}, 16) || v.token_stride * es % 16 || v.head_stride * es % 16) return GDN_ERR_ALIGN;
    *bytes = ((size_t)((int64_t)d.C * d.N - 1) * v.token_stride + (size_t)(heads - 1) * v.head_stride + d.D) * es;
    return GDN_OK;
}

gdn::HeadsView view_of(const gdn_heads_view &v) { return gdn::HeadsView{v.p, v.token_stride, v.head_stride}; }

}  // namespace

extern "C" {

int gdn_rope_kv_write(const gdn_attn_shape *sh, int32_t x_dtype, const gdn_heads_view *q, const gdn_heads_view *k,
                      const gdn_heads_view *v, const gdn_rope *rope, void *k_cache, void *v_cache,
                      const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                      const int32_t *parents, const int32_t *lane_nodes, void *q_out, int32_t *status,
                      hipStream_t stream) {
    gdn::AttnDims d;
    if (int r = check_attn(sh, parents != nullptr, &d)) return r;
    if (!q || !k || !v || !rope || !q->p || !k->p || !v->p || !rope->inv_freq || !k_cache || !v_cache || !slot_ids ||
        !page_table || !seq_len || !q_out)
        return GDN_ERR_NULL;
    if (!known_dtype(x_dtype) || rope->n_axes < 1 || rope->rot_dim <= 0 || rope->rot_dim % 16 || rope->rot_dim > d.D ||
        (rope->interleaved != 0 && rope->interleaved != 1) || !(rope->eps >= 0.f))
        return GDN_ERR_SHAPE;
    if ((x_dtype != d.dtype && x_dtype != GDN_DTYPE_F32) || rope->n_axes > 16) return GDN_ERR_UNSUPPORTED;
    if (!rope->positions && rope->n_axes != 1) return GDN_ERR_SHAPE;
    size_t qb, kb, vb;
    if (int r = check_view(*q, d, d.Hq, x_dtype, &qb)) return r;
    if (int r = check_view(*k, d, d.Hkv, x_dtype, &kb)) return r;
    if (int r = check_view(*v, d, d.Hkv, x_dtype, &vb)) return r;
    if (!aligned({k_cache, v_cache, q_out}, 16) || !aligned({rope->inv_freq}, 8) ||
        !aligned({rope->positions, rope->pair_axis, rope->q_norm, rope->k_norm, slot_ids, page_table, seq_len, parents,
                  lane_nodes, status}, 4))
        return GDN_ERR_ALIGN;
    const size_t rows = (size_t)d.C * d.N, half = (size_t)rope->rot_dim / 2, cb = cache_bytes(d);
    if (any_alias({{k_cache, cb}, {v_cache, cb}, {q_out, rows * d.Hq * d.D * value_bytes(d.dtype)}, {status, I}},
                  {{q->p, qb}, {k->p, kb}, {v->p, vb}, {rope->inv_freq, half * 8},
                   {rope->positions, rows * rope->n_axes * I}, {rope->pair_axis, half * I},
                   {rope->q_norm, d.D * F}, {rope->k_norm, d.D * F}, {slot_ids, (size_t)d.C * I},
                   {page_table, (size_t)d.P * d.max_pages * I}, {seq_len, (size_t)d.P * I}, {parents, rows * I},
                   {lane_nodes, (size_t)d.C * I}}))
        return GDN_ERR_ALIAS;
    gdn::RopeArgs a{};
    a.d = d;
    a.l = gdn::PagedLanes{slot_ids, page_table, seq_len, parents, lane_nodes, status};
    a.x_dtype = x_dtype;
    a.q = view_of(*q);
    a.k = view_of(*k);
    a.v = view_of(*v);
    a.inv_freq = rope->inv_freq;
    a.positions = rope->positions;
    a.pair_axis = rope->pair_axis;
    a.n_axes = rope->n_axes;
    a.half = rope->rot_dim / 2;
    a.interleaved = rope->interleaved;
    a.q_norm = rope->q_norm;
    a.k_norm = rope->k_norm;
    a.eps = rope->eps;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.q_out = q_out;
    return gdn::launch_rope_kv_write(a, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_paged_attention_workspace_size(const gdn_attn_shape *sh) {
    gdn::AttnDims d;
    if (check_attn(sh, false, &d)) return 0;
    return gdn::attn_workspace_floats(d) * F;
}

int gdn_paged_attention(const gdn_attn_shape *sh, const void *q, const void *k_cache, const void *v_cache,
                        const int32_t *slot_ids, const int32_t *page_table, const int32_t *seq_len,
                        const int32_t *parents, const int32_t *lane_nodes, float scale, const gdn_heads_view *gate,
                        int32_t gate_mode, void *out, void *workspace, size_t workspace_bytes, int32_t *status,
                        hipStream_t stream) {
    gdn::AttnDims d;
    if (int r = check_attn(sh, parents != nullptr, &d)) return r;
    if (!q || !k_cache || !v_cache || !slot_ids || !page_table || !seq_len || !out || (gate && !gate->p))
        return GDN_ERR_NULL;
    const float scale_log2 = scale * 1.4426950408889634f;  // the kernels' exponentials are of base 2
    if (!(scale_log2 > 0.f) || !std::isfinite(scale_log2) || (gate_mode != 0 && gate_mode != 1)) return GDN_ERR_SHAPE;
    size_t gb = 0;
    if (gate)
        if (int r = check_view(*gate, d, d.Hq, d.dtype, &gb)) return r;
    const size_t ws_b = gdn::attn_workspace_floats(d) * F;
    if (ws_b && !workspace) return GDN_ERR_NULL;
    if (workspace_bytes < ws_b) return GDN_ERR_WORKSPACE;
    if (!aligned({q, k_cache, v_cache, out, workspace}, 16) ||
        !aligned({slot_ids, page_table, seq_len, parents, lane_nodes, status}, 4))
        return GDN_ERR_ALIGN;
    const size_t rows = (size_t)d.C * d.N, cb = cache_bytes(d), ob = rows * d.Hq * d.D * value_bytes(d.dtype);
    if (any_alias({{out, ob}, {workspace, ws_b}, {status, I}},
                  {{q, ob}, {k_cache, cb}, {v_cache, cb}, {slot_ids, (size_t)d.C * I},
                   {page_table, (size_t)d.P * d.max_pages * I}, {seq_len, (size_t)d.P * I}, {parents, rows * I},
                   {lane_nodes, (size_t)d.C * I}, {gate ? gate->p : nullptr, gb}}))
        return GDN_ERR_ALIAS;
    gdn::AttnArgs a{};
    a.d = d;
    a.l = gdn::PagedLanes{slot_ids, page_table, seq_len, parents, lane_nodes, status};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.scale_log2 = scale_log2;
    if (gate) a.gate = view_of(*gate);
    a.gate_mode = gate_mode;
    a.out = out;
    a.workspace = static_cast<float *>(workspace);
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

// Argument checks shared by the host entry points over paged caches and logits: byte ranges, alignment, shapes and
// views.  Nothing here calls the device.
#pragma once

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "round_internal.h"

namespace {

struct Range {
    const void *p;
    size_t bytes;
};

inline bool overlap(const Range &a, const Range &b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const char *a0 = static_cast<const char *>(a.p), *b0 = static_cast<const char *>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// every output range against every input and every other output
inline bool any_alias(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Range &i : ins)
            if (overlap(*o, i)) return true;
        for (auto o2 = o + 1; o2 != outs.end(); ++o2)
            if (overlap(*o, *o2)) return true;
    }
    return false;
}

inline bool aligned(std::initializer_list<const void *> ps, uintptr_t a) {
    for (const void *p : ps)
        if (reinterpret_cast<uintptr_t>(p) % a) return false;
    return true;
}

constexpr size_t F = sizeof(float), I = sizeof(int32_t);
inline size_t value_bytes(int dtype) { return dtype == GDN_DTYPE_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) { return dtype >= GDN_DTYPE_F32 && dtype <= GDN_DTYPE_F16; }

inline int check_attn(const gdn_attn_shape *sh, bool tree, gdn::AttnDims *d) {
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

inline size_t cache_bytes(const gdn::AttnDims &d) {
    return (size_t)d.n_pages * d.Hkv * d.page.d * d.D * value_bytes(d.dtype);
}

// A view's strides; its extent in bytes where they are sound.
inline int check_view(const gdn_heads_view &v, const gdn::AttnDims &d, int heads, int dtype, size_t *bytes) {
    const size_t es = value_bytes(dtype);
    constexpr int64_t kMost = 1ll << 40;
    if (v.token_stride < 0 || v.head_stride < 0 || v.token_stride > kMost || v.head_stride > kMost) return GDN_ERR_SHAPE;
    if (!aligned({v.p}, 16) || v.token_stride * es % 16 || v.head_stride * es % 16) return GDN_ERR_ALIGN;
    *bytes = ((size_t)((int64_t)d.C * d.N - 1) * v.token_stride + (size_t)(heads - 1) * v.head_stride + d.D) * es;
    return GDN_OK;
}

inline gdn::HeadsView view_of(const gdn_heads_view &v) { return gdn::HeadsView{v.p, v.token_stride, v.head_stride}; }

// One layer's cache: values of the shape's dtype, or (with scales) codes of 4 bits.
struct CacheArrays {
    void *k, *v, *k_scales, *v_scales;
    Range codes(const gdn::AttnDims &d, int side) const {
        return Range{side ? v : k, k_scales ? (size_t)d.n_pages * d.Hkv * d.page.d * (d.D / 2) : cache_bytes(d)};
    }
    Range scales(const gdn::AttnDims &d, int side) const {
        return Range{side ? v_scales : k_scales, (size_t)d.n_pages * d.Hkv * d.page.d * (d.D / 32)};
    }
};

// Checks of the rotary cache writes, and the launcher's arguments
inline int check_rope(const gdn_attn_shape *sh, int32_t x_dtype, const gdn_heads_view *q, const gdn_heads_view *k,
               const gdn_heads_view *v, const gdn_rope *rope, const CacheArrays &cache, const int32_t *slot_ids,
               const int32_t *page_table, const int32_t *seq_len, const int32_t *parents, const int32_t *lane_nodes,
               void *q_out, int32_t *status, gdn::RopeArgs *a) {
    gdn::AttnDims d;
    if (int r = check_attn(sh, parents != nullptr, &d)) return r;
    if (!q || !k || !v || !rope || !q->p || !k->p || !v->p || !rope->inv_freq || !cache.k || !cache.v || !slot_ids ||
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
    if (!aligned({cache.k, cache.v, q_out}, 16) || !aligned({cache.k_scales, cache.v_scales}, d.D / 32) || !aligned({rope->inv_freq}, 8) ||
        !aligned({rope->positions, rope->pair_axis, rope->q_norm, rope->k_norm, slot_ids, page_table, seq_len, parents,
                  lane_nodes, status}, 4))
        return GDN_ERR_ALIGN;
    const size_t rows = (size_t)d.C * d.N, half = (size_t)rope->rot_dim / 2;
    if (any_alias({cache.codes(d, 0), cache.codes(d, 1), cache.scales(d, 0), cache.scales(d, 1), {q_out, rows * d.Hq * d.D * value_bytes(d.dtype)}, {status, I}},
                  {{q->p, qb}, {k->p, kb}, {v->p, vb}, {rope->inv_freq, half * 8},
                   {rope->positions, rows * rope->n_axes * I}, {rope->pair_axis, half * I},
                   {rope->q_norm, d.D * F}, {rope->k_norm, d.D * F}, {slot_ids, (size_t)d.C * I},
                   {page_table, (size_t)d.P * d.max_pages * I}, {seq_len, (size_t)d.P * I}, {parents, rows * I},
                   {lane_nodes, (size_t)d.C * I}}))
        return GDN_ERR_ALIAS;
    a->d = d;
    a->l = gdn::PagedLanes{slot_ids, page_table, seq_len, parents, lane_nodes, status};
    a->x_dtype = x_dtype;
    a->q = view_of(*q);
    a->k = view_of(*k);
    a->v = view_of(*v);
    a->inv_freq = rope->inv_freq;
    a->positions = rope->positions;
    a->pair_axis = rope->pair_axis;
    a->n_axes = rope->n_axes;
    a->half = rope->rot_dim / 2;
    a->interleaved = rope->interleaved;
    a->q_norm = rope->q_norm;
    a->k_norm = rope->k_norm;
    a->eps = rope->eps;
    a->k_cache = cache.k;
    a->v_cache = cache.v;
    a->k_scales = cache.k_scales;
    a->v_scales = cache.v_scales;
    a->q_out = q_out;
    return GDN_OK;
}

// Checks of the attention calls, and the launcher's arguments; plan: how the call is divided
inline int check_attention(const gdn_attn_shape *sh, const void *q, const CacheArrays &cache, const int32_t *slot_ids,
                    const int32_t *page_table, const int32_t *seq_len, const int32_t *parents, const int32_t *lane_nodes,
                    float scale, const gdn_heads_view *gate, int32_t gate_mode, void *out, void *workspace,
                    size_t workspace_bytes, gdn::AttnPlan (*plan)(const gdn::AttnDims &), int32_t *status, gdn::AttnArgs *a) {
    gdn::AttnDims d;
    if (int r = check_attn(sh, parents != nullptr, &d)) return r;
    if (!q || !cache.k || !cache.v || !slot_ids || !page_table || !seq_len || !out || (gate && !gate->p))
        return GDN_ERR_NULL;
    const float scale_log2 = scale * 1.4426950408889634f;  // the kernels' exponentials are of base 2
    if (!(scale_log2 > 0.f) || !std::isfinite(scale_log2) || (gate_mode != 0 && gate_mode != 1)) return GDN_ERR_SHAPE;
    size_t gb = 0;
    if (gate)
        if (int r = check_view(*gate, d, d.Hq, d.dtype, &gb)) return r;
    const size_t ws_b = gdn::attn_workspace_floats(d, plan(d)) * F;
    if (ws_b && !workspace) return GDN_ERR_NULL;
    if (workspace_bytes < ws_b) return GDN_ERR_WORKSPACE;
    if (!aligned({q, cache.k, cache.v, out, workspace}, 16) || !aligned({cache.k_scales, cache.v_scales}, d.D / 32) ||
        !aligned({slot_ids, page_table, seq_len, parents, lane_nodes, status}, 4))
        return GDN_ERR_ALIGN;
    const size_t rows = (size_t)d.C * d.N, ob = rows * d.Hq * d.D * value_bytes(d.dtype);
    if (any_alias({{out, ob}, {workspace, ws_b}, {status, I}},
                  {{q, ob}, cache.codes(d, 0), cache.codes(d, 1), cache.scales(d, 0), cache.scales(d, 1), {slot_ids, (size_t)d.C * I},
                   {page_table, (size_t)d.P * d.max_pages * I}, {seq_len, (size_t)d.P * I}, {parents, rows * I},
                   {lane_nodes, (size_t)d.C * I}, {gate ? gate->p : nullptr, gb}}))
        return GDN_ERR_ALIAS;
    a->d = d;
    a->l = gdn::PagedLanes{slot_ids, page_table, seq_len, parents, lane_nodes, status};
    a->q = q;
    a->k_cache = cache.k;
    a->v_cache = cache.v;
    a->k_scales = cache.k_scales;
    a->v_scales = cache.v_scales;
    a->scale_log2 = scale_log2;
    if (gate) a->gate = view_of(*gate);
    a->gate_mode = gate_mode;
    a->out = out;
    a->workspace = static_cast<float *>(workspace);
    return GDN_OK;
}

}  // namespace

// Host entry point of gdn_logits.h: argument validation, byte-range alias checks and kernel dispatch on the caller's
// stream.  Every check runs before anything is enqueued; nothing is allocated, synchronised or kept between calls.
#include "logits_internal.h"
#include "round_checks.h"

namespace {

int check_logits(const gdn_logits_shape *sh) {
    if (!sh) return GDN_ERR_NULL;
    if (sh->n_seqs <= 0 || sh->n_nodes <= 0 || sh->n_slots <= 0 || sh->vocab <= 0 || sh->max_history < 0 || sh->max_bias < 0 ||
        !known_dtype(sh->dtype) || !known_dtype(sh->out_dtype))
        return GDN_ERR_SHAPE;
    constexpr int64_t kEntries = 1 << 30;
    if (sh->n_seqs > GDN_MAX_SEQS || sh->n_nodes > GDN_MAX_NODES || sh->vocab > (1 << 24) || sh->max_history > (1 << 20) ||
        sh->max_bias > 1024 || (int64_t)sh->n_slots * sh->max_history > kEntries || (int64_t)sh->n_slots * sh->max_bias > kEntries ||
        (sh->out_dtype != sh->dtype && sh->out_dtype != GDN_DTYPE_F32))
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_adjust_logits_workspace_size(const gdn_logits_shape *sh) {
    if (check_logits(sh)) return 0;
    return gdn::logit_workspace_bytes(sh->n_seqs, sh->n_nodes, sh->vocab);
}

int gdn_adjust_logits(const gdn_logits_shape *sh, const void *logits, int64_t row_stride, const gdn_logit_rules *rules,
                      const int32_t *mask, const int32_t *tokens, const int32_t *parents, const int32_t *lane_nodes,
                      const int32_t *slot_ids, void *out, void *workspace, size_t workspace_bytes, int32_t *status,
                      hipStream_t stream) {
    if (int r = check_logits(sh)) return r;
    if (!logits || !rules || !slot_ids || !out || (rules->history && !rules->history_len) || (!rules->bias_tokens) != (!rules->bias))
        return GDN_ERR_NULL;
    const int C = sh->n_seqs, N = sh->n_nodes, P = sh->n_slots, V = sh->vocab;
    if (row_stride < V || row_stride > (1ll << 40)) return GDN_ERR_SHAPE;
    const size_t es = value_bytes(sh->dtype), os = value_bytes(sh->out_dtype);
    const size_t ws_b = rules->temperature ? gdn::logit_workspace_bytes(C, N, V) : 0;
    if (ws_b && !workspace) return GDN_ERR_NULL;
    if (workspace_bytes < ws_b) return GDN_ERR_WORKSPACE;
    const gdn_logit_rules &u = *rules;
    if (!aligned({logits}, es) || !aligned({out}, os) || !aligned({workspace}, 16) ||
        !aligned({u.history, u.history_len, u.prompt_len, u.repetition, u.presence, u.frequency, u.bias_tokens, u.bias, u.temperature,
                  mask, tokens, parents, lane_nodes, slot_ids, status}, 4))
        return GDN_ERR_ALIGN;
    const size_t rows = (size_t)C * N, slots = (size_t)P * I, lanes = (size_t)C * I;
    if (any_alias({{out, rows * V * os}, {workspace, ws_b}, {status, I}},
                  {{logits, ((rows - 1) * row_stride + V) * es}, {u.history, slots * sh->max_history}, {u.history_len, slots},
                   {u.prompt_len, slots}, {u.repetition, slots}, {u.presence, slots}, {u.frequency, slots},
                   {u.bias_tokens, slots * sh->max_bias}, {u.bias, slots * sh->max_bias}, {u.temperature, slots},
                   {mask, rows * ((V + 31) / 32) * I}, {tokens, rows * I}, {parents, rows * I}, {lane_nodes, lanes}, {slot_ids, lanes}}))
        return GDN_ERR_ALIAS;
    gdn::LogitArgs a{};
    a.C = C;
    a.N = N;
    a.P = P;
    a.V = V;
    a.H = sh->max_history;
    a.B = sh->max_bias;
    a.dtype = sh->dtype;
    a.out_dtype = sh->out_dtype;
    a.logits = logits;
    a.stride = row_stride;
    a.r = u;
    a.mask = mask;
    a.tokens = tokens;
    a.parents = parents;
    a.lane_nodes = lane_nodes;
    a.slot_ids = slot_ids;
    a.out = out;
    a.stats = static_cast<float *>(workspace);
    a.status = status;
    return gdn::launch_adjust_logits(a, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"

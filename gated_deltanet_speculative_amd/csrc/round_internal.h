// Internal declarations shared by the host entry points of gdn_round.h and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_round.h"

namespace gdn {

// Division of 0 <= t < 2^31 by a fixed d in 1..65536: with 2^s >= d the smallest power of two,
// m = ceil(2^(31+s) / d) < 2^32 has an error e = m d - 2^(31+s) < d <= 2^s, so
// t e < 2^(31+s) and (t m) >> (31+s) is the quotient.
struct Divisor {
    uint32_t d, mul, shift;
    static Divisor of(uint32_t d) {
        uint32_t s = 0;
        while ((1u << s) < d) ++s;
        const uint64_t p = 1ull << (31 + s);
        return Divisor{d, (uint32_t)((p + d - 1) / d), 31 + s};
    }
    __host__ __device__ uint32_t operator()(uint32_t t) const { return (uint32_t)(((uint64_t)t * mul) >> shift); }
};

struct AttnDims {
    int C, N, P, Hq, Hkv, G, D, n_pages, max_pages, dtype;
    Divisor page;
};

// What every paged call looks at to place a lane's rows.
struct PagedLanes {
    const int32_t *slot_ids, *page_table, *seq_len;
    const int32_t *parents;     // may be null: a chain
    const int32_t *lane_nodes;  // may be null: every lane has N nodes
    int32_t *status;            // may be null except for the commit
};

struct HeadsView {
    const void *p;
    int64_t token, head;  // strides in values
};

struct RopeArgs {
    AttnDims d;
    PagedLanes l;
    int x_dtype;
    HeadsView q, k, v;
    const double *inv_freq;
    const int32_t *positions, *pair_axis;
    int n_axes, half, interleaved;
    const float *q_norm, *k_norm;
    float eps;
    void *k_cache, *v_cache, *q_out;
    void *k_scales, *v_scales;  // of a 4-bit cache (the two above are its codes), else null
};
hipError_t launch_rope_kv_write(const RopeArgs &a, hipStream_t stream);

struct AttnArgs {
    AttnDims d;
    PagedLanes l;
    const void *q, *k_cache, *v_cache;  // (a 4-bit cache: its codes)
    float scale_log2;  // scale * log2(e)
    HeadsView gate;    // p null: no gate
    int gate_mode;
    void *out;
    float *workspace;
    const void *k_scales, *v_scales;  // of a 4-bit cache, else null
};
// How the rows and the cache of a call are divided over workgroups, by the shape alone.
struct AttnPlan {
    int rows_per_group;  // query rows of a workgroup
    int tiles;           // row tiles of one (lane, kv head)
    int splits;          // parts of the cache, joined by a second launch if more than one
};
AttnPlan attn_plan(const AttnDims &d);
AttnPlan attn_plan_kv4(const AttnDims &d);
inline size_t attn_workspace_floats(const AttnDims &d, const AttnPlan &p) {
    return p.splits == 1 ? 0 : (size_t)p.splits * d.C * d.N * d.Hq * (d.D + 2);
}
hipError_t launch_paged_attention(const AttnArgs &a, hipStream_t stream);
hipError_t launch_paged_attention_kv4(const AttnArgs &a, hipStream_t stream);
hipError_t launch_attention_join(const AttnArgs &a, const AttnPlan &p, hipStream_t stream);  // of the parts in the workspace

struct CacheLayers {
    void *k[GDN_MAX_LAYERS], *v[GDN_MAX_LAYERS];
};
hipError_t launch_kv_commit(const AttnDims &d, int n_layers, const CacheLayers &cl, const PagedLanes &l,
                            const int32_t *accept_node, int32_t *new_len, hipStream_t stream);

// 4-bit caches of a call's layers: codes in `codes`, scales in `scales`
struct Cache4Layers {
    CacheLayers codes, scales;
};
hipError_t launch_kv4_commit(const AttnDims &d, int n_layers, const Cache4Layers &cl, const PagedLanes &l,
                             const int32_t *accept_node, int32_t *new_len, hipStream_t stream);
// Rows from first_row on as values; either output may be null
hipError_t launch_kv4_read(const AttnDims &d, int n_layers, const Cache4Layers &cl, const PagedLanes &l,
                           const int32_t *first_row, void *k_out, void *v_out, hipStream_t stream);

struct AcceptArgs {
    int C, N, V, dtype;
    const void *target, *root, *draft;
    const int32_t *tokens, *parents, *lane_nodes, *slot_ids;
    const float *u_accept, *u_next;
    int32_t *accept_node, *n_accept, *next_token;
    void *workspace;
    int32_t *status;
};
constexpr int kAcceptChunk = 1024;  // vocabulary entries of one wave of the sampled form
__host__ __device__ inline int accept_chunks(int V) { return (V + kAcceptChunk - 1) / kAcceptChunk; }
// Sampling keeps two 64-bit sums per (lane, chunk) and 16 bytes per lane; greedy a (value, index)
// pair per (row, 4096 values).
inline size_t accept_workspace_bytes(int C, int N, int V) {
    const size_t pairs = (size_t)C * (N + 1) * ((V + 4095) / 4096) * 8, sums = (size_t)C * (accept_chunks(V) + 1) * 16;
    return ((pairs > sums ? pairs : sums) + 15) / 16 * 16;
}
hipError_t launch_draft_accept(const AcceptArgs &a, hipStream_t stream);

}  // namespace gdn

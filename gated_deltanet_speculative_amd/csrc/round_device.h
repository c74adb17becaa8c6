// Device helpers of the paged-cache and acceptance kernels: a lane's checks, its draft tree and
// the place of a cache row.
#pragma once

#include "gdn_device.h"
#include "round_internal.h"

namespace gdn {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

// The status bits of one lane's slot, node count and length; slot -1 (a padding lane) gives
// none and slot -1 back.  Reads nothing through a slot outside the pool.
struct Lane {
    int slot, nodes, len, bits;
};
__device__ inline Lane paged_lane(const AttnDims &d, const PagedLanes &l, int c) {
    Lane r{l.slot_ids[c], l.lane_nodes ? l.lane_nodes[c] : d.N, 0, 0};
    if (r.slot == -1) return r;
    if (r.nodes < 0 || r.nodes > d.N) r.bits |= GDN_STATUS_NODES;
    if (r.slot < -1 || r.slot >= d.P) {
        r.bits |= GDN_STATUS_SLOT_RANGE;
    } else {
        r.len = l.seq_len[r.slot];
        if (r.len < 0 || (int64_t)r.len + max(r.nodes, 0) > (int64_t)d.max_pages * d.page.d) r.bits |= GDN_STATUS_LENGTH;
    }
    return r;
}

// A draft tree of at most GDN_MAX_NODES nodes, one node per lane of a wave: lane i receives the
// set of i and its ancestors as a bit mask (pointer jumping: five rounds of lane shuffles), and
// `bad` whether a present node's parent lies outside [-1, i-1].  Every lane of the wave calls it.
__device__ inline unsigned tree_ancestors(const int32_t *__restrict__ parents, int nodes, bool &bad) {
    const int lane = threadIdx.x & 63;
    const bool has = lane < nodes && lane < GDN_MAX_NODES;
    const int par = has ? parents[lane] : -1;
    bad = __builtin_amdgcn_ballot_w64(has && (par < -1 || par >= lane)) != 0;
    int jump = par >= 0 && par < lane ? par : -1;
    unsigned anc = has ? 1u << lane : 0u;
#pragma unroll
    for (int r = 1; r < GDN_MAX_NODES; r <<= 1) {
        const int src = jump < 0 ? lane : jump;
        const unsigned aj = __shfl(anc, src);
        const int jj = __shfl(jump, src);
        if (jump >= 0) {
            anc |= aj;
            jump = jj;
        }
    }
    return anc;
}

// Whether another lane of the call uses slot s (every thread of the workgroup looks at a share
// of the lanes; the answer is this thread's share only).
__device__ inline bool slot_shared(const int32_t *__restrict__ slot_ids, int C, int c, int s, int tid, int threads) {
    bool dup = false;
    for (int o = tid; o < C; o += threads) dup |= o != c && slot_ids[o] == s;
    return dup;
}

// Row number (in units of D values) of place `t % page_size` of page `pid` for kv head h.
__device__ inline uint32_t cache_row(const AttnDims &d, int pid, int h, uint32_t t, uint32_t entry) {
    return ((uint32_t)pid * d.Hkv + h) * d.page.d + (t - entry * d.page.d);
}

}  // namespace gdn

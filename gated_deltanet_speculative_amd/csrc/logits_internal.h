// Internal declarations shared by the host entry point of gdn_logits.h and its kernels.
#pragma once

#include "gdn_logits.h"
#include "round_internal.h"

namespace gdn {

struct LogitArgs {
    int C, N, P, V, H, B, dtype, out_dtype;
    const void *logits;
    int64_t stride;  // of a row, in values
    gdn_logit_rules r;
    const int32_t *mask, *tokens, *parents, *lane_nodes, *slot_ids;
    void *out;
    float *stats;  // a row's maximum, sum and place of the maximum, 16 bytes per wave that shares the row
    int32_t *status;
    int rows;  // nodes of a workgroup
};

constexpr int kLogitThreads = 256;
// Tokens of a thread: 16, or 8 where there would be too few workgroups
struct LogitPlan {
    int per, rows;  // tokens a thread, nodes a workgroup
    int chunks(int V) const { return (V + per * kLogitThreads - 1) / (per * kLogitThreads); }
    int waves(int V) const { return chunks(V) * (kLogitThreads / 64); }
};
inline LogitPlan logit_plan(int C, int N, int V) {
    LogitPlan p{16, N};
    if ((int64_t)C * N * p.chunks(V) < 1024) p.per = 8;
    const int64_t groups = (int64_t)C * p.chunks(V), parts = (1023 + groups) / groups;
    p.rows = parts >= N ? 1 : (int)((N + parts - 1) / parts);
    return p;
}
inline size_t logit_workspace_bytes(int C, int N, int V) { return (size_t)C * N * logit_plan(C, N, V).waves(V) * 16; }

hipError_t launch_adjust_logits(const LogitArgs &a, hipStream_t stream);

}  // namespace gdn

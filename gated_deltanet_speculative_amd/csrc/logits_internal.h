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
    float *stats;  // a row's maximum, sum and place of the maximum, 16 bytes per wave that has a piece of it
    int32_t *status;
    int rows;  // nodes of a workgroup
};

constexpr int kLogitThreads = 512, kLogitTokens = 8, kLogitChunk = kLogitThreads * kLogitTokens;  // a stretch of the vocabulary
inline int logit_chunks(int V) { return (V + kLogitChunk - 1) / kLogitChunk; }
// Nodes of a workgroup: all of a lane's, fewer where there would be less than 512 workgroups, two a CU (4 lanes of 16 nodes,
// 130001 tokens, probabilities: with 512 workgroups 31 us, with 256 34.8)
inline int logit_rows(int C, int N, int V) {
    const int64_t groups = (int64_t)C * logit_chunks(V), parts = (511 + groups) / groups;
    return parts >= N ? 1 : (int)((N + parts - 1) / parts);
}
inline size_t logit_workspace_bytes(int C, int N, int V) { return (size_t)C * N * logit_chunks(V) * (kLogitThreads / 64) * 16; }

hipError_t launch_adjust_logits(const LogitArgs &a, hipStream_t stream);

}  // namespace gdn

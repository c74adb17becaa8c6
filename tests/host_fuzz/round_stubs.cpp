// Host-only stand-ins for the launchers of gdn_round.h: validation is what is under test.
#include "round_internal.h"
int g_launches = 0;
namespace gdn {
hipError_t launch_rope_kv_write(const RopeArgs &, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_paged_attention(const AttnArgs &, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_draft_accept(const AcceptArgs &, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_kv_commit(const AttnDims &, int, const CacheLayers &, const PagedLanes &, const int32_t *, int32_t *,
                            hipStream_t) {
    ++g_launches; return hipSuccess;
}
AttnPlan attn_plan(const AttnDims &d) {
    AttnPlan p{};
    p.splits = d.N < 64 ? 4 : 1;
    return p;
}
}  // namespace gdn

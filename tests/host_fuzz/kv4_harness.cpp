// Host-only fuzz of the argument validation of gdn_kv4.h: every entry point with fake (never dereferenced) device
// pointers over random and extreme shapes, NULL, misaligned and overlapping arguments.  Built with the sanitizers;
// the launchers below stand in for the kernels'.
#include <cstdio>
#include <random>
#include "gdn_kv4.h"
#include "round_internal.h"
static int g_launches = 0;
namespace gdn {
hipError_t launch_rope_kv_write(const RopeArgs &, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_paged_attention_kv4(const AttnArgs &, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_kv4_commit(const AttnDims &, int, const Cache4Layers &, const PagedLanes &, const int32_t *, int32_t *, hipStream_t) {
    ++g_launches; return hipSuccess;
}
hipError_t launch_kv4_read(const AttnDims &, int, const Cache4Layers &, const PagedLanes &, const int32_t *, void *, void *, hipStream_t) {
    ++g_launches; return hipSuccess;
}
AttnPlan attn_plan_kv4(const AttnDims &d) {
    AttnPlan p{};
    p.splits = d.N < 64 ? 4 : 1;
    return p;
}
}  // namespace gdn
static std::mt19937_64 rng(99);
static long long R(long long lo, long long hi) { return std::uniform_int_distribution<long long>(lo, hi)(rng); }
static char *F(long long slot) { return reinterpret_cast<char *>(0x100000000000ull + (unsigned long long)slot * (1ull << 40)); }
static void *maybe(void *p) { int r = (int)R(0, 60); if (r == 0) return nullptr; if (r == 1) return (char *)p + 4; if (r == 2) return (char *)p + 1; if (r == 3) return F(0); return p; }
static int32_t *mi(long long s) { return (int32_t *)maybe(F(s)); }
static int dims[] = {64, 128, 256, 32, 0, -64, 512};
static gdn_attn_shape shape() {
    gdn_attn_shape s;
    const bool wild = R(0, 3) == 0;
    auto pick = [&](long long a, long long b) { return (int)R(a, b); };
    s.n_seqs = wild ? pick(-1, 2000) : pick(1, 1024);
    s.n_nodes = wild ? pick(-1, 70000) : (R(0, 1) ? pick(1, 32) : pick(1, 65536));
    s.n_slots = wild ? pick(-1, 1 << 30) : pick(1, 2048);
    s.n_kv_heads = wild ? pick(-1, 1 << 20) : pick(1, 16);
    s.n_q_heads = (int)((unsigned)s.n_kv_heads * (unsigned)R(1, 8)) + (wild ? (int)R(0, 1) : 0);
    s.head_dim = dims[R(0, wild ? 6 : 2)];
    s.page_size = wild ? pick(-1, 1 << 20) : pick(1, 256);
    s.n_pages = wild ? pick(-1, 0x7fffffff) : pick(1, 4096);
    s.max_pages = wild ? pick(-1, 0x7fffffff) : pick(1, 4096);
    s.dtype = wild ? pick(-1, 3) : pick(0, 2);
    return s;
}
static gdn_heads_view view(long long s) {
    const long long strides[] = {0, 64, 128, 8, 4, 3, -8, 1ll << 50, 4096};
    return gdn_heads_view{maybe(F(s)), strides[R(0, 8)], strides[R(0, 8)]};
}
static gdn_kv4_cache cache(long long s) { return gdn_kv4_cache{maybe(F(s)), maybe(F(s + 1)), maybe(F(s + 2)), maybe(F(s + 3))}; }
int main() {
    int counts[9] = {0};
    for (int it = 0; it < 200000; ++it) {
        gdn_attn_shape s = shape();
        const gdn_attn_shape *sp = R(0, 50) ? &s : nullptr;
        const long long b = R(1, 20);
        const gdn_kv4_cache one = cache(b + 20), *cp = R(0, 40) ? &one : nullptr;
        gdn_kv4_cache many[70];
        for (int l = 0; l < 70; ++l) many[l] = gdn_kv4_cache{F(b + 40 + 4 * l), F(b + 41 + 4 * l), F(b + 42 + 4 * l), F(b + 43 + 4 * l)};
        if (R(0, 4) == 0) many[R(0, 5)] = cache(b + 40 + R(0, 30));
        const int L = (int)R(R(0, 9) ? 1 : -1, R(0, 9) ? 64 : 70);
        int r = 0;
        switch (R(0, 3)) {
        case 0: {
            const gdn_heads_view q = view(b), k = view(b + 1), v = view(b + 2);
            const gdn_rope rope{(const double *)maybe(F(b + 3)), mi(b + 4), R(0, 1) ? mi(b + 5) : nullptr, (int32_t)R(R(0, 5) ? 1 : -1, R(0, 5) ? 3 : 20),
                                (int32_t)(R(0, 3) ? 16 * R(1, 8) : R(-1, 300)), (int32_t)R(0, R(0, 9) ? 1 : 2), (const float *)(R(0, 1) ? maybe(F(b + 6)) : nullptr),
                                nullptr, R(0, 20) ? 1e-6f : -1.f};
            r = gdn_rope_kv4_write(sp, (int32_t)R(-1, 3), R(0, 40) ? &q : nullptr, &k, &v, R(0, 40) ? &rope : nullptr, cp, mi(b + 9), mi(b + 10),
                                   mi(b + 11), R(0, 1) ? mi(b + 12) : nullptr, R(0, 1) ? mi(b + 13) : nullptr, maybe(F(b + 14)), mi(b + 15), nullptr);
            break;
        }
        case 1: {
            const gdn_heads_view g = view(b);
            const size_t need = gdn_paged_attention_kv4_workspace_size(sp);
            r = gdn_paged_attention_kv4(sp, maybe(F(b + 1)), cp, mi(b + 4), mi(b + 5), mi(b + 6), R(0, 1) ? mi(b + 7) : nullptr,
                                        R(0, 1) ? mi(b + 8) : nullptr, R(0, 20) ? 0.1f : (R(0, 1) ? 0.f : 1e38f * 1e38f), R(0, 1) ? &g : nullptr,
                                        (int32_t)R(0, R(0, 9) ? 1 : 2), maybe(F(b + 9)), maybe(F(b + 10)), R(0, 5) ? need : need / 2, mi(b + 11), nullptr);
            break;
        }
        case 2:
            r = gdn_kv4_commit_layers(sp, L, R(0, 30) ? many : nullptr, mi(b), mi(b + 1), mi(b + 2), R(0, 1) ? mi(b + 3) : nullptr,
                                      R(0, 1) ? mi(b + 4) : nullptr, mi(b + 5), mi(b + 6), mi(b + 7), nullptr);
            break;
        default:
            r = gdn_kv4_read_layers(sp, L, R(0, 30) ? many : nullptr, mi(b), mi(b + 1), mi(b + 2), R(0, 1) ? mi(b + 3) : nullptr,
                                    R(0, 3) ? maybe(F(b + 4)) : nullptr, R(0, 3) ? maybe(F(b + 5)) : nullptr, R(0, 1) ? mi(b + 6) : nullptr, nullptr);
        }
        if (r < 0 || r > 8) { std::printf("unknown return %d\n", r); return 1; }
        ++counts[r];
    }
    std::printf("launches %d; codes:", g_launches);
    for (int k = 0; k < 9; ++k) std::printf(" %d:%d", k, counts[k]);
    std::printf("\n");
    return 0;
}

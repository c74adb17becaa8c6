// Host-only fuzz of the argument validation of gdn_logits.h: the call with fake (never dereferenced) device pointers over
// random and extreme shapes, NULL, misaligned and overlapping arguments.  Built with the sanitizers; the launcher below
// stands in for the kernels', and checks what they take for granted of a call that is let through.
#include <cstdio>
#include <cstdlib>
#include <random>
#include "logits_internal.h"
static int g_launches = 0;
namespace gdn {
hipError_t launch_adjust_logits(const LogitArgs &a, hipStream_t) {
    ++g_launches;
    // every node and token has a workgroup, the grid is within its limits, and the stretches' parts fit the workspace
    const int rows = logit_rows(a.C, a.N, a.V), chunks = logit_chunks(a.V);
    const long long groups = rows > 0 ? (a.N + rows - 1) / rows : 0;
    if (rows < 1 || rows > a.N || groups * rows < a.N || (long long)chunks * kLogitChunk < a.V || groups > 65535 ||
        logit_workspace_bytes(a.C, a.N, a.V) != (size_t)a.C * a.N * chunks * (kLogitThreads / 64) * 16) {
        std::printf("plan of C %d N %d V %d\n", a.C, a.N, a.V);
        std::abort();
    }
    return hipSuccess;
}
}  // namespace gdn
static std::mt19937_64 rng(5);
static long long R(long long lo, long long hi) { return std::uniform_int_distribution<long long>(lo, hi)(rng); }
static char *F(long long slot) { return reinterpret_cast<char *>(0x100000000000ull + (unsigned long long)slot * (1ull << 42)); }
static void *maybe(void *p) { int r = (int)R(0, 120); if (r == 0) return nullptr; if (r == 1) return (char *)p + 4; if (r == 2) return (char *)p + 1; if (r == 3) return F(0); return p; }
static int32_t *mi(long long s) { return (int32_t *)maybe(F(s)); }
static float *mf(long long s) { return (float *)(R(0, 2) ? maybe(F(s)) : nullptr); }
int main() {
    int counts[9] = {0};
    for (int it = 0; it < 200000; ++it) {
        const bool wild = R(0, 3) == 0;
        gdn_logits_shape s{(int32_t)R(wild ? -1 : 1, wild ? 1100 : 1024), (int32_t)R(wild ? -1 : 1, wild ? 40 : 32), (int32_t)R(wild ? -1 : 1, wild ? 1 << 30 : 2048),
                           (int32_t)R(wild ? -1 : 1, wild ? 0x7fffffff : R(0, 9) ? 300000 : 1 << 24), (int32_t)R(wild ? -1 : 0, wild ? 0x7fffffff : 100000),
                           (int32_t)R(wild ? -1 : 0, wild ? 2000 : 1024), (int32_t)R(wild ? -1 : 0, wild ? 3 : 2), 0};
        s.out_dtype = R(0, 1) ? s.dtype : (int32_t)R(wild ? -1 : 0, wild ? 3 : 0);
        const gdn_logits_shape *sp = R(0, 50) ? &s : nullptr;
        const long long b = R(1, 5);
        gdn_logit_rules u{R(0, 2) ? mi(b) : nullptr, mi(b + 1), R(0, 1) ? mi(b + 2) : nullptr, mf(b + 3), mf(b + 4), mf(b + 5), nullptr, nullptr, mf(b + 8)};
        if (R(0, 1)) { u.bias_tokens = mi(b + 6); u.bias = (float *)maybe(F(b + 7)); }
        const size_t need = gdn_adjust_logits_workspace_size(sp);
        const int r = gdn_adjust_logits(sp, maybe(F(b + 9)), R(0, 9) ? (long long)s.vocab + R(0, 100) : R(-10, 1ll << 50), R(0, 50) ? &u : nullptr,
                                        R(0, 1) ? mi(b + 10) : nullptr, R(0, 1) ? mi(b + 11) : nullptr, R(0, 1) ? mi(b + 12) : nullptr, R(0, 1) ? mi(b + 13) : nullptr,
                                        mi(b + 14), maybe(F(b + 15)), maybe(F(b + 16)), R(0, 9) ? need : need / 2, R(0, 1) ? mi(b + 17) : nullptr, nullptr);
        if (r < 0 || r > 8) { std::printf("unknown return %d\n", r); return 1; }
        ++counts[r];
    }
    std::printf("launches %d; codes:", g_launches);
    for (int k = 0; k < 9; ++k) std::printf(" %d:%d", k, counts[k]);
    std::printf("\n");
    return 0;
}

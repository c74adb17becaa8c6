// Host-only fuzz of the argument validation of gdn_round.h: every entry point with fake (never
// dereferenced) device pointers over random and extreme shapes, strides, NULL, misaligned and
// overlapping arguments, and the page divisor over random and extreme numbers.  Built with the
// sanitizers against stand-in launchers (round_stubs.cpp).
#include <cstdio>
#include <random>
#include "round_internal.h"
extern int g_launches;
static std::mt19937_64 rng(4321);
static long long R(long long lo, long long hi) { return std::uniform_int_distribution<long long>(lo, hi)(rng); }
static char *F(long long slot) { return reinterpret_cast<char *>(0x100000000000ull + (unsigned long long)slot * (1ull << 40)); }
static void *maybe(void *p) { int r = (int)R(0, 40); if (r == 0) return nullptr; if (r == 1) return (char *)p + 4; if (r == 2) return (char *)p + 1; if (r == 3) return F(0); return p; }
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
int main() {
    for (int k = 0; k < 300000; ++k) {  // the quotient is exact up to 2^31 - 1
        const uint32_t d = k < 70000 ? (uint32_t)(k % 65536) + 1 : (uint32_t)R(1, 65536);
        const gdn::Divisor by = gdn::Divisor::of(d);
        const uint32_t q = (uint32_t)R(0, 0x7fffffff / d);
        const uint32_t ts[] = {0x7fffffffu, (uint32_t)R(0, 0x7fffffff), q * d, q * d + (d - 1 < 0x7fffffffu - q * d ? d - 1 : 0), q ? q * d - 1 : 0};
        for (uint32_t t : ts)
            if (by(t) != t / d) { std::printf("%u / %u gave %u\n", t, d, by(t)); return 1; }
    }
    int counts[9] = {0};
    for (int it = 0; it < 200000; ++it) {
        gdn_attn_shape s = shape();
        const gdn_attn_shape *sp = R(0, 50) ? &s : nullptr;
        const gdn_accept_shape as{(int32_t)R(R(0, 9) ? 1 : -1, 1100), (int32_t)R(R(0, 9) ? 1 : -1, 34),
                                  (int32_t)R(0, 9) ? (int32_t)R(1, 300000) : (int32_t)R(-1, 0x7fffffff), (int32_t)R(R(0, 9) ? 0 : -1, R(0, 9) ? 2 : 3)};
        const long long b = R(1, 20);
        int r = 0;
        switch (R(0, 3)) {
        case 0: {
            const gdn_heads_view q = view(b), k = view(b + 1), v = view(b + 2);
            const gdn_rope rope{(const double *)maybe(F(b + 3)), mi(b + 4), R(0, 1) ? mi(b + 5) : nullptr, (int32_t)R(R(0, 5) ? 1 : -1, R(0, 5) ? 3 : 20),
                                (int32_t)(R(0, 3) ? 16 * R(1, 8) : R(-1, 300)), (int32_t)R(0, R(0, 9) ? 1 : 2), (const float *)(R(0, 1) ? maybe(F(b + 6)) : nullptr),
                                nullptr, R(0, 20) ? 1e-6f : -1.f};
            r = gdn_rope_kv_write(sp, (int32_t)R(-1, 3), R(0, 40) ? &q : nullptr, &k, &v, R(0, 40) ? &rope : nullptr, maybe(F(b + 7)), maybe(F(b + 8)),
                                  mi(b + 9), mi(b + 10), mi(b + 11), R(0, 1) ? mi(b + 12) : nullptr, R(0, 1) ? mi(b + 13) : nullptr, maybe(F(b + 14)),
                                  mi(b + 15), nullptr);
            break;
        }
        case 1: {
            const gdn_heads_view g = view(b);
            const size_t need = gdn_paged_attention_workspace_size(sp);
            r = gdn_paged_attention(sp, maybe(F(b + 1)), maybe(F(b + 2)), maybe(F(b + 3)), mi(b + 4), mi(b + 5), mi(b + 6), R(0, 1) ? mi(b + 7) : nullptr,
                                    R(0, 1) ? mi(b + 8) : nullptr, R(0, 20) ? 0.1f : (R(0, 1) ? 0.f : 1e38f * 1e38f), R(0, 1) ? &g : nullptr, (int32_t)R(0, R(0, 9) ? 1 : 2),
                                    maybe(F(b + 9)), maybe(F(b + 10)), R(0, 5) ? need : need / 2, mi(b + 11), nullptr);
            break;
        }
        case 2: {
            const gdn_accept_shape *ap = R(0, 50) ? &as : nullptr;
            const size_t need = gdn_draft_accept_workspace_size(ap);
            const bool greedy = R(0, 2) == 0;
            r = gdn_draft_accept(ap, maybe(F(b)), R(0, 1) ? maybe(F(b + 1)) : nullptr, R(0, 1) ? maybe(F(b + 2)) : nullptr, mi(b + 3),
                                 R(0, 2) ? nullptr : mi(b + 4), R(0, 1) ? mi(b + 5) : nullptr, R(0, 1) ? mi(b + 6) : nullptr,
                                 (const float *)(greedy ? nullptr : maybe(F(b + 7))), (const float *)(greedy ? nullptr : maybe(F(b + 8))), mi(b + 9), mi(b + 10), mi(b + 11),
                                 maybe(F(b + 12)), R(0, 5) ? need : need / 2, mi(b + 13), nullptr);
            break;
        }
        default: {
            const int L = (int)R(R(0, 9) ? 1 : -1, R(0, 9) ? 64 : 70);
            void *k[70], *v[70];
            for (int l = 0; l < 70; ++l) { k[l] = F(b + 30 + 2 * l); v[l] = F(b + 31 + 2 * l); }
            if (R(0, 5) == 0) k[R(0, 63)] = maybe(F(b + 30 + R(0, 100)));
            r = gdn_kv_commit_layers(sp, L, R(0, 30) ? k : nullptr, v, mi(b), mi(b + 1), mi(b + 2), R(0, 1) ? mi(b + 3) : nullptr, R(0, 1) ? mi(b + 4) : nullptr,
                                     mi(b + 5), mi(b + 6), mi(b + 7), nullptr);
        }
        }
        if (r < 0 || r > 8) { std::printf("unknown return %d\n", r); return 1; }
        ++counts[r];
    }
    std::printf("launches %d; codes:", g_launches);
    for (int k = 0; k < 9; ++k) std::printf(" %d:%d", k, counts[k]);
    std::printf("\n");
    return 0;
}

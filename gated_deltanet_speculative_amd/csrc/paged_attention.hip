// Attention over the paged cache of values of the queries' type, for gfx950: the kernels of paged_attention.h, how
// a call is divided over them, and their launches.
#include "paged_attention.h"

namespace gdn {
namespace {

constexpr int kJoinWaves = 4;
// Joins the parts of the cache, in their order: a wave per query row, D / 64 columns a lane.  What there is to
// join stands beside the parts (join_pairs), so that no read waits for another but the first.
template <typename T, int D>
__global__ __launch_bounds__(64 * kJoinWaves) void attn_join_kernel(AttnArgs a, AttnPlan plan) {
    constexpr int W = D / 64, kAhead = 8;  // parts loaded together
    typedef float vw __attribute__((ext_vector_type(W)));
    typedef T tw __attribute__((ext_vector_type(W)));
    const AttnDims &d = a.d;
    const int lane = threadIdx.x & 63, parts = plan.splits;
    const size_t all_rows = (size_t)d.C * d.N * d.Hq, row = (size_t)blockIdx.x * kJoinWaves + (threadIdx.x >> 6);
    if (row >= all_rows) return;
    const float *ml = join_pairs(a, plan) + row * 2, *po = a.workspace + row * D + lane * W;
    vw v[kAhead];
    auto load = [&](int p0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            v[j] = *reinterpret_cast<const vw *>(po + (size_t)min(p0 + j, parts - 1) * all_rows * D);
    };
    load(0);
    const float mine = ml[(size_t)min(lane, parts - 1) * all_rows * 2];
    const float part_sum = lane < parts ? ml[(size_t)lane * all_rows * 2 + 1] : 0.f;
    if (__builtin_amdgcn_ballot_w64(mine != mine)) return;  // an absent row
    float mx = mine;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) mx = fmaxf(mx, __shfl_xor(mx, k));
    // (a part without any attended row has weight 0; NaN sums stay NaN)
    const float wgt = mine == kNegInf ? 0.f : __builtin_amdgcn_exp2f(mine - mx);
    float sum = part_sum == 0.f ? 0.f : part_sum * wgt;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) sum += __shfl_xor(sum, k);
    vw acc = 0.f;
    for (int p0 = 0; p0 < parts; p0 += kAhead) {
        if (p0) load(p0);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const float w = p0 + j < parts ? __shfl(wgt, p0 + j) : 0.f;
            if (w != 0.f) acc += v[j] * w;
        }
    }
    const int per = d.N * d.G, r = (int)(row % per), ch = (int)(row / per), h = ch % d.Hkv, c = ch / d.Hkv;
    const int token = r / d.G, head = h * d.G + r - token * d.G;
    const int64_t node = (int64_t)c * d.N + token;
    acc = sum == 0.f ? vw(0.f) : acc / sum;
    if (a.gate.p && sum != 0.f) {
        const tw z = *reinterpret_cast<const tw *>(static_cast<const T *>(a.gate.p) + node * a.gate.token + head * a.gate.head + lane * W);
#pragma unroll
        for (int i = 0; i < W; ++i) acc[i] = gated(acc[i], (float)z[i], a.gate_mode);
    }
    tw res;
#pragma unroll
    for (int i = 0; i < W; ++i) res[i] = (T)acc[i];
    *reinterpret_cast<tw *>(static_cast<T *>(a.out) + (node * d.Hq + head) * D + lane * W) = res;
}

template <typename T>
void launch_join(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    const size_t rows = (size_t)a.d.C * a.d.N * a.d.Hq;
    const dim3 grid((unsigned)((rows + kJoinWaves - 1) / kJoinWaves)), block(64 * kJoinWaves);
    if (a.d.D == 64)
        hipLaunchKernelGGL((attn_join_kernel<T, 64>), grid, block, 0, stream, a, p);
    else if (a.d.D == 128)
        hipLaunchKernelGGL((attn_join_kernel<T, 128>), grid, block, 0, stream, a, p);
    else
        hipLaunchKernelGGL((attn_join_kernel<T, 256>), grid, block, 0, stream, a, p);
}

}  // namespace

// By the shape alone: the lanes' lengths are on the device, so `held` below is what the page table has room for.  The
// figures are of tables as long as the cache.  Under a wider one more parts are cut than the lengths would give, some
// without a row (one lane of 1003 tokens, 16 / 2 heads of 128: 8 parts, 64 under a table for 128k rows, the join 3.2 us and
// 6.2; trees of 4 x 16 behind 1000: 15.5 us and 17.2), and the bound of 2048 rows on further rounds is one on capacity.
AttnPlan attn_plan(const AttnDims &d) {
    AttnPlan p;
    const int row_bytes = d.D * (d.dtype == GDN_DTYPE_F32 ? 4 : 2);
    const int64_t rows = (int64_t)d.N * d.G;
    const bool few = rows <= kFewRows && row_bytes < 1024, wide = row_bytes >= 512, f32 = d.dtype == GDN_DTYPE_F32;
    // Wide float32 rows take 64 query rows, four waves of up to 512 registers: within 256, the outputs, queries and
    // staged rows of a wave do not fit (31 nodes, 4 heads each, D = 256, 136 rows: 52 us with 128 query rows, 28 with
    // 64; two lanes of 73 nodes at 1.4k 196 and 98).  Rows of 512 bytes do nearly fit, and a long prompt's share of
    // loads then counts for more (D = 128: 92 query rows 23 us and 18; 5296 of them at 870 rows 245 us and 288).
    p.rows_per_group = few ? kFewRows
                       : row_bytes == 1024 || (wide ? f32 && rows <= 128 : rows <= 64) ? 64
                       : wide || f32 || rows <= 128 ? 128 : 256;
    p.tiles = (int)((rows + p.rows_per_group - 1) / p.rows_per_group);
    const int64_t groups = (int64_t)d.C * d.Hkv * p.tiles;
    // the least cache rows of a part: a short cache is otherwise read by few workgroups, one tile after another (426
    // nodes, 8 heads, D = 256, 151 rows: 36 us with parts of 256 rows, 32 with 128; float32, 31 nodes at 136: 109 and,
    // with 64, 52)
    const int64_t least = few ? few_tile(row_bytes, false) * kFewWaves : f32 ? 64 : 128;
    const int64_t held = (int64_t)d.max_pages * d.page.d, most = std::min<int64_t>((held + least - 1) / least, 64);
    // One round of workgroups: one of eight waves, or of four that hold more than 256 registers, fills a CU, two others
    // do.  Not one more: a round of few costs as much as a full one (rounded up, to 512 in every kernel, against this:
    // three lanes of 710 nodes, 4 heads each, D = 64: 62 us and 35; 21 nodes of 4, D = 256, six lanes at 19k 289 and
    // 201; 24 nodes of 8, D = 128, seven lanes at 7.6k 41 and 31).
    const int64_t round = p.rows_per_group >= 128 || (f32 && p.rows_per_group == 64) ? 256 : 512;
    auto rounds = [&](int64_t s) { return (groups * s + round - 1) / round; };
    int64_t s = groups < round ? round / groups : 1;
    s = s > most ? most : s;
    // More rounds of shorter parts where they leave the last one fuller, by 15% and more, and the parts are long beside
    // what writing and joining one costs (42 lanes of 32 nodes, 4 heads each, D = 128, at 11k: 410 us and 364; 2278
    // nodes of 8 at 2k, D = 256, float32 2000 and 1550; but 710 nodes of D = 64 without the bound of 2048 rows 35 and 62;
    // float32 products cost eight times as much a row).
    for (int64_t more = s + 1; more <= most && (f32 ? 192 : 2048) * more <= held && groups * more <= 4 * round; ++more)
        if (20 * rounds(more) * s < 17 * rounds(s) * more) s = more;
    p.splits = (int)s;
    return p;
}

hipError_t launch_attention_join(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    if (a.d.dtype == GDN_DTYPE_BF16)
        launch_join<__bf16>(a, p, stream);
    else if (a.d.dtype == GDN_DTYPE_F16)
        launch_join<_Float16>(a, p, stream);
    else
        launch_join<float>(a, p, stream);
    return hipGetLastError();
}

hipError_t launch_paged_attention(const AttnArgs &a, hipStream_t stream) {
    return launch_attention<false>(a, attn_plan(a.d), stream);
}

}  // namespace gdn

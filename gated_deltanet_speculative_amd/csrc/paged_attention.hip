// Attention over the paged cache of values of the queries' type, for gfx950: the kernels of paged_attention.h, how
// a call is divided over them, and their launches.
#include "paged_attention.h"

namespace gdn {
namespace {

template <typename T, int D, int BM>
__global__ __launch_bounds__(64 * group_waves(BM), group_blocks(sizeof(T), BM)) void attn_rows_kernel(AttnArgs a, AttnPlan plan) {
    attn_rows<T, D, BM, false>(a, plan);
}
template <typename T>
__global__ __launch_bounds__(kPairThreads, 2) void attn_pair_kernel(AttnArgs a, AttnPlan plan) {
    attn_pair<T, false>(a, plan);
}
template <typename T, int D>
__global__ __launch_bounds__(64 * kFewWaves, 2) void attn_few_kernel(AttnArgs a, AttnPlan plan) {
    attn_few<T, D, false>(a, plan);
}
template <typename T, int D>
__global__ __launch_bounds__(64 * kJoinWaves) void attn_join_kernel(AttnArgs a, AttnPlan plan) {
    attn_join<T, D>(a, plan);
}

template <typename T, int D, int BM>
void launch_rows(const AttnArgs &a, const AttnPlan &p, unsigned units, hipStream_t stream) {
    const dim3 grid(p.tiles > 1 ? (units + 7) / 8 * 8 : units);
    hipLaunchKernelGGL((attn_rows_kernel<T, D, BM>), grid, dim3(64 * group_waves(BM)), 0, stream, a, p);
}

template <typename T, int D>
hipError_t launch(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    constexpr int RB = D * sizeof(T);
    const unsigned units = (unsigned)a.d.C * a.d.Hkv * p.tiles * p.splits;
    if constexpr (RB < 1024)
        if (p.rows_per_group == kFewRows)
            hipLaunchKernelGGL((attn_few_kernel<T, D>), dim3(units), dim3(64 * kFewWaves), 0, stream, a, p);
    if constexpr (RB < 512 || sizeof(T) == 4)
        if (p.rows_per_group == 64) launch_rows<T, D, 64>(a, p, units, stream);
    if constexpr (RB < 512 && sizeof(T) == 2)
        if (p.rows_per_group == 256) launch_rows<T, D, 256>(a, p, units, stream);
    if constexpr (D == 256 && sizeof(T) == 2) {
        if (p.rows_per_group == kPairRows)
            hipLaunchKernelGGL((attn_pair_kernel<T>), dim3(p.tiles > 1 ? (units + 7) / 8 * 8 : units), dim3(kPairThreads), 0,
                               stream, a, p);
    } else if constexpr (RB < 1024) {
        if (p.rows_per_group == 128) launch_rows<T, D, 128>(a, p, units, stream);
    }
    if (p.splits > 1) {
        const size_t rows = (size_t)a.d.C * a.d.N * a.d.Hq;
        hipLaunchKernelGGL((attn_join_kernel<T, D>), dim3((unsigned)((rows + kJoinWaves - 1) / kJoinWaves)),
                           dim3(64 * kJoinWaves), 0, stream, a, p);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    if (a.d.D == 64) return launch<T, 64>(a, p, stream);
    if (a.d.D == 128) return launch<T, 128>(a, p, stream);
    return launch<T, 256>(a, p, stream);
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

hipError_t launch_paged_attention(const AttnArgs &a, hipStream_t stream) {
    const AttnPlan p = attn_plan(a.d);
    if (a.d.dtype == GDN_DTYPE_BF16) return launch_t<__bf16>(a, p, stream);
    if (a.d.dtype == GDN_DTYPE_F16) return launch_t<_Float16>(a, p, stream);
    return launch_t<float>(a, p, stream);
}

}  // namespace gdn

// Attention over the paged cache of 4-bit values, for gfx950: the kernels of paged_attention.h with rows that become
// values of the queries' type on their way into LDS (many query rows) or into an operand (few), how a call is divided
// over them, and their launches.
//
// What bounds them: many query rows the products and the softmax, as over 16 bits (two chunks of 2048 behind 16k, D = 256,
// bfloat16: 1243 us, 734 TFLOP/s, and 1270 over a 16-bit cache); 17 to 64 rows the tiles' chain of load, conversion, LDS
// and products, with two waves a SIMD to cover it (trees of 4 x 16 nodes behind 8192, 32 / 8 heads of 128: 25 us for 19 MB
// and 8.6 GFLOP, and 5.4 for the join; over 16 bits 34); few rows the bytes.
#include "paged_attention.h"

namespace gdn {
namespace {

// Workgroups of the kernel for few rows a CU.  Float32 rows of 256 values: one, whose waves use 414 registers; within the 256
// of two, 95 of them go through memory (ragged lanes, D = 256, with two and with one: 32 of decode up to 8192 tokens 639 us
// and 308, five of eight nodes up to 2999 97 and 51, one of decode at 1000 20.5 and 15.7).  Narrower ones keep two, with 15
// to 25 registers in memory (the 32 lanes at D = 128 106 us and 133, at D = 64 55 and 69).
constexpr int few_blocks(int row_bytes) { return row_bytes == 1024 ? 1 : 2; }

template <typename T, int D, int BM>
__global__ __launch_bounds__(64 * group_waves(BM), group_blocks(sizeof(T), BM)) void attn_rows_kv4_kernel(AttnArgs a, AttnPlan plan) {
    attn_rows<T, D, BM, true>(a, plan);
}
template <typename T>
__global__ __launch_bounds__(kPairThreads, 2) void attn_pair_kv4_kernel(AttnArgs a, AttnPlan plan) {
    attn_pair<T, true>(a, plan);
}
template <typename T, int D>
__global__ __launch_bounds__(64 * kFewWaves, few_blocks(D * sizeof(T))) void attn_few_kv4_kernel(AttnArgs a, AttnPlan plan) {
    attn_few<T, D, true>(a, plan);
}
template <typename T, int D>
__global__ __launch_bounds__(64 * kJoinWaves) void attn_join_kv4_kernel(AttnArgs a, AttnPlan plan) {
    attn_join<T, D>(a, plan);
}

template <typename T, int D, int BM>
void launch_rows(const AttnArgs &a, const AttnPlan &p, unsigned units, hipStream_t stream) {
    const dim3 grid(p.tiles > 1 ? (units + 7) / 8 * 8 : units);
    hipLaunchKernelGGL((attn_rows_kv4_kernel<T, D, BM>), grid, dim3(64 * group_waves(BM)), 0, stream, a, p);
}

template <typename T, int D>
hipError_t launch(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    constexpr int RB = D * sizeof(T);
    const unsigned units = (unsigned)a.d.C * a.d.Hkv * p.tiles * p.splits;
    if (p.rows_per_group == kFewRows)
        hipLaunchKernelGGL((attn_few_kv4_kernel<T, D>), dim3(units), dim3(64 * kFewWaves), 0, stream, a, p);
    if constexpr (RB < 512 || sizeof(T) == 4)
        if (p.rows_per_group == 64) launch_rows<T, D, 64>(a, p, units, stream);
    if constexpr (RB < 512 && sizeof(T) == 2)
        if (p.rows_per_group == 256) launch_rows<T, D, 256>(a, p, units, stream);
    if constexpr (D == 256 && sizeof(T) == 2) {
        if (p.rows_per_group == kPairRows)
            hipLaunchKernelGGL((attn_pair_kv4_kernel<T>), dim3(p.tiles > 1 ? (units + 7) / 8 * 8 : units), dim3(kPairThreads), 0,
                               stream, a, p);
    } else if constexpr (RB < 1024) {
        if (p.rows_per_group == 128) launch_rows<T, D, 128>(a, p, units, stream);
    }
    if (p.splits > 1) {
        const size_t rows = (size_t)a.d.C * a.d.N * a.d.Hq;
        hipLaunchKernelGGL((attn_join_kv4_kernel<T, D>), dim3((unsigned)((rows + kJoinWaves - 1) / kJoinWaves)),
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

// As attn_plan, but for two things.  Up to 16 query rows take the kernel for few in every type, float32 rows of 1024 bytes
// too: its tiles of K are codes, of the same size for all types.  And workgroups of four waves, two of which fill a CU, are
// divided into one for each CU instead where they would have no more than 256 cache rows: what a workgroup does before and
// after its tiles then costs more than the second one hides (trees of 16 nodes, 4 heads each, 8 kv heads of 128, bfloat16,
// with two and with one: a lane at 8192 tokens 22.6 us and 18.5, three at 3000 22.1 and 18.4, four at 2000 19.0 and 17.5,
// eight at 1000 20.0 and 17.8, twelve at 1000 22.2 and 22.8; but four at 8192, 512 rows, 29.0 and 31.7).
AttnPlan attn_plan_kv4(const AttnDims &d) {
    const int row_bytes = d.D * (d.dtype == GDN_DTYPE_F32 ? 4 : 2);
    const int64_t rows = (int64_t)d.N * d.G, held = (int64_t)d.max_pages * d.page.d, groups = (int64_t)d.C * d.Hkv;
    if (rows > kFewRows) {
        AttnPlan p = attn_plan(d);
        if (p.rows_per_group == 64 && d.dtype != GDN_DTYPE_F32 && held <= 256 * p.splits)
            p.splits = (int)std::min<int64_t>(p.splits, std::max<int64_t>(256 / groups, 1));
        return p;
    }
    AttnPlan p{kFewRows, 1, 1};
    const int64_t least = few_tile(row_bytes, true) * kFewWaves, most = std::min<int64_t>((held + least - 1) / least, 64);
    const int64_t round = 256 * few_blocks(row_bytes);  // of workgroups
    p.splits = (int)std::min<int64_t>(most, groups < round ? round / groups : 1);
    return p;
}

hipError_t launch_paged_attention_kv4(const AttnArgs &a, hipStream_t stream) {
    const AttnPlan p = attn_plan_kv4(a.d);
    if (a.d.dtype == GDN_DTYPE_BF16) return launch_t<__bf16>(a, p, stream);
    if (a.d.dtype == GDN_DTYPE_F16) return launch_t<_Float16>(a, p, stream);
    return launch_t<float>(a, p, stream);
}

}  // namespace gdn

// Attention over the paged cache of 4-bit values, for gfx950: the kernels of paged_attention.h with rows that become
// values of the queries' type on their way into LDS (many query rows) or into an operand (few), how a call is divided
// over them, and their launches.
//
// What bounds them: many query rows the products and the softmax, as over 16 bits (two chunks of 2048 behind 16k, D = 256,
// bfloat16: 1226 us, 726 TFLOP/s, and 1277 over a 16-bit cache); 17 to 64 rows the tiles' chain of load, conversion, LDS
// and products, with two waves a SIMD to cover it (trees of 4 x 16 nodes behind 8192, 32 / 8 heads of 128: 24 us for 19 MB
// and 8.6 GFLOP, and 5.4 for the join; over 16 bits 36); few rows the bytes.
#define GDN_ATTN_PAIR __device__ __forceinline__ void attn_pair
#include "paged_attention.h"

namespace gdn {
namespace {

template <typename T, bool kFour>
__global__ __launch_bounds__(kPairThreads, 2) void attn_pair_kernel(AttnArgs a, AttnPlan plan) {
    attn_pair<T, kFour>(a, plan);
}

}  // namespace

// As attn_plan, but for two things.  Up to 16 query rows take the kernel for few in every type, float32 rows of 1024 bytes
// too: its tiles of K are codes, of the same size for all types.  And workgroups of four waves, two of which fill a CU, are
// divided into one for each CU instead where they would have no more than 256 cache rows: what a workgroup does before and
// after its tiles then costs more than the second one hides (trees of 16 nodes, 4 heads each, 8 kv heads of 128, bfloat16,
// with two and with one: a lane at 8192 tokens 22.6 us and 18.5, three at 3000 22.1 and 18.4, four at 2000 19.0 and 17.5,
// eight at 1000 20.0 and 17.8, twelve at 1000 22.2 and 22.8; but four at 8192, 512 rows, 29.0 and 31.7).  As in attn_plan what is
// held is the page table's width: under one for 128k rows there are always two (the lane at 8192 22.5 us and, under a table as
// long as the cache, 18.6; trees of 4 x 16 at 1000 17.1 and 15.0; one lane of decode at 1003, with 64 parts for 4, 13.9 and 10.5).
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
    const int64_t round = 256 * few_blocks(row_bytes, true);  // of workgroups
    p.splits = (int)std::min<int64_t>(most, groups < round ? round / groups : 1);
    return p;
}

hipError_t launch_paged_attention_kv4(const AttnArgs &a, hipStream_t stream) {
    return launch_attention<true>(a, attn_plan_kv4(a.d), stream);
}

}  // namespace gdn

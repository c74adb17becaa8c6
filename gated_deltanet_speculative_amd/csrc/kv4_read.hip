// Rows of 4-bit caches as values, for gfx950: every layer's rows first .. first + N_c - 1 of the lanes' slots.
//
// Bound by bytes: 0.53 bytes of a value read and 2 or 4 written.  A lane carries 8 values (a word of codes): D / 8 lanes
// a row, consecutive (row, head) pairs in the output's order, so that stores are whole lines.  A workgroup takes
// either K or V, and finds its tokens' pages first, one thread a token; four rows of a thread are in flight.
//
// 4095 rows of 16 layers, 8 heads of 128, float16: 70 us, 4.9 TB/s (K and V in one workgroup, one row of a thread at a time: 76);
// 64 lanes of 32 rows of 16 layers, 8 heads of 128: 41.1 us, 4.1 TB/s (46.6); 64 rows of a layer: 4.0 us (6.8).
#include "round_device.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;  // tokens of a workgroup
constexpr int kAhead = 4;     // rows of a thread that are requested together

template <typename T>
__device__ inline void four_out(T *p, int w, unsigned scale) {
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h) reinterpret_cast<v4i *>(p)[h] = four_values<T>(w, scale, h);
}

// Grid: (tokens / kTokens, lanes, 2 layers + (K or V)).
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(AttnDims d, Cache4Layers cl, PagedLanes l,
                                                            const int32_t *__restrict__ first_row, T *__restrict__ k_out,
                                                            T *__restrict__ v_out) {
    constexpr int LPR = D / 8, kStep = kThreads / LPR;  // lanes a row, rows a round
    __shared__ int s_row[kTokens];                      // cache row of a token for kv head 0, -1 without a page
    const int tid = threadIdx.x, c = blockIdx.y, layer = blockIdx.z >> 1, side = blockIdx.z & 1, i0 = blockIdx.x * kTokens;
    const int slot = l.slot_ids[c], nodes = l.lane_nodes ? l.lane_nodes[c] : d.N, first = first_row[c];
    if (slot == -1) return;
    int bits = 0;
    if (nodes < 0 || nodes > d.N) bits |= GDN_STATUS_NODES;
    if (slot < -1 || slot >= d.P) bits |= GDN_STATUS_SLOT_RANGE;
    if (first < 0 || (int64_t)first + max(nodes, 0) > (int64_t)d.max_pages * d.page.d) bits |= GDN_STATUS_LENGTH;
    if (bits) {
        if (tid == 0 && i0 == 0 && blockIdx.z == 0 && l.status) atomicOr(l.status, bits);
        return;
    }
    const int n = min(nodes - i0, kTokens);
    if (n <= 0) return;
    if (tid < n) {
        const uint32_t t = (uint32_t)(first + i0 + tid), entry = d.page(t);
        const int pid = l.page_table[(int64_t)slot * d.max_pages + entry];
        const bool paged = (unsigned)pid < (unsigned)d.n_pages;
        s_row[tid] = paged ? (int)cache_row(d, pid, 0, t, entry) : -1;
        if (!paged && blockIdx.z == 0 && l.status) atomicOr(l.status, GDN_STATUS_PAGE);
    }
    T *out = side ? v_out : k_out;
    if (!out) return;
    lds_barrier();
    const int *codes = static_cast<const int *>(side ? cl.codes.v[layer] : cl.codes.k[layer]);
    const unsigned char *scales = static_cast<const unsigned char *>(side ? cl.scales.v[layer] : cl.scales.k[layer]);
    out += (((size_t)layer * d.C + c) * d.N + i0) * d.Hkv * D;
    // this thread's rows (token, head), kStep apart
    const int sub = tid % LPR, rows = n * d.Hkv, step_i = kStep / d.Hkv, step_h = kStep - step_i * d.Hkv;
    int r = tid / LPR, i = r / d.Hkv, h = r - i * d.Hkv;
    while (r < rows) {
        int w[kAhead], at[kAhead];
        unsigned s[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int row = r < rows ? s_row[i] : -1;
            at[j] = row < 0 ? -1 : r;
            const size_t from = (size_t)max(row, 0) + (size_t)(row < 0 ? 0 : h) * d.page.d;
            w[j] = codes[from * LPR + sub];
            s[j] = scales[from * (D / 32) + sub / 4];
            r += kStep;
            i += step_i;
            h += step_h;
            if (h >= d.Hkv) h -= d.Hkv, ++i;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (at[j] >= 0) four_out<T>(out + (size_t)at[j] * D + 8 * sub, w[j], s[j]);
    }
}

template <typename T>
hipError_t launch(const AttnDims &d, int n_layers, const Cache4Layers &cl, const PagedLanes &l, const int32_t *first_row,
                  void *k_out, void *v_out, hipStream_t stream) {
    const dim3 grid((d.N + kTokens - 1) / kTokens, d.C, 2 * n_layers);
    T *k = static_cast<T *>(k_out), *v = static_cast<T *>(v_out);
    if (d.D == 64)
        hipLaunchKernelGGL((kv4_read_kernel<T, 64>), grid, dim3(kThreads), 0, stream, d, cl, l, first_row, k, v);
    else if (d.D == 128)
        hipLaunchKernelGGL((kv4_read_kernel<T, 128>), grid, dim3(kThreads), 0, stream, d, cl, l, first_row, k, v);
    else
        hipLaunchKernelGGL((kv4_read_kernel<T, 256>), grid, dim3(kThreads), 0, stream, d, cl, l, first_row, k, v);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_read(const AttnDims &d, int n_layers, const Cache4Layers &cl, const PagedLanes &l,
                           const int32_t *first_row, void *k_out, void *v_out, hipStream_t stream) {
    if (d.dtype == GDN_DTYPE_BF16) return launch<__bf16>(d, n_layers, cl, l, first_row, k_out, v_out, stream);
    if (d.dtype == GDN_DTYPE_F16) return launch<_Float16>(d, n_layers, cl, l, first_row, k_out, v_out, stream);
    return launch<float>(d, n_layers, cl, l, first_row, k_out, v_out, stream);
}

}  // namespace gdn

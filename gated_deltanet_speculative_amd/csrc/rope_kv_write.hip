// Rotary positions of the round's queries and keys and the write of keys and values into the
// slot's pages, for gfx950.
//
// Mathematics.  Pair j of a head's first 2 * half values turns by the angle
// phi = position[axis_j] * inv_freq_j:  (a, b) -> (a cos phi - b sin phi, b cos phi + a sin phi),
// after an optional x * rsqrt(mean(x^2) + eps) * w over the head.  Positions reach 10^6 and more,
// where a 32-bit angle is off by up to 0.03 rad: the product and its reduction to a fraction of a
// turn are done in 64 bits (two multiplications and a rint per pair), the sine and cosine of the
// remainder in 32.
//
// Bound by the bytes of q, k, v (read) and q_out, K, V rows (written); a decode step by the chain of
// dependent reads.  A workgroup takes one token at a time: its rows are requested first (the first token's ahead of
// the lane's checks), its threads compute the half cosines and sines once into LDS, and groups of D / 8
// lanes, 8 values a lane, then carry one head each; a pair (j, j + half) lies half / 8 lanes
// apart (rot_dim is a multiple of 16), its partner comes by a lane shuffle.
//
// A 4-bit cache takes the rotated rows quantised, a block of 32 values held by four adjacent lanes: the block's
// largest magnitude is the largest of the values' bit patterns without the sign (as integers, NaN above infinity), adding a quarter
// of its power of two to it carries into the exponent exactly where it rounds up to the next one, and the conversion
// instruction rounds the codes to nearest even and saturates.
//
// 2 x 4096 tokens, 16 + 2 + 2 heads of 256, three axes, norms, float32 to bfloat16: 65.3 us, 3.9 TB/s (a copy of as many
// bytes 53 us); 4 tokens of 32 + 8 + 8 heads of 128: 5.9 us.  The same into a 4-bit cache: 71.8 us, 3.3 TB/s (a copy 47 us; the
// waves that quantise take longest, and the rotation's work is no less for fewer bytes), and 6.0 us.
#include <type_traits>

#include "round_device.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// Eight values of a head as they are loaded
template <typename T>
struct Raw8 {
    typedef T t __attribute__((ext_vector_type(16 / sizeof(T))));
    static constexpr int W = 16 / sizeof(T);
    t v[8 / W];
    __device__ void load(const T *p) {
#pragma unroll
        for (int b = 0; b < 8 / W; ++b) v[b] = *reinterpret_cast<const t *>(p + b * W);
    }
    __device__ void get(float (&x)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)v[e / W][e % W];
    }
};
template <typename T>
__device__ inline void store8(T *p, const float (&x)[8]) {
    typedef T t __attribute__((ext_vector_type(16 / sizeof(T))));
    constexpr int W = 16 / sizeof(T);
#pragma unroll
    for (int b = 0; b < 8; b += W) {
        t v;
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = (T)x[b + e];
        *reinterpret_cast<t *>(p + b) = v;
    }
}

// Eight values as codes, and the scale of their block of 32 in this lane and three neighbours (every lane of the wave calls it)
struct Quantised {
    int codes;
    unsigned scale;
};
template <typename T>
__device__ inline Quantised quantised(const float (&x)[8]) {
    constexpr int kMost = std::is_same_v<T, _Float16> ? 140 : 252;  // 6 * 2^(kMost - 127) is finite in the type
    unsigned m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
    m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));  // lane ^ 1
    m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));  // lane ^ 2
    if (m >= 0x7f800000u) return Quantised{0, 255u};
    const unsigned scale = (unsigned)min(max((int)((m + 0x200000u) >> 23) - 2, 2), kMost);
    const float s = __uint_as_float(scale << 23);
    unsigned w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
    return Quantised{(int)w, scale};
}

constexpr int kAhead = 3;  // rounds of rows requested together: 48 rows of 128, 24 of 256

// Over 4 bits four workgroups a CU, as the other has by itself (as this was chosen, 2 x 4096 tokens with 141 registers 94 us and with
// 128 78): from float32 two registers are in memory at D = 64 and 128.  The text is the kernel itself: as a function that the
// kernels call, the prompt takes 66.2 us and 65.4 over values, and with its rows read 83.1 and 76.2 over 4 bits.
template <typename X, typename T, int D, bool kFour>
__global__ __launch_bounds__(kThreads, kFour ? 4 : 1) void rope_kv_write_kernel(RopeArgs a) {
    constexpr int LPR = D / 8, RPB = kThreads / LPR;  // lanes per head row, rows a workgroup carries at a time
    __shared__ float s_cos[2][D / 2], s_sin[2][D / 2];
    __shared__ int s_bits;
    const AttnDims &d = a.d;
    const int tid = threadIdx.x, sub = tid % LPR, first_row = tid / LPR, c = blockIdx.y;
    const int rows = d.Hq + 2 * d.Hkv;

    // Rows of q, k and v of node i, from row0 on, requested together (past the last row: that one again)
    Raw8<X> raw[kAhead];
    auto request = [&](int64_t node, int row0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int row = min(row0 + first_row + RPB * j, rows - 1);
            const int kind = row < d.Hq ? 0 : row < d.Hq + d.Hkv ? 1 : 2;  // q, k, v
            const HeadsView &v = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
            const int h = kind == 0 ? row : kind == 1 ? row - d.Hq : row - d.Hq - d.Hkv;
            raw[j].load(static_cast<const X *>(v.p) + node * v.token + h * v.head + 8 * sub);
        }
    };
    request((int64_t)c * d.N + blockIdx.x, 0);  // (every node has its rows, present or not)

    const Lane ln = paged_lane(d, a.l, c);
    if (ln.slot == -1) return;
    // ---- the lane's checks; every workgroup of the lane comes to the same verdict
    int bits = ln.bits;
    if (!(bits & GDN_STATUS_SLOT_RANGE) && slot_shared(a.l.slot_ids, d.C, c, ln.slot, tid, kThreads))
        bits |= GDN_STATUS_SLOT_DUP;
    const int axis = a.pair_axis && tid < a.half ? a.pair_axis[tid] : 0;
    if ((unsigned)axis >= (unsigned)a.n_axes) bits |= GDN_STATUS_AXIS;
    const double freq = tid < a.half ? a.inv_freq[tid] * 0.15915494309189533577 : 0.0;  // turns per position
    unsigned anc = 0;
    if (a.l.parents && !(bits & GDN_STATUS_NODES)) {
        bool bad;
        anc = tree_ancestors(a.l.parents + (int64_t)c * d.N, ln.nodes, bad);
        if (bad) bits |= GDN_STATUS_PARENT;
    }
    if (tid == 0) s_bits = 0;
    lds_barrier();
    if (bits) atomicOr(&s_bits, bits);
    lds_barrier();
    bits = s_bits;
    if (bits) {
        if (tid == 0 && blockIdx.x == 0 && a.l.status) atomicOr(a.l.status, bits);
        return;
    }

    int buf = 0;
    for (int i = blockIdx.x; i < ln.nodes; i += gridDim.x, buf ^= 1) {
        const int64_t node = (int64_t)c * d.N + i;
        const uint32_t t = ln.len + i, entry = d.page(t);
        const int pid = a.l.page_table[(int64_t)ln.slot * d.max_pages + entry];
        const bool paged = (unsigned)pid < (unsigned)d.n_pages;
        const int depth = a.l.parents ? __popc(__shfl(anc, i & 63)) - 1 : i;
        if (tid < a.half) {
            const int pos = a.positions ? a.positions[node * a.n_axes + axis] : ln.len + depth;
            const double turns = (double)pos * freq;  // its fraction in [-1/2, 1/2] is the angle
            sincospif(2.0f * (float)(turns - rint(turns)), &s_sin[buf][tid], &s_cos[buf][tid]);
        }
        if (!paged && tid == 0 && a.l.status) atomicOr(a.l.status, GDN_STATUS_PAGE);
        lds_barrier();  // (one a node: the next node's go to the other half)
        const float *cs = s_cos[buf], *sn = s_sin[buf];
        for (int row0 = 0; row0 < rows; row0 += RPB * kAhead) {
            if (row0) request(node, row0);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (row0 + RPB * j >= rows) break;  // (the same for every thread)
                const int row = row0 + first_row + RPB * j;
                const bool has = row < rows;
                const int kind = row < d.Hq ? 0 : row < d.Hq + d.Hkv ? 1 : 2;
                const int h = kind == 0 ? row : kind == 1 ? row - d.Hq : row - d.Hq - d.Hkv;
                float x[8];
                raw[j].get(x);
                if (a.q_norm || a.k_norm) {  // (the sums of rows without a norm are not used)
                    const float *w = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
                    float sq = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
#pragma unroll
                    for (int k = 1; k < LPR; k <<= 1) sq += __shfl_xor(sq, k);
                    if (w) {
                        const float r = 1.0f / sqrtf(sq * (1.0f / D) + a.eps);
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[8 * sub + e];
                    }
                }
                if (a.interleaved) {
                    if (kind < 2 && 8 * sub < 2 * a.half)
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float co = cs[4 * sub + e / 2], si = sn[4 * sub + e / 2], u = x[e], z = x[e + 1];
                            x[e] = u * co - z * si;
                            x[e + 1] = z * co + u * si;
                        }
                } else {
                    const int hl = a.half / 8;  // lanes of one half
                    const bool first = sub < hl, turns = sub < 2 * hl;
                    const int from = (tid & 63) + (first ? hl : turns ? -hl : 0), at = turns ? 8 * (first ? sub : sub - hl) : 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y = __shfl(x[e], from), co = cs[at + e], si = first ? -sn[at + e] : sn[at + e];
                        x[e] = kind < 2 && turns ? x[e] * co + y * si : x[e];
                    }
                }
                Quantised four{};
                if constexpr (kFour)
                    if (__builtin_amdgcn_ballot_w64(kind > 0)) four = quantised<T>(x);
                if (!has) continue;
                if (kind == 0) {
                    store8(static_cast<T *>(a.q_out) + (node * d.Hq + h) * D + 8 * sub, x);
                } else if (paged && kFour) {
                    const size_t at = cache_row(d, pid, h, t, entry);
                    static_cast<int *>(kind == 1 ? a.k_cache : a.v_cache)[at * (D / 8) + sub] = four.codes;
                    if (sub % 4 == 0)
                        static_cast<unsigned char *>(kind == 1 ? a.k_scales : a.v_scales)[at * (D / 32) + sub / 4] = (unsigned char)four.scale;
                } else if (paged) {
                    T *cache = static_cast<T *>(kind == 1 ? a.k_cache : a.v_cache);
                    store8(cache + (size_t)cache_row(d, pid, h, t, entry) * D + 8 * sub, x);
                }
            }
        }
        if (i + (int)gridDim.x < ln.nodes) request(node + gridDim.x, 0);
    }
}

template <typename X, typename T, int D>
void launch_d(const RopeArgs &a, dim3 grid, hipStream_t stream) {
    if (a.k_scales)
        hipLaunchKernelGGL((rope_kv_write_kernel<X, T, D, true>), grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((rope_kv_write_kernel<X, T, D, false>), grid, dim3(kThreads), 0, stream, a);
}

template <typename X, typename T>
hipError_t launch(const RopeArgs &a, hipStream_t stream) {
    // one round of workgroups (124 registers: four of them a CU), each with several nodes of a long chunk: 2x4096
    // tokens, as this was chosen, 68.6 us, with 2048 70.2, 4096 74.8, 8192 82.8
    const int most = (1024 + a.d.C - 1) / a.d.C;
    const dim3 grid(a.d.N < most ? a.d.N : most, a.d.C);
    if (a.d.D == 64)
        launch_d<X, T, 64>(a, grid, stream);
    else if (a.d.D == 128)
        launch_d<X, T, 128>(a, grid, stream);
    else
        launch_d<X, T, 256>(a, grid, stream);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_kv_write(const RopeArgs &a, hipStream_t stream) {
    const bool wide = a.x_dtype == GDN_DTYPE_F32;
    if (a.d.dtype == GDN_DTYPE_BF16) return wide ? launch<float, __bf16>(a, stream) : launch<__bf16, __bf16>(a, stream);
    if (a.d.dtype == GDN_DTYPE_F16) return wide ? launch<float, _Float16>(a, stream) : launch<_Float16, _Float16>(a, stream);
    return launch<float, float>(a, stream);
}

}  // namespace gdn

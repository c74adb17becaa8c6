// Penalties, biases and masks on the logits after every node of a draft, and the probabilities at a temperature, for
// gfx950.
//
// A workgroup takes a stretch of the vocabulary for some nodes of one lane.  What a token's occurrences do to its
// logit hangs on the token alone, but for the nodes' own tokens: the workgroup counts its stretch's tokens in
// the slot's history once into LDS (a word a token: occurrences behind the prompt, and flags), a thread takes the
// words of its tokens into registers, and every row then costs one read and a few operations a value.  The nodes'
// own tokens, at most 32, carry a flag and are counted along the path where they are met.
//
// Probabilities take two passes over the logits: the first leaves every wave's maximum and sum of exponentials of
// a row, the second joins them and computes each value again (reading a logit twice costs less than writing
// it in 32 bits and reading that).  Bound by bytes where there are many rows, by the chain slot, history,
// LDS, logits and by launches where there are few.
#include "logits_internal.h"
#include "round_device.h"

namespace gdn {
namespace {

constexpr int kThreads = kLogitThreads, kWaves = kThreads / 64;
constexpr float kNegInf = -__builtin_inff();

// Flags of a token's word above its count (at most 2^20 entries of history)
constexpr unsigned kCount = (1u << 24) - 1u, kPrompt = 1u << 24, kBias = 1u << 25, kDraft = 1u << 26;

enum { kLogits, kStats, kProbabilities };  // what a launch leaves

// A (value, index) pair of which the larger value, then the lower index, wins; NaN never does.
struct Best {
    float v;
    int x;
};
__device__ inline Best better(Best a, Best b) { return b.v > a.v || (b.v == a.v && b.x < a.x) ? b : a; }
__device__ inline Best wave_best(Best b) {
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) b = better(b, Best{__shfl_xor(b.v, k), __shfl_xor(b.x, k)});
    return b;
}
__device__ inline float wave_sum(float x) {
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) x += __shfl_xor(x, k);
    return x;
}
// log2(e) / T within the normal numbers: finite for T = 0, and never 0, so that -infinity times it is -infinity
__device__ inline float per_temperature(float temp) { return fminf(fmaxf(1.4426950408889634f / temp, 0x1p-126f), 3.4e38f); }
// e^{(z - m) / T} with k = log2(e) / T; 1 at the maximum even where that is infinite, 0 for -infinity
__device__ inline float weight(float z, float m, float k) {
    const float top = m == kNegInf ? 0.f : m;
    return __builtin_amdgcn_exp2f(z == top ? 0.f : (z - top) * k);
}

template <typename T, typename O, int W, int MODE>
__global__ __launch_bounds__(kThreads) void adjust_logits_kernel(LogitArgs a) {
    constexpr int VEC = 16 / sizeof(T), GR = W / VEC, kChunk = kThreads * W;
    typedef T tv __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
    typedef O ov __attribute__((ext_vector_type(VEC), aligned(sizeof(O))));
    typedef int v4a __attribute__((ext_vector_type(4), aligned(4)));
    __shared__ __attribute__((aligned(16))) unsigned s_word[kChunk];
    __shared__ __attribute__((aligned(16))) float s_bias[kChunk];
    __shared__ int s_tok[GDN_MAX_NODES], s_again;
    __shared__ unsigned s_anc[GDN_MAX_NODES];
    __shared__ float s_max[GDN_MAX_NODES], s_inv[GDN_MAX_NODES];
    __shared__ int s_best[GDN_MAX_NODES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = blockIdx.y, x0 = blockIdx.x * kChunk;
    const int i0 = blockIdx.z * a.rows;

    // ---- the lane's checks; every wave of every workgroup comes to the same verdict
    const int slot = a.slot_ids[c], nodes = a.lane_nodes ? a.lane_nodes[c] : a.N;
    if (slot == -1) return;
    int bits = 0;
    if (nodes < 0 || nodes > a.N) bits |= GDN_STATUS_NODES;
    float rep = 1.f, pres = 0.f, freq = 0.f, temp = 1.f;
    int held = 0, prompt = 0;
    if (slot < -1 || slot >= a.P) {
        bits |= GDN_STATUS_SLOT_RANGE;
    } else {
        if (a.r.repetition) rep = a.r.repetition[slot];
        if (a.r.presence) pres = a.r.presence[slot];
        if (a.r.frequency) freq = a.r.frequency[slot];
        if (a.r.temperature) temp = a.r.temperature[slot];
        if (a.r.history) held = a.r.history_len[slot];
        if (a.r.history && a.r.prompt_len) prompt = a.r.prompt_len[slot];
        if (!(rep > 0.f) || !__builtin_isfinite(rep) || !__builtin_isfinite(pres) || !__builtin_isfinite(freq) || !(temp >= 0.f) ||
            !__builtin_isfinite(temp))
            bits |= GDN_STATUS_RULE;
        if (held < 0 || held > a.H || prompt < 0 || prompt > held) bits |= GDN_STATUS_LENGTH;
    }
    int tok = -1;
    unsigned anc = 0;
    if (!(bits & GDN_STATUS_NODES)) {
        const bool has = lane < nodes;  // (at most 32)
        anc = has ? (2u << lane) - 1u : 0u;
        bool bad = false;
        if (a.parents) anc = tree_ancestors(a.parents + (int64_t)c * a.N, nodes, bad);
        if (bad) bits |= GDN_STATUS_PARENT;
        if (a.tokens && has) tok = a.tokens[(int64_t)c * a.N + lane];
        if (__builtin_amdgcn_ballot_w64(a.tokens && has && (unsigned)tok >= (unsigned)a.V)) bits |= GDN_STATUS_TOKEN;
    }
    if (bits) {
        if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0 && a.status && MODE != kProbabilities) atomicOr(a.status, bits);
        return;
    }
    const int i1 = min(i0 + a.rows, nodes);
    if (i0 >= i1) return;

    // ---- the stretch's words
#pragma unroll
    for (int k = 0; k < W / 4; ++k) reinterpret_cast<v4i *>(s_word)[k * kThreads + tid] = v4i{0, 0, 0, 0};
    const bool biased = a.r.bias_tokens && a.B > 0;
    if (biased)
#pragma unroll
        for (int k = 0; k < W / 4; ++k) reinterpret_cast<v4f *>(s_bias)[k * kThreads + tid] = v4f{0.f, 0.f, 0.f, 0.f};
    if (tid < GDN_MAX_NODES) {
        s_tok[tid] = tok;
        s_anc[tid] = anc;
    }
    if (tid == 0) s_again = 0;
    if constexpr (MODE == kProbabilities) {  // the rows' maxima and sums, a row a wave
        const int parts = gridDim.x * kWaves;
        const float k2 = per_temperature(temp);
        for (int i = i0 + wave; i < i1; i += kWaves) {
            const v4f *st = reinterpret_cast<const v4f *>(a.stats) + ((size_t)c * a.N + i) * parts;
            Best b{kNegInf, 0x7fffffff};
            for (int k = lane; k < parts; k += 64) b = better(b, Best{st[k][0], __float_as_int(st[k][2])});
            b = wave_best(b);
            float sum = 0.f;
            for (int k = lane; k < parts; k += 64) {
                const float m = st[k][0], s = st[k][1];
                if (s != 0.f) sum += s * weight(m, b.v, k2);
            }
            sum = wave_sum(sum);
            if (lane == 0) {
                s_max[i - i0] = b.v;
                s_inv[i - i0] = sum == 0.f ? 0.f : 1.f / sum;
                s_best[i - i0] = b.v == kNegInf ? -1 : b.x;
            }
        }
    }
    lds_barrier();
    if (held > 0) {
        const int32_t *past = a.r.history + (int64_t)slot * a.H;
        auto count = [&](int at, int t) {
            const int x = t - x0;
            if ((unsigned)x < (unsigned)kChunk && t < a.V) {
                if (at >= prompt)
                    atomicAdd(&s_word[x], 1u);
                else
                    atomicOr(&s_word[x], kPrompt);
            }
        };
        const int whole = held / 4;
        for (int k = tid; k < whole; k += kThreads) {
            const v4a t = *reinterpret_cast<const v4a *>(past + 4 * k);
#pragma unroll
            for (int e = 0; e < 4; ++e) count(4 * k + e, t[e]);
        }
        if (4 * whole + tid < held && tid < 4) count(4 * whole + tid, past[4 * whole + tid]);
    }
    if (tok >= x0 && tok < x0 + kChunk && tid < GDN_MAX_NODES) atomicOr(&s_word[tok - x0], kDraft);
    if (biased) {
        const int32_t *toks = a.r.bias_tokens + (int64_t)slot * a.B;
        const float *vals = a.r.bias + (int64_t)slot * a.B;
        for (int j = tid; j < a.B; j += kThreads) {
            const int t = toks[j], x = t - x0;
            if ((unsigned)x < (unsigned)kChunk && t < a.V) {
                if (atomicOr(&s_word[x], kBias) & kBias) s_again = 1;
                s_bias[x] = vals[j];
            }
        }
        lds_barrier();
        if (s_again)  // a token twice: its first entry's thread adds them up in the list's order
            for (int j = tid; j < a.B; j += kThreads) {
                const int t = toks[j], x = t - x0;
                if ((unsigned)x >= (unsigned)kChunk || t >= a.V) continue;
                bool first = true;
                for (int k = 0; k < j; ++k) first &= toks[k] != t;
                if (!first) continue;
                float sum = vals[j];
                for (int k = j + 1; k < a.B; ++k)
                    if (toks[k] == t) sum += vals[k];
                s_bias[x] = sum;
            }
    }
    lds_barrier();
    // ---- this thread's tokens: group g from x0 + (g kThreads + tid) VEC on
    unsigned w[W];
    float b[W];
#pragma unroll
    for (int g = 0; g < GR; ++g)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[g * VEC + e] = s_word[(g * kThreads + tid) * VEC + e];
            b[g * VEC + e] = biased ? s_bias[(g * kThreads + tid) * VEC + e] : 0.f;
        }
    const float inv = 1.f / rep;
    const float k2 = per_temperature(temp);
    const int mask_words = (a.V + 31) / 32;

    tv raw[GR];
    unsigned allow[GR];
    auto load = [&](int i) {
        const int64_t row = (int64_t)c * a.N + i;
        const T *p = static_cast<const T *>(a.logits) + row * a.stride;
#pragma unroll
        for (int g = 0; g < GR; ++g) {
            const int x = x0 + (g * kThreads + tid) * VEC;
            if (x + VEC <= a.V) {
                raw[g] = *reinterpret_cast<const tv *>(p + x);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) raw[g][e] = x + e < a.V ? p[x + e] : (T)0.f;
            }
            allow[g] = 0xffffffffu;
            if (a.mask && x < a.V) allow[g] = (unsigned)a.mask[row * mask_words + x / 32] >> (x & 31);
        }
    };
    load(i0);
    for (int i = i0; i < i1; ++i) {
        float z[W];
        const unsigned path = s_anc[i];
#pragma unroll
        for (int g = 0; g < GR; ++g)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int q = g * VEC + e, x = x0 + (g * kThreads + tid) * VEC + e;
                unsigned n = w[q] & kCount;
                bool seen = (w[q] & (kCount | kPrompt)) != 0;
                if (w[q] & kDraft)
                    for (unsigned p = path; p; p &= p - 1u)
                        if (s_tok[__builtin_ctz(p)] == x) ++n, seen = true;
                float v = (float)raw[g][e] + b[q];
                const float scaled = v * (v > 0.f ? inv : rep);
                v = seen ? scaled : v;
                const float less = fmaf(-freq, (float)n, v) - pres;
                v = n ? less : v;
                z[q] = (allow[g] >> e) & 1 && x < a.V ? v : kNegInf;
            }
        if (i + 1 < i1) load(i + 1);
        if constexpr (MODE == kStats) {
            Best top{kNegInf, 0x7fffffff};
#pragma unroll
            for (int g = 0; g < GR; ++g)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (z[g * VEC + e] > top.v) top = Best{z[g * VEC + e], x0 + (g * kThreads + tid) * VEC + e};
            top = wave_best(top);
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < W; ++q) sum += weight(z[q], top.v, k2);
            sum = wave_sum(sum);
            if (lane == 0)
                reinterpret_cast<v4f *>(a.stats)[((size_t)c * a.N + i) * gridDim.x * kWaves + blockIdx.x * kWaves + wave] =
                    v4f{top.v, sum, __int_as_float(top.x), 0.f};
            continue;
        }
        if constexpr (MODE == kProbabilities) {
            const float m = s_max[i - i0], scale = s_inv[i - i0];
            const int best = s_best[i - i0];
#pragma unroll
            for (int g = 0; g < GR; ++g)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int q = g * VEC + e, x = x0 + (g * kThreads + tid) * VEC + e;
                    z[q] = temp > 0.f ? weight(z[q], m, k2) * scale : x == best ? 1.f : 0.f;
                }
        }
        O *out = static_cast<O *>(a.out) + ((int64_t)c * a.N + i) * a.V;
#pragma unroll
        for (int g = 0; g < GR; ++g) {
            const int x = x0 + (g * kThreads + tid) * VEC;
            if (x + VEC <= a.V) {
                ov o;
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = (O)z[g * VEC + e];
                *reinterpret_cast<ov *>(out + x) = o;
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (x + e < a.V) out[x + e] = (O)z[g * VEC + e];
            }
        }
    }
}

template <typename T, typename O, int W>
hipError_t launch_w(const LogitArgs &a, dim3 grid, hipStream_t stream) {
    if (!a.r.temperature) {
        hipLaunchKernelGGL((adjust_logits_kernel<T, O, W, kLogits>), grid, dim3(kThreads), 0, stream, a);
    } else {
        hipLaunchKernelGGL((adjust_logits_kernel<T, O, W, kStats>), grid, dim3(kThreads), 0, stream, a);
        hipLaunchKernelGGL((adjust_logits_kernel<T, O, W, kProbabilities>), grid, dim3(kThreads), 0, stream, a);
    }
    return hipGetLastError();
}

template <typename T, typename O>
hipError_t launch(LogitArgs a, hipStream_t stream) {
    const LogitPlan p = logit_plan(a.C, a.N, a.V);
    a.rows = p.rows;
    const dim3 grid(p.chunks(a.V), a.C, (a.N + p.rows - 1) / p.rows);
    return p.per == 16 ? launch_w<T, O, 16>(a, grid, stream) : launch_w<T, O, 8>(a, grid, stream);
}

}  // namespace

hipError_t launch_adjust_logits(const LogitArgs &a, hipStream_t stream) {
    const bool wide = a.out_dtype == GDN_DTYPE_F32;
    if (a.dtype == GDN_DTYPE_BF16) return wide ? launch<__bf16, float>(a, stream) : launch<__bf16, __bf16>(a, stream);
    if (a.dtype == GDN_DTYPE_F16) return wide ? launch<_Float16, float>(a, stream) : launch<_Float16, _Float16>(a, stream);
    return launch<float, float>(a, stream);
}

}  // namespace gdn

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
//
// 4 lanes of 16 nodes, 130001 tokens, every rule, bfloat16 to float32 probabilities: 15.5 + 16.3 us for 17 and 17 + 33 MB (some
// 5 us of each until the first row is worked on, then about 15 operations and an exponential a value); 32 lanes of 32:
// 348 us, 3.2 TB/s over both launches, and without a temperature, to bfloat16, 140 us, 3.9 TB/s; one node of 4 lanes, 32768
// tokens, bfloat16 logits: 5.2 us.  Eight tokens a thread and
// 512 threads: with 16 and 256 the constants of a thread's tokens went through memory (54.6 us and 44).  Two rows in flight
// instead of one: 30.7 us and 30.3, 32 lanes of 32 369 and 352 (as this was chosen).
#include "logits_internal.h"
#include "round_device.h"

namespace gdn {
namespace {

constexpr int kThreads = kLogitThreads, kWaves = kThreads / 64;
constexpr float kNegInf = -__builtin_inff();

// Flags of a token's word above its count (at most 2^20 entries of history)
constexpr unsigned kCount = (1u << 24) - 1u, kPrompt = 1u << 24, kBias = 1u << 25, kDraft = 1u << 26, kTwice = 1u << 27;

constexpr int kMostBiases = 1024;  // the longest list
static_assert(kMostBiases % kThreads == 0, "");

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
// Largest and sum over a wave, the same in every lane: rotations within the rows of 16 lanes (no LDS), then the four rows
template <int N>
__device__ inline float row_rotated(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + N, 0xF, 0xF, false));
}
__device__ inline float lane_of(float x, int j) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), j)); }
// (as integers of the same order, whose maximum takes no quieting of NaN; a NaN is above infinity there)
__device__ inline int ordered(float x) { return __float_as_int(x) ^ ((__float_as_int(x) >> 31) & 0x7fffffff); }
template <int N>
__device__ inline int row_rotated(int x) { return __builtin_amdgcn_update_dpp(x, x, 0x120 + N, 0xF, 0xF, false); }
__device__ inline float wave_max(float v) {
    int x = ordered(v);
    x = max(x, row_rotated<8>(x));
    x = max(x, row_rotated<4>(x));
    x = max(x, row_rotated<2>(x));
    x = max(x, row_rotated<1>(x));
    const int a = max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16));
    const int b = max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48));
    const int top = max(a, b);
    return __int_as_float(top ^ ((top >> 31) & 0x7fffffff));
}
__device__ inline float wave_sum(float x) {
    x += row_rotated<8>(x);
    x += row_rotated<4>(x);
    x += row_rotated<2>(x);
    x += row_rotated<1>(x);
    return (lane_of(x, 0) + lane_of(x, 16)) + (lane_of(x, 32) + lane_of(x, 48));
}
constexpr int kAhead = 4;  // loads of a thread that are requested together
// A temperature that is no normal number: its factor would pass the largest number, and halves of differences of its size lose
// their last bit.
__device__ inline bool steep(float temp) { return temp > 0.f && temp < 0x1p-126f; }
// 2 log2(e) / T, finite for T = 0; never 0 (2^-127 for the largest T: not a normal number, but exact to 2^-22), so that
// -infinity times it is -infinity.  It multiplies half of z - m, which no two finite numbers carry out of range; for a steep
// T, log2(e) / (2^64 T), of 2^64 (z - m): out of range only where the weight is 0.
__device__ inline float per_temperature(float temp) {
    return steep(temp) ? 1.4426950408889634f / (temp * 0x1p64f) : fminf(2.8853900817779268f / temp, 3.4e38f);
}
__device__ inline float half_below(float z, float half_m) { return fmaf(z, 0.5f, -half_m); }
// e^{(z - m) / T}; 1 at the maximum even where that is infinite, 0 for -infinity
struct Weight {
    float k;  // per_temperature(temp)
    bool is_steep;
    __device__ float operator()(float z, float m) const {
        const float top = m == kNegInf ? 0.f : m;
        return __builtin_amdgcn_exp2f(z == top ? 0.f : (is_steep ? (z - top) * 0x1p64f : half_below(z, 0.5f * top)) * k);
    }
};

// Entries of a slot's history from k0 on, four at a time: entry 4 (j kThreads + tid) + k0 and the next three, or, where
// these would pass the end, the last four (of which `from` leaves out what another thread has; fewer than four in all:
// one at a time).
struct Past {
    typedef int v4a __attribute__((ext_vector_type(4), aligned(4)));
    v4a t[kAhead];
    __device__ static int from(int k0, int j) { return k0 + 4 * (j * kThreads + (int)threadIdx.x); }
    __device__ static int at(const LogitArgs &a, int k0, int j) { return max(min(from(k0, j), a.H - 4), 0); }
    __device__ void load(const LogitArgs &a, int slot, int k0) {
        const int32_t *p = a.r.history + (int64_t)slot * a.H;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            t[j] = v4a{-1, -1, -1, -1};
            if (k0 + 4 * j * kThreads >= a.H) continue;  // (the same for every thread)
            if (a.H >= 4) {
                t[j] = *reinterpret_cast<const v4a *>(p + at(a, k0, j));
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (e < a.H) t[j][e] = p[e];
            }
        }
    }
};

// A row's maximum, sum of exponentials below it and place of the maximum.  Every wave that has a piece of the row leaves
// its own; by a wave, the whole from these: a lane takes every 64th, in order, the lanes are joined in a fixed tree.
struct Total {
    float top, sum;
    int at;
};
constexpr int kParts = 4;  // a lane's parts that are requested together
struct Parts {
    v4f v[kParts];
    __device__ static const v4f *of(const LogitArgs &a, int c, int i) {
        return reinterpret_cast<const v4f *>(a.stats) + ((size_t)c * a.N + i) * gridDim.x * kWaves;
    }
    __device__ void load(const v4f *row, int k0) {
        const int parts = gridDim.x * kWaves;
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
            const int k = k0 + 64 * j + (int)(threadIdx.x & 63);
            v[j] = row[min(k, parts - 1)];
            if (k >= parts) v[j] = v4f{kNegInf, 0.f, __int_as_float(0x7fffffff), 0.f};
        }
    }
};
__device__ inline Total row_total(const LogitArgs &a, int c, int i, float temp, Parts &p) {  // p: the first ones, loaded
    const int parts = gridDim.x * kWaves;
    const Weight weight{per_temperature(temp), steep(temp)};
    const v4f *row = Parts::of(a, c, i);
    Best b{kNegInf, 0x7fffffff};
    float sum = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < parts; k0 += 64 * kParts) {
        if (k0) p.load(row, k0);
        Best to = b;
#pragma unroll
        for (int j = 0; j < kParts; ++j) to = better(to, Best{p.v[j][0], __float_as_int(p.v[j][2])});
        if (k0) sum = sum == 0.f ? 0.f : sum * weight(b.v, to.v);  // (a part of nothing has sum 0; NaN sums stay NaN)
#pragma unroll
        for (int j = 0; j < kParts; ++j) sum += p.v[j][1] == 0.f ? 0.f : p.v[j][1] * weight(p.v[j][0], to.v);
        b = to;
    }
    Best all{wave_max(b.v), 0x7fffffff};
    if (temp == 0.f) all = wave_best(b);
    return Total{all.v, wave_sum(sum == 0.f ? 0.f : sum * weight(b.v, all.v)), all.x};
}

template <typename T, typename O, int MODE>
__global__ __launch_bounds__(kThreads, 4) void adjust_logits_kernel(LogitArgs a) {
    constexpr int W = kLogitTokens, VEC = 16 / sizeof(T), GR = W / VEC, kChunk = kLogitChunk;
    typedef T tv __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
    typedef O ov __attribute__((ext_vector_type(VEC), aligned(sizeof(O))));
    __shared__ __attribute__((aligned(16))) unsigned s_word[kChunk];
    __shared__ __attribute__((aligned(16))) float s_bias[kChunk];
    __shared__ int s_again;
    __shared__ unsigned s_anc[GDN_MAX_NODES];
    __shared__ Total s_total[GDN_MAX_NODES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = blockIdx.y, x0 = blockIdx.x * kChunk;
    const int i0 = blockIdx.z * a.rows;

    const int slot = a.slot_ids[c], nodes = a.lane_nodes ? a.lane_nodes[c] : a.N;
    if (slot == -1) return;
    // ---- requested ahead of the checks: the tree, a row's parts, the first row (every node has one, present or not), the first of the history
    // (its length not known yet: what lies behind it is not counted) and the biases of the slot
    const bool in_lane = lane < a.N;  // (at most 32)
    const int64_t node = (int64_t)c * a.N + min(lane, a.N - 1);
    int parent = lane - 1, tok = -1;
    if (a.parents) parent = a.parents[node];
    if (a.tokens) tok = a.tokens[node];
    Parts parts;
    if constexpr (MODE == kProbabilities) parts.load(Parts::of(a, c, min(i0 + wave, a.N - 1)), 0);
    // (a row's words of the mask stay as they are until the row's turn: to take a bit out of one is to wait for every load)
    const int mask_words = (a.V + 31) / 32;
    tv raw[GR];
    unsigned allow[GR];
#pragma unroll
    for (int g = 0; g < GR; ++g) allow[g] = ~0u;
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
            if (a.mask) allow[g] = (unsigned)a.mask[row * mask_words + min(x, a.V - 1) / 32];
        }
    };
    load(i0);
    const int known = slot < -1 || slot >= a.P ? 0 : slot;
    Past past;
    if (a.r.history) past.load(a, known, 0);
    constexpr int kBiases = kMostBiases / kThreads;
    int bias_tok[kBiases];
    float bias_val[kBiases];
    if (a.r.bias_tokens)
#pragma unroll
        for (int j = 0; j < kBiases; ++j) {
            bias_tok[j] = -1;
            if (j * kThreads < a.B) {  // (the same for every thread)
                const int64_t at = (int64_t)known * a.B + min(j * kThreads + tid, a.B - 1);
                bias_tok[j] = a.r.bias_tokens[at];
                bias_val[j] = a.r.bias[at];
            }
        }

    // ---- the lane's checks; every wave of every workgroup comes to the same verdict
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
        if (!(rep >= 0x1p-126f && rep <= 0x1p126f) || !__builtin_isfinite(pres) || !__builtin_isfinite(freq) || !(temp >= 0.f) ||
            !__builtin_isfinite(temp))
            bits |= GDN_STATUS_RULE;
        if (held < 0 || held > a.H || prompt < 0 || prompt > held) bits |= GDN_STATUS_LENGTH;
    }
    const bool has = in_lane && lane < nodes;
    if (!has) tok = -1;
    if (!(bits & GDN_STATUS_NODES)) {
        if (__builtin_amdgcn_ballot_w64(has && (parent < -1 || parent >= lane))) bits |= GDN_STATUS_PARENT;
        if (__builtin_amdgcn_ballot_w64(a.tokens && has && (unsigned)tok >= (unsigned)a.V)) bits |= GDN_STATUS_TOKEN;
    }
    if (bits) {
        if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0 && a.status && MODE != kProbabilities) atomicOr(a.status, bits);
        return;
    }
    const int i1 = min(i0 + a.rows, nodes);
    if (i0 >= i1) return;
    const unsigned inside = min(kChunk, a.V - x0);  // (an id outside the stretch, or the vocabulary, is not below it from x0 on)

    // ---- the stretch's words
    const bool biased = a.r.bias_tokens && a.B > 0;
#pragma unroll
    for (int k = 0; k < W / 4; ++k) {
        reinterpret_cast<v4i *>(s_word)[k * kThreads + tid] = v4i{0, 0, 0, 0};
        if (biased) reinterpret_cast<v4f *>(s_bias)[k * kThreads + tid] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    if (tid == 0) s_again = 0;
    if (a.tokens && wave == kWaves - 1) {  // (while the history is on its way)
        bool bad;
        const unsigned anc = a.parents ? tree_sets(parent, has, bad) : has ? (2u << lane) - 1u : 0u;
        if (lane < GDN_MAX_NODES) s_anc[lane] = anc;
    }
    if constexpr (MODE == kProbabilities)
        for (int i = i0 + wave; i < i1; i += kWaves) {  // a row a wave
            if (i != i0 + wave) parts.load(Parts::of(a, c, i), 0);
            const Total t = row_total(a, c, i, temp, parts);
            if (lane == 0) s_total[i - i0] = t;
        }
    lds_barrier();
    if (a.r.history) {
#pragma unroll 1
        for (int k0 = 0; k0 == 0 || k0 < held; k0 += 4 * kThreads * kAhead) {
            if (k0) past.load(a, slot, k0);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (k0 + 4 * j * kThreads >= held) continue;  // (the same for every thread)
                const int at = past.at(a, k0, j), low = past.from(k0, j) - at, high = held - at;
                if (__builtin_amdgcn_ballot_w64(low > 0 || high < 4))
#pragma unroll
                    for (int e = 0; e < 4; ++e) past.t[j][e] = e >= low && e < high ? past.t[j][e] : -1;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const unsigned x = (unsigned)(past.t[j][e] - x0);
                    if (x < inside) {
                        if (at + e >= prompt)
                            atomicAdd(&s_word[x], 1u);
                        else
                            atomicOr(&s_word[x], kPrompt);
                    }
                }
            }
        }
    }
    if ((unsigned)(tok - x0) < inside && tid < GDN_MAX_NODES) atomicOr(&s_word[tok - x0], kDraft);
    bool first[kBiases] = {};  // of a token's entries, to come here
    if (biased) {
#pragma unroll
        for (int j = 0; j < kBiases; ++j) {
            const unsigned x = (unsigned)(bias_tok[j] - x0);
            if (x < inside && j * kThreads + tid < a.B) {
                first[j] = !(atomicOr(&s_word[x], kBias) & kBias);
                if (!first[j]) {
                    atomicOr(&s_word[x], kTwice);
                    s_again = 1;
                }
                s_bias[x] = bias_val[j];
            }
        }
    }
    lds_barrier();
    // Tokens with several biases: the wave that was first at one finds its entries and adds them, in the list's order (1024 biases, 4
    // rows of 32768: one token twice 5.4 us and 4.4 without, all of one token 37; each entry's thread going through the list
    // 207 and 202).  The list comes from memory again: with a copy in LDS, 8 KiB, a workgroup fewer fits a CU (32 x 32 rows of 130001
    // without a temperature 151 us and 140).
    if (biased && s_again) {
        int t[kMostBiases / 64];  // entries 64 i + lane
        float v[kMostBiases / 64];
#pragma unroll
        for (int i = 0; i < kMostBiases / 64; ++i) {
            const int64_t at = (int64_t)slot * a.B + min(64 * i + lane, a.B - 1);
            t[i] = a.r.bias_tokens[at];
            v[i] = a.r.bias[at];
            if (64 * i + lane >= a.B) t[i] = -1;
        }
#pragma unroll
        for (int j = 0; j < kBiases; ++j) {
            unsigned long long todo = __builtin_amdgcn_ballot_w64(first[j] && (s_word[bias_tok[j] - x0] & kTwice));
            for (; todo; todo &= todo - 1) {
                const int u = __builtin_amdgcn_readlane(bias_tok[j], __builtin_ctzll(todo));
                float sum = -0.f;
#pragma unroll
                for (int i = 0; i < kMostBiases / 64; ++i)
                    for (unsigned long long same = __builtin_amdgcn_ballot_w64(t[i] == u); same; same &= same - 1)
                        sum += lane_of(v[i], __builtin_ctzll(same));
                if (lane == 0) s_bias[u - x0] = sum;
            }
        }
        lds_barrier();
    }
    // ---- this thread's tokens: group g from x0 + (g kThreads + tid) VEC on.  A logit l becomes (l + b) up - less above zero and
    // (l + b) down - less elsewhere.  `on`: the nodes with this token.
    auto token_of = [&](int q) { return (q / VEC * kThreads + tid) * VEC + q % VEC; };
    float b[W], up[W], down[W], less[W];
    unsigned w[W], on[W], drafts = 0;
    // (a repetition is a product with the rounded reciprocal, at most one step beside the quotient: 4 x 16 rows of 130001 29.7 us, with
    // the product corrected to the rounded quotient 31.3, with divisions 34.0)
    const float inv = 1.f / rep, k2 = per_temperature(temp);
    const Weight weight{k2, steep(temp)};
#pragma unroll
    for (int q = 0; q < W; ++q) {
        w[q] = s_word[token_of(q)];
        b[q] = biased ? s_bias[token_of(q)] : 0.f;
        const bool seen = (w[q] & (kCount | kPrompt)) != 0;
        up[q] = seen ? inv : 1.f;
        down[q] = seen ? rep : 1.f;
        less[q] = w[q] & kCount ? fmaf(freq, (float)(w[q] & kCount), pres) : 0.f;
        on[q] = 0;
        drafts |= w[q];
    }
    const bool drafted = __builtin_amdgcn_ballot_w64((drafts & kDraft) != 0) != 0;  // (of this wave)
    if (drafted) {
        const int base = x0 + __builtin_amdgcn_readfirstlane(tid & ~63) * VEC;  // of the wave's first group
#pragma unroll 1
        for (int j = 0; j < nodes; ++j) {
            const int t = __builtin_amdgcn_readlane(tok, j) - base;
            if (GR == 1 && (unsigned)t >= 64u * VEC) continue;  // (the same for the wave)
#pragma unroll
            for (int q = 0; q < W; ++q) on[q] |= t == q / VEC * kThreads * VEC + lane * VEC + q % VEC ? 1u << j : 0u;
        }
    }
    unsigned edge[GR];  // the group's tokens inside the vocabulary
#pragma unroll
    for (int g = 0; g < GR; ++g) {
        const int held_back = min(max(x0 + (g * kThreads + tid + 1) * VEC - a.V, 0), VEC);
        edge[g] = ((1u << VEC) - 1u) >> held_back;
    }
    const bool cut = a.mask || x0 + kChunk > a.V;  // some token of the stretch may not be allowed
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        float z[W];
#pragma unroll
        for (int q = 0; q < W; ++q) {
            const float v = (float)raw[q / VEC][q % VEC] + b[q];
            z[q] = fmaf(v, v > 0.f ? up[q] : down[q], -less[q]);
        }
        if (drafted) {
            const unsigned path = s_anc[i];
#pragma unroll
            for (int q = 0; q < W; ++q) {
                const unsigned here = on[q] & path, n = (w[q] & kCount) + __popc(here);
                const float v = (float)raw[q / VEC][q % VEC] + b[q];
                z[q] = here ? v * (v > 0.f ? inv : rep) - fmaf(freq, (float)n, pres) : z[q];
            }
        }
        if (cut)
#pragma unroll
            for (int g = 0; g < GR; ++g) {  // (bit by bit: all ones where the token is allowed; opaque, or it becomes compares and selects)
                const int x = x0 + (g * kThreads + tid) * VEC;
                const unsigned bits = (allow[g] >> (x & 31)) & edge[g];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    int keep = (int)(bits << (31 - e)) >> 31;
                    asm("" : "+v"(keep));
                    float &zz = z[g * VEC + e];
                    zz = __int_as_float((keep & __float_as_int(zz)) | (~keep & __float_as_int(kNegInf)));
                }
            }
        if (i + 1 < i1) load(i + 1);
        if constexpr (MODE == kStats) {
            Best top{kNegInf, 0x7fffffff};
            if (temp > 0.f) {  // (the place of the maximum is for T = 0 only)
#pragma unroll
                for (int q = 0; q < W; ++q) top.v = fmaxf(top.v, z[q]);
                top.v = wave_max(top.v);
            } else {
#pragma unroll
                for (int q = 0; q < W; ++q)
                    if (z[q] > top.v) top = Best{z[q], x0 + token_of(q)};
                top = wave_best(top);
            }
            float sum = 0.f;
            if (fabsf(top.v) < __builtin_inff() && !steep(temp)) {
#pragma unroll
                for (int q = 0; q < W; ++q) sum += __builtin_amdgcn_exp2f(half_below(z[q], 0.5f * top.v) * k2);
            } else {
#pragma unroll
                for (int q = 0; q < W; ++q) sum += weight(z[q], top.v);
            }
            sum = wave_sum(sum);
            if (lane == 0)
                reinterpret_cast<v4f *>(a.stats)[(((size_t)c * a.N + i) * gridDim.x + blockIdx.x) * kWaves + wave] =
                    v4f{top.v, sum, __int_as_float(top.x), 0.f};
        } else {
            if constexpr (MODE == kProbabilities) {
                const Total t = s_total[i - i0];
                const float scale = t.sum == 0.f ? 0.f : 1.f / t.sum;
                if (temp >= 0x1p-126f && fabsf(t.top) < __builtin_inff()) {
#pragma unroll
                    for (int q = 0; q < W; ++q) z[q] = __builtin_amdgcn_exp2f(half_below(z[q], 0.5f * t.top) * k2) * scale;
                } else {
                    const int best = t.top == kNegInf ? -1 : t.at;
#pragma unroll
                    for (int q = 0; q < W; ++q)
                        z[q] = temp > 0.f ? weight(z[q], t.top) * scale : x0 + token_of(q) == best ? 1.f : 0.f;
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
}

template <typename T, typename O>
hipError_t launch(LogitArgs a, hipStream_t stream) {
    a.rows = logit_rows(a.C, a.N, a.V);
    const dim3 grid(logit_chunks(a.V), a.C, (a.N + a.rows - 1) / a.rows);
    if (!a.r.temperature) {
        hipLaunchKernelGGL((adjust_logits_kernel<T, O, kLogits>), grid, dim3(kThreads), 0, stream, a);
    } else {
        hipLaunchKernelGGL((adjust_logits_kernel<T, O, kStats>), grid, dim3(kThreads), 0, stream, a);
        hipLaunchKernelGGL((adjust_logits_kernel<T, O, kProbabilities>), grid, dim3(kThreads), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adjust_logits(const LogitArgs &a, hipStream_t stream) {
    const bool wide = a.out_dtype == GDN_DTYPE_F32;
    if (a.dtype == GDN_DTYPE_BF16) return wide ? launch<__bf16, float>(a, stream) : launch<__bf16, __bf16>(a, stream);
    if (a.dtype == GDN_DTYPE_F16) return wide ? launch<_Float16, float>(a, stream) : launch<_Float16, _Float16>(a, stream);
    return launch<float, float>(a, stream);
}

}  // namespace gdn

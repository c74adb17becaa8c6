// Attention of a round's new tokens over a slot's paged key/value cache, for gfx950.
//
// Mathematics.  For node i of a lane and query head h (kv head h / G) with the rows t that i
// attends to:  x_t = scale q.K[t],  out = sum_t e^{x_t} V[t] / sum_t e^{x_t}.  One pass over the
// cache keeps, per query row, the running maximum m, the sum l of e^{x - m} and the unnormalised
// output o; a new block of rows rescales l and o by e^{m_old - m_new} (all in 32 bits).
//
// Layout of a workgroup's work.  The query rows of one (lane, kv head) are its N*G pairs
// (token, head of the group), in that order: they share every K and V row.  A wave owns RT tiles
// of 16 query rows and computes S^T = K Q^T with 16x16 matrix instructions: the accumulator of
// a tile holds, in lane l, the scores of query row l % 16 against cache rows 4 (l / 16) + 0..3.  So
// the softmax statistics of a query row are scalars of its lanes, and the weights are, as they
// stand, the right operand of O^T = V^T P^T (the contraction runs over cache rows in the order
// the accumulators hold them, which the left operand follows); no score goes through memory.
// The left operand V^T takes four cache rows of one column per lane: the 16-bit path reads it
// with the transposing LDS load, the 32-bit path with plain loads of one value.
//
// The cache holds values of the queries' type, or (kFour) 4-bit numbers with a power of two for every 32 values of a
// row: those become values of the queries' type, exactly but for float16's range, on their way into LDS or into an
// operand, and everything behind that is the same.  Internal linkage: paged_attention.hip has the kernels of the
// first and the join, paged_attention_kv4.hip those of the second.
#pragma once

#include <algorithm>
#include <type_traits>

#include "round_device.h"

namespace gdn {
namespace {

constexpr float kNegInf = -__builtin_inff();
// What may be scheduled across a step of the products: vector, scalar and transcendental arithmetic and global
// memory, not the LDS reads and products themselves, whose order is the reading ahead.
constexpr int kArithmetic = 0x2 | 0x4 | 0x10 | 0x400;
constexpr float kSlack = 6.f;  // how far, in powers of two, a running maximum may lead its base
constexpr float kFar = 1048576.f;  // bases beyond this: scores as differences first (from_maximum)
typedef short s4 __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));

// ---- the value types: 16-byte operand fragments and the matrix instructions on them.
// A fragment holds 64 bytes' worth of one row over the four lane groups: 32 16-bit or 16 32-bit
// contraction indices per step.
// 16-bit weights are rounded to their type for the second product (the 16-bit matrix instructions take no others,
// and two of them, for a weight in two parts, would double that product); the sum keeps them in 32 bits.  kLift: how
// many powers of two the exponentials' base lies below the running maximum.  float16 holds numbers below 2^-14 with
// a fixed error of 2^-25: with a base at the maximum, weights 15 powers of two and more below it would lose their
// last bits and those 25 below it vanish, while the sum counts them (one row 16 nats above 262144 equal ones: the output is
// 6% off).  Nine powers lower the largest weight is 2^(9 + kSlack) = 2^15, inside the type's range, and a row's
// weight is off by half a step or by 2^-34 of the largest one.  Costs nothing: the base is one number a row.
template <typename T>
struct Type;
template <>
struct Type<__bf16> {
    static constexpr unsigned kExp = 0x7f80u, kOne = 0x3f80u;
    static constexpr float kLift = 0.f;
    static __device__ v4f mma(v4i a, v4i b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
    }
    // sixteen contraction indices, four a lane
    static __device__ v4f mma16(v2i a, v2i b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s4, a), __builtin_bit_cast(s4, b), c, 0, 0, 0);
    }
    static __device__ v4i pack(v4f a, v4f b) {
        return __builtin_bit_cast(v4i, bf8{(__bf16)a[0], (__bf16)a[1], (__bf16)a[2], (__bf16)a[3], (__bf16)b[0],
                                           (__bf16)b[1], (__bf16)b[2], (__bf16)b[3]});
    }
};
template <>
struct Type<_Float16> {
    static constexpr unsigned kExp = 0x7c00u, kOne = 0x3c00u;
    static constexpr float kLift = 9.f;
    static __device__ v4f mma(v4i a, v4i b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
    }
    static __device__ v4f mma16(v2i a, v2i b, v4f c) {
        typedef _Float16 h4 __attribute__((ext_vector_type(4)));
        return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(h4, a), __builtin_bit_cast(h4, b), c, 0, 0, 0);
    }
    static __device__ v4i pack(v4f a, v4f b) {
        return __builtin_bit_cast(v4i, h8{(_Float16)a[0], (_Float16)a[1], (_Float16)a[2], (_Float16)a[3],
                                          (_Float16)b[0], (_Float16)b[1], (_Float16)b[2], (_Float16)b[3]});
    }
};
template <>
struct Type<float> {
    static constexpr unsigned kExp = 0x7f800000u, kOne = 0x3f800000u;
    static constexpr float kLift = 0.f;
    static __device__ v4f mma(v4i a, v4i b, v4f c) { return mfma4(__builtin_bit_cast(v4f, a), __builtin_bit_cast(v4f, b), c); }
};

// Base of the exponentials for a running maximum (nothing attended yet: any, every weight is 2^-inf)
template <typename T>
__device__ inline float weight_base(float m) { return (m == kNegInf ? 0.f : m) - Type<T>::kLift; }

// The exponent of a weight is scale * score - base in one operation, exact but for one rounding, while base is a product
// that has been rounded: the remainder of the largest score is up to 2^-25 of the base.  Beyond a base of 2^32 that
// is a weight of 2^128 or of 0.  So far out the product is rounded as the maximum's was (never fused: the largest
// one's remainder is 0) and the difference taken before the base is: scores become exponents, against the base
// that is returned.  A wave takes this way for a tile where one of its rows' bases is beyond kFar, where a rounded product
// is off by at most 2^-4, no more than the sum of a score in 32 bits.
template <typename T, int N>
__device__ inline float from_maximum(v4f (&s)[N], float m, float scale) {
#pragma clang fp contract(off)
    const float top = m == kNegInf ? 0.f : m;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = s[k][i] * scale;
            s[k][i] = x - top;
        }
    return -Type<T>::kLift;
}

// Cache rows of a tile: 16 KiB of K and as much of V, at most 64 rows (a set of them is 64 bits).
constexpr int tile_rows(int row_bytes) { return row_bytes < 256 ? 64 : 16384 / row_bytes; }
// A workgroup of the row kernel: its waves, and tiles of 16 query rows per wave, by its query rows.  Two tiles per wave
// halve the LDS reads per product; rows of 512 bytes and more leave room for one (its outputs and queries alone are
// 96 registers and more), and so do float32 ones (two lanes of 64 nodes, 4 heads each, D = 64, 88 rows: 40 us with 256
// query rows, 16 with 128).  Eight waves share a tile's loads and staging registers.
constexpr int group_waves(int rows) { return rows == 64 ? 4 : 8; }
constexpr int group_tiles(int rows) { return rows == 256 ? 2 : 1; }

// A tile row of D values in LDS is D * sizeof(T) / 16 chunks of 16 bytes; chunk c of row r is kept
// at place c ^ swizzle(r).  Eight lanes that read one column of eight rows (the first product) and sixteen that
// read a 32-byte piece of four rows each (the second) then use distinct banks; the latter need the rows' pieces
// two chunks apart (with r & 15 instead, rows 2k and 2k + 1 shared theirs: V reads took twice as long).
template <int kRowBytes>
__device__ inline int swizzle(int r) {
    return kRowBytes == 128 ? ((r >> 1) & 3) << 1 : (r & 7) << 1;
}
// kTurned: for a 4-bit cache's tile of 16-bit values, whose lanes write several chunks in a row each: eight lanes write at a
// time, to 32 banks, and would share them two or four at a time, as all are at the same one of their chunks.  So
// chunks are placed one (and two) further along by the bits of their number (a row of 128 bytes: the row's) that tell
// those lanes apart; what is read together has the same such bits.  (Without: 44% of the LDS time of chunks at
// D = 256 are conflicts, 23% of that of trees of 64 rows at D = 128; the chunks 1472 us and 1226.)
template <int kRowBytes, bool kTurned = false>
__device__ inline int lds_at(int r, int chunk) {
    int at = chunk ^ swizzle<kRowBytes>(r);
    if constexpr (kTurned) at ^= kRowBytes == 512 ? (chunk >> 3) & 3 : kRowBytes == 256 ? (chunk >> 3) & 1 : r & 1;
    return r * kRowBytes + (at << 4);
}
template <typename T, bool kFour = true>
constexpr bool turned() { return kFour && sizeof(T) == 2; }

// The left operand of the second product: contraction step u (32 cache rows of a 16-bit tile, 16
// of a 32-bit one) and output columns 16 dt .. 16 dt + 15.  Slot j = 4t + i of lane group g is cache
// row 32u + 16t + 4g + i (t = 0 only for 32-bit).
// (kPairs false: 16 cache rows of a 16-bit tile, in the first two words.)
template <typename T, int D, bool kPairs = true, bool kFour = false>
__device__ inline v4i v_operand(const char *vt, int u, int dt, int lane) {
    constexpr int RB = D * sizeof(T);
    const int g = lane >> 4, n = lane & 15;
    if constexpr (sizeof(T) == 2) {
        v2i part[2] = {};
#pragma unroll
        for (int t = 0; t < (kPairs ? 2 : 1); ++t) {
            const int row = (kPairs ? 32 : 16) * u + 16 * t + 4 * g + (n >> 2);
            const char *p = vt + lds_at<RB, turned<T, kFour>()>(row, 2 * dt + ((n & 3) >> 1)) + 8 * (n & 1);
            part[t] = __builtin_bit_cast(
                v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4 *)p));
        }
        return v4i{part[0][0], part[0][1], part[1][0], part[1][1]};
    } else {
        v4i r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = *reinterpret_cast<const int *>(vt + lds_at<RB>(16 * u + 4 * g + i, 4 * dt + (n >> 2)) + 4 * (n & 3));
        return r;
    }
}

// Replaces the values of an operand that are infinite or NaN by zeros; whether there was one.
template <typename T>
__device__ inline bool drop_nonfinite(v4i &f) {
    bool any = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const unsigned w = (unsigned)f[j];
        if constexpr (sizeof(T) == 2) {
            const bool lo = (w & Type<T>::kExp) == Type<T>::kExp, hi = ((w >> 16) & Type<T>::kExp) == Type<T>::kExp;
            any |= lo | hi;
            f[j] = (int)((lo ? 0u : w & 0xffffu) | (hi ? 0u : w & 0xffff0000u));
        } else {
            const bool b = (w & Type<T>::kExp) == Type<T>::kExp;
            any |= b;
            f[j] = b ? 0 : (int)w;
        }
    }
    return any;
}

// One where a value is infinite with this sign, or NaN; zero elsewhere.
template <typename T>
__device__ inline v4i nonfinite_ones(v4i f, bool negative) {
    constexpr unsigned E = Type<T>::kExp, S = sizeof(T) == 2 ? 0x8000u : 0x80000000u, one = Type<T>::kOne;
    auto is = [&](unsigned x) { return (x & E) == E && ((x & (S - 1u)) != E || ((x & S) != 0) == negative); };
    v4i r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const unsigned w = (unsigned)f[j];
        if constexpr (sizeof(T) == 2)
            r[j] = (int)((is(w & 0xffffu) ? one : 0u) | (is(w >> 16) ? one << 16 : 0u));
        else
            r[j] = (int)(is(w) ? one : 0u);
    }
    return r;
}

// The lowest k bits, k of any sign and size
__device__ inline unsigned long long low_bits(int k) { return k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1ull; }

__device__ inline float lane_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ inline float lane_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// What rows r0 .. r0 + rows - 1 of a lane's N_c * G query rows attend to at most: cache rows
// 0 .. end - 1, divided into parts of whole tiles.
struct Reach {
    int end, part;
};
__device__ inline Reach reach(bool tree, int len, int nodes, int last_token, int splits, int tok) {
    const int end = len + (tree ? nodes : min(last_token, nodes - 1) + 1);
    const int tiles = (end + tok - 1) / tok;
    return Reach{end, (tiles + splits - 1) / splits * tok};
}

template <typename T>
__device__ inline void store4(T *p, v4f v) {
    typedef T t4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<t4 *>(p) = t4{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
}
template <typename T>
__device__ inline v4f load4(const T *p) {
    typedef T t4 __attribute__((ext_vector_type(4)));
    const t4 v = *reinterpret_cast<const t4 *>(p);
    return v4f{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}
__device__ inline float gated(float o, float z, int mode) { return o * (mode == 0 ? fast_silu(z) : fast_sigmoid(z)); }

// The cache rows of a tile of at most 64: lane j of a wave finds row t + j from its page id (requested a tile
// earlier), the others' rows come by a lane shuffle.  `have`: the rows before t1 that lie in a page of the pool, as a
// bit set, the same in every wave; any other row stands for the pool's first one, so that every load is in bounds.
struct TileRows {
    unsigned long long have;
    uint32_t mine;
    __device__ uint32_t at(int j) const { return (uint32_t)__shfl((int)mine, j); }
};
template <int kTok>
__device__ inline TileRows tile_rows_of(const AttnDims &d, int t, int t1, int pid, int h) {
    const int lane = threadIdx.x & 63;
    const uint32_t tk = t + lane;
    const bool ok = (lane < kTok) & ((int)tk < t1) & ((unsigned)pid < (unsigned)d.n_pages);
    return TileRows{__builtin_amdgcn_ballot_w64(ok), ok ? cache_row(d, pid, h, tk, d.page(tk)) : 0u};
}
template <int kTok>
__device__ inline unsigned long long rows_absent(unsigned long long have, int t, int t1) {
    return low_bits(min(kTok, t1 - t)) & ~have;
}

// What a workgroup leaves for the join, one pair per (split, query row) behind the partial outputs: the running
// maximum and sum; maximum -inf and sum 0 where the part holds nothing; a NaN maximum where the row is absent or its
// lane is not computed, so that the join looks at nothing else of the lane.
__device__ inline float *join_pairs(const AttnArgs &a, const AttnPlan &plan) {
    return a.workspace + (size_t)plan.splits * a.d.C * a.d.N * a.d.Hq * a.d.D;
}
// The same pair for rows r0 .. r0 + n - 1 of a (lane, kv head), by the whole workgroup.
__device__ inline void leave_nothing(const AttnArgs &a, const AttnPlan &plan, int split, int c, int h, int r0, int n, float mx) {
    const AttnDims &d = a.d;
    const int per = d.N * d.G;
    float *p = join_pairs(a, plan) + 2 * ((size_t)split * d.C * d.N * d.Hq + ((size_t)c * d.Hkv + h) * per);
    for (int r = r0 + (int)threadIdx.x; r < min(r0 + n, per); r += blockDim.x) {
        p[2 * r] = mx;
        p[2 * r + 1] = 0.f;
    }
}

// ---- 4-bit rows: D / 2 bytes of codes, the lower nibble first, and D / 32 bytes of scales
// B bytes of codes of a row (8: half a block of 32 values, 16: a block) and their scale
template <int B>
struct Codes {
    typedef int words __attribute__((ext_vector_type(B / 4)));
    words w;
    unsigned scale;
    // piece `part` of a row
    template <int D>
    __device__ void load(const void *codes, const void *scales, uint32_t row, int part) {
        w = *reinterpret_cast<const words *>(static_cast<const char *>(codes) + (size_t)row * (D / 2) + B * part);
        scale = static_cast<const unsigned char *>(scales)[(size_t)row * (D / 32) + B * part / 16];
    }
    // its values into a tile row of LDS
    template <typename T, int D>
    __device__ void store(char *tile, int r, int part) const {
        constexpr int H = sizeof(T) == 2 ? 1 : 2;  // chunks a word of codes
#pragma unroll
        for (int j = 0; j < B / 4; ++j)
#pragma unroll
            for (int h = 0; h < H; ++h)
                *reinterpret_cast<v4i *>(tile + lds_at<D * sizeof(T), turned<T>()>(r, (B / 4 * part + j) * H + h)) = four_values<T>(w[j], scale, h);
    }
    // zeros for a row without a page
    __device__ void drop(bool ok) {
#pragma unroll
        for (int j = 0; j < B / 4; ++j) w[j] = ok ? w[j] : 0;
        scale = ok ? scale : 127u;
    }
};

// A workgroup's share of a tile of K and of V: pieces of 16 bytes where there are enough of them for every thread, else
// of 8; with fewer pieces than threads, the lower half of the threads carries K and the upper half V.
template <typename T, int D, int TOK, int THREADS>
struct FourTile {
    static constexpr int B = TOK * D / 32 >= THREADS ? 16 : 8, PPR = D / 2 / B, ALL = TOK * PPR;
    static constexpr bool kBoth = ALL >= THREADS;
    static constexpr int NP = kBoth ? ALL / THREADS : 1;
    static constexpr unsigned long long kAll = TOK == 64 ? ~0ull : (1ull << TOK) - 1ull;
    static_assert(kBoth ? ALL % THREADS == 0 : 2 * ALL == THREADS, "");
    Codes<B> k[NP], v[kBoth ? NP : 1];
    template <typename Rows>
    __device__ void load_k(const AttnArgs &a, const Rows &rows) {
        const bool mine = kBoth || threadIdx.x < ALL;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int at = (int)threadIdx.x % ALL + THREADS * p;
            k[p].template load<D>(mine ? a.k_cache : a.v_cache, mine ? a.k_scales : a.v_scales, rows.at(at / PPR), at % PPR);
        }
    }
    template <typename Rows>
    __device__ void load_v(const AttnArgs &a, const Rows &rows) {
        if constexpr (kBoth)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int at = (int)threadIdx.x + THREADS * p;
                v[p].template load<D>(a.v_cache, a.v_scales, rows.at(at / PPR), at % PPR);
            }
    }
    __device__ void store_k(unsigned long long have, char *s_k, char *s_v) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int at = (int)threadIdx.x % ALL + THREADS * p, r = at / PPR;
            if (have != kAll) k[p].drop((have >> r) & 1);
            k[p].template store<T, D>(kBoth || threadIdx.x < ALL ? s_k : s_v, r, at % PPR);
        }
    }
    __device__ void store_v(unsigned long long have, char *s_v) {
        if constexpr (kBoth)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int at = (int)threadIdx.x + THREADS * p, r = at / PPR;
                if (have != kAll) v[p].drop((have >> r) & 1);
                v[p].template store<T, D>(s_v, r, at % PPR);
            }
    }
};

// Query rows split over the waves (16 RT each), cache tiles shared through LDS: each wave's products
// read the tile once, so the LDS traffic per product falls with RT.  Two tiles of LDS, one barrier
// per tile: the next tile's rows are loaded to registers while the current one is worked on (its page
// ids a tile earlier) and written to the other half before the barrier.
//
// Bound by the products and the softmax beside them where there are many rows: a prompt of 4096 (32 / 8 heads of
// 128, bfloat16) takes 155 us, 887 TFLOP/s; the matrix pipes are busy 38% of the time and the vector units, two thirds
// of it exponentials, about half, two waves a SIMD covering for each other.  Bound by bytes where there are few: trees
// of 4 x 16 nodes behind 8192 tokens 34 us, 4.0 TB/s.  256 rows a workgroup instead of 128 took the prompt from 233
// to 205 us (staging registers and page look-ups shared by twice the rows), operands read four products ahead 205 to 195.
constexpr int group_blocks(int value_bytes, int rows) { return value_bytes == 4 && rows == 64 ? 1 : 2; }  // waves a SIMD, at least

template <typename T, int D, int BM, bool kFour>
__global__ __launch_bounds__(64 * group_waves(BM), group_blocks(sizeof(T), BM)) void attn_rows_kernel(AttnArgs a, AttnPlan plan) {
    constexpr int RB = D * sizeof(T), TOK = tile_rows(RB), kWaves = group_waves(BM), kThreads = 64 * kWaves, RT = group_tiles(BM), NT = TOK / 16, NS = RB / 64, ND = D / 16;
    constexpr int TPR = RB / 16, RPP = kThreads / TPR, NP = TOK / RPP;  // staging: threads per row, rows a pass, passes
    static_assert(BM == 16 * RT * kWaves && RPP <= TOK, "");
    constexpr int NU = sizeof(T) == 2 ? TOK / 32 : TOK / 16;
    __shared__ __attribute__((aligned(16))) char s_kv[2][2][TOK * RB];

    const AttnDims &d = a.d;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane >> 4;
    const bool tree = a.l.parents != nullptr;
    // Workgroups that share a (lane, kv head) read the same cache rows: with several row tiles,
    // consecutive units of work go to one XCD (workgroups are dealt to the 8 XCDs in turn).
    unsigned b = blockIdx.x;
    const unsigned units = (unsigned)d.C * d.Hkv * plan.tiles * plan.splits;
    if (plan.tiles > 1) b = (b & 7) * (gridDim.x >> 3) + (b >> 3);
    if (b >= units) return;
    const int split = b % plan.splits;
    // heavy row tiles of a chain (the last tokens) first
    const int tile = plan.tiles - 1 - (b / plan.splits) % plan.tiles;
    const int ch = b / (plan.splits * plan.tiles), h = ch % d.Hkv, c = ch / d.Hkv, r0 = tile * BM;
    const float skip = __builtin_nanf("");

    const Lane ln = paged_lane(d, a.l, c);
    if (ln.slot == -1) {
        if (plan.splits > 1) leave_nothing(a, plan, split, c, h, r0, BM, skip);
        return;
    }
    int bits = ln.bits;
    unsigned anc = 0;
    if (tree && !(bits & GDN_STATUS_NODES)) {
        bool bad;
        anc = tree_ancestors(a.l.parents + (int64_t)c * d.N, ln.nodes, bad);
        if (bad) bits |= GDN_STATUS_PARENT;
    }
    if (bits) {
        if (a.l.status && split == 0 && tile == 0 && h == 0 && tid == 0) atomicOr(a.l.status, bits);
        if (plan.splits > 1) leave_nothing(a, plan, split, c, h, r0, BM, skip);
        return;
    }
    const int rows = ln.nodes * d.G, L = ln.len;
    if (plan.splits > 1 && rows < r0 + BM) leave_nothing(a, plan, split, c, h, max(r0, rows), BM, skip);
    if (r0 >= rows) return;
    const Reach rc = reach(tree, L, ln.nodes, (r0 + BM - 1) / d.G, plan.splits, TOK);
    const int t0 = split * rc.part, t1 = min(t0 + rc.part, rc.end);
    if (t0 >= t1) {  // (only with several splits)
        leave_nothing(a, plan, split, c, h, r0, min(BM, rows - r0), kNegInf);
        return;
    }

    // ---- this wave's query rows (zeros behind the last one) and what they attend to
    const int rw = r0 + wave * 16 * RT;
    const bool working = rw < rows;
    const int last_token = min(rw + 16 * RT - 1, rows - 1) / d.G;
    v4i qf[RT][NS];
    int token[RT];
    unsigned sees[RT];  // tree: the nodes a row attends to
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = rw + 16 * rt + (lane & 15);
        token[rt] = min(r, rows - 1) / d.G;
        sees[rt] = __shfl(anc, token[rt] & 63);
        const int gh = min(r, rows - 1) - token[rt] * d.G;
        const T *q = static_cast<const T *>(a.q) + (((int64_t)c * d.N + token[rt]) * d.Hq + h * d.G + gh) * D;
#pragma unroll
        for (int ks = 0; ks < NS; ++ks) {
            const v4i v = *reinterpret_cast<const v4i *>(reinterpret_cast<const char *>(q) + 64 * ks + 16 * g);
            qf[rt][ks] = r < rows ? v : v4i{0, 0, 0, 0};
        }
    }

    // ---- staging: thread tid carries chunk tid % TPR of rows tid / TPR + RPP p of the tile
    const int32_t *table = a.l.page_table + (int64_t)ln.slot * d.max_pages;
    const int chunk = tid % TPR, row_in = tid / TPR;
    v4i kr[NP], vr[NP];
    FourTile<T, D, TOK, kThreads> four;
    auto lookup = [&](int t) { return table[d.page((uint32_t)min(t + lane, t1 - 1))]; };
    auto load = [&](int t, int pid) {
        const TileRows rows = tile_rows_of<TOK>(d, t, t1, pid, h);
        if constexpr (kFour) {
            four.load_k(a, rows);
            four.load_v(a, rows);
        } else {
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const size_t at = (size_t)rows.at(row_in + RPP * p) * RB + chunk * 16;
                kr[p] = *reinterpret_cast<const v4i *>(static_cast<const char *>(a.k_cache) + at);
                vr[p] = *reinterpret_cast<const v4i *>(static_cast<const char *>(a.v_cache) + at);
            }
        }
        return rows.have;
    };
    // The rows of the tile behind t, and the page ids of the one behind that
    int pid = lookup(t0);
    unsigned long long have = load(t0, pid);
    pid = lookup(t0 + TOK);
    auto request = [&](int t) {
        if (t + TOK < t1) {
            have = load(t + TOK, pid);
            pid = lookup(t + 2 * TOK);
        }
    };

    v4f o[RT][ND];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = kNegInf;
        l[rt] = 0.f;
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) o[rt][dt] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    // One tile for this wave.  `masked`: some row does not attend to some of it.
    auto work = [&](auto masked, const char *s_k, const char *s_v, int t, unsigned long long gone) {
        constexpr bool kMasked = decltype(masked)::value;
        request(t);
        // ---- S^T = K Q^T
        v4f s[RT][NT];
        constexpr int kDeep = 4;  // operands read ahead of their products
        {
            constexpr int kSteps = NS * NT;  // (contraction outermost: the products of one score tile depend on each other)
            auto operand = [&](int k) {
                return *reinterpret_cast<const v4i *>(s_k + lds_at<RB, turned<T, kFour>()>(16 * (k % NT) + (lane & 15), 4 * (k / NT) + g));
            };
            v4i kf[kDeep];
#pragma unroll
            for (int k = 0; k < kDeep; ++k) kf[k] = operand(k);
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    s[rt][k % NT] = Type<T>::mma(kf[k % kDeep], qf[rt][k / NT], k >= NT ? s[rt][k % NT] : v4f{0.f, 0.f, 0.f, 0.f});
                if (k + kDeep < kSteps) kf[k % kDeep] = operand(k + kDeep);
                __builtin_amdgcn_sched_barrier(kArithmetic);
            }
        }
        // ---- rows that are not attended weigh nothing, whatever their scores are: the tile's rows that a query
        // row attends to as a bit set, shifted so that this lane's rows are bits 16 tt + i
        unsigned long long see[RT];
        if constexpr (kMasked) {
            int g4 = 4 * g;
            asm volatile("" : "+v"(g4));  // (keeps what follows out of the other tiles' registers)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const int rel = L - t;
                unsigned long long x = low_bits(min(tree ? rel : rel + token[rt] + 1, t1 - t));
                if (tree) {
                    const unsigned long long nodes = sees[rt];
                    x |= (rel >= 64 || rel <= -32 ? 0 : rel >= 0 ? nodes << rel : nodes >> -rel) & low_bits(t1 - t);
                }
                see[rt] = (x & ~gone) >> g4;
#pragma unroll
                for (int tt = 0; tt < NT; ++tt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[rt][tt][i] = (see[rt] >> (16 * tt + i)) & 1 ? s[rt][tt][i] : kNegInf;
            }
        }
        // ---- running maximum and sum; the sum keeps the weights unrounded.  The base of the exponentials follows
        // the maximum only when that has grown by more than 2^kSlack: weights up to 2^kSlack lose nothing (their
        // relative rounding is the same), and most tiles need no rescaling of o.
        float mx[RT];
        bool lead = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            mx[rt] = kNegInf;
#pragma unroll
            for (int tt = 0; tt < NT; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[rt] = fmaxf(mx[rt], s[rt][tt][i]);
            mx[rt] = lane_max(mx[rt]) * a.scale_log2;
            lead |= mx[rt] > m[rt] + kSlack;  // (a first score is more than -inf + kSlack)
        }
        if (__builtin_amdgcn_ballot_w64(lead)) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const float to = fmaxf(m[rt], mx[rt]), base = to == kNegInf ? 0.f : to;
                const float shrink = __builtin_amdgcn_exp2f(m[rt] - base);
                m[rt] = to;
                l[rt] *= shrink;
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) o[rt][dt] *= shrink;
            }
        }
        float base[RT], scale = a.scale_log2;
        bool far = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            base[rt] = weight_base<T>(m[rt]);
            far |= fabsf(base[rt]) > kFar;
        }
        if (__builtin_amdgcn_ballot_w64(far)) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) base[rt] = from_maximum<T>(s[rt], m[rt], scale);
            scale = 1.f;
        }
        auto weigh = [&](int rt, int e) {  // score e of this lane becomes its weight
            const float x = __builtin_amdgcn_exp2f(fmaf(s[rt][e >> 2][e & 3], scale, -base[rt]));
            s[rt][e >> 2][e & 3] = x;
            l[rt] += x;
        };
        // ---- O^T += V^T P^T, operand reads kDeep steps ahead of their products (left to itself the compiler reads
        // one operand, waits for it and goes on), and the weights of the next step of the contraction a few at a
        // time beside the products of this one
        bool strange = false;
        constexpr int kSteps = NU * ND;
        constexpr int kScores = 4 * NT / NU, kPart = (kScores + ND - 1) / ND;  // a step's scores per query row, and per product
        v4i vf[kDeep], pf[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < kScores; ++e) weigh(rt, e);
#pragma unroll
        for (int k = 0; k < kDeep; ++k) vf[k] = v_operand<T, D, true, kFour>(s_v, k / ND, k % ND, lane);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int u = k / ND, dt = k % ND;
            if (dt == 0) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    if constexpr (sizeof(T) == 2)
                        pf[rt] = Type<T>::pack(s[rt][2 * u], s[rt][2 * u + 1]);
                    else
                        pf[rt] = __builtin_bit_cast(v4i, s[rt][u]);
                }
            }
            if constexpr (kMasked) strange |= drop_nonfinite<T>(vf[k % kDeep]);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) o[rt][dt] = Type<T>::mma(vf[k % kDeep], pf[rt], o[rt][dt]);
            if (k + kDeep < kSteps) vf[k % kDeep] = v_operand<T, D, true, kFour>(s_v, (k + kDeep) / ND, (k + kDeep) % ND, lane);
            if (u + 1 < NU)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int e = kPart * dt; e < kPart * dt + kPart && e < kScores; ++e) weigh(rt, kScores * (u + 1) + e);
            if constexpr (!kMasked) __builtin_amdgcn_sched_barrier(0);
        }
        // A weight of zero times an infinity or NaN is NaN: such values were left out above.  They go to the
        // rows that do attend to them by two products of ones (values of +inf or NaN, of -inf or NaN) with
        // ones (rows attended): a positive count adds +inf, -inf, and both together NaN.
        if constexpr (kMasked)
            if (__builtin_amdgcn_ballot_w64(strange)) {
#pragma unroll 1
                for (int side = 0; side < 2; ++side) {
                    const float inf = side ? kNegInf : -kNegInf;
#pragma unroll
                    for (int u = 0; u < NU; ++u) {
                        v4i reads[RT];
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            float one[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                one[j] = (see[rt] >> ((sizeof(T) == 2 ? 32 * u + 16 * (j >> 2) : 16 * u) + (j & 3))) & 1 ? 1.f : 0.f;
                            const v4f lo{one[0], one[1], one[2], one[3]}, hi{one[4], one[5], one[6], one[7]};
                            if constexpr (sizeof(T) == 2)
                                reads[rt] = Type<T>::pack(lo, hi);
                            else
                                reads[rt] = __builtin_bit_cast(v4i, lo);
                        }
#pragma unroll
                        for (int dt = 0; dt < ND; ++dt) {
                            const v4i vf = nonfinite_ones<T>(v_operand<T, D, true, kFour>(s_v, u, dt, lane), side);
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt) {
                                const v4f n = Type<T>::mma(vf, reads[rt], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                                for (int i = 0; i < 4; ++i) o[rt][dt][i] += n[i] > 0.f ? inf : 0.f;
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                }
            }
    };

    // Writes the loaded tile to LDS (rows without a page as zeros) and waits for the workgroup: the tile's absent rows.
    auto turn = [&](int t, char *s_k, char *s_v) {
        const unsigned long long gone = rows_absent<TOK>(have, t, t1);
        if (gone || t + TOK > t1) {
#pragma unroll
            for (int p = 0; p < (kFour ? 0 : NP); ++p) {
                const bool ok = (have >> (row_in + RPP * p)) & 1;
                kr[p] = v4i{ok ? kr[p][0] : 0, ok ? kr[p][1] : 0, ok ? kr[p][2] : 0, ok ? kr[p][3] : 0};
                vr[p] = v4i{ok ? vr[p][0] : 0, ok ? vr[p][1] : 0, ok ? vr[p][2] : 0, ok ? vr[p][3] : 0};
            }
            if (gone && tid == 0 && a.l.status) atomicOr(a.l.status, GDN_STATUS_PAGE);
        }
        if constexpr (kFour) {
            four.store_k(have, s_k, s_v);
            four.store_v(have, s_v);
        } else {
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int at = lds_at<RB>(row_in + RPP * p, chunk);
                *reinterpret_cast<v4i *>(s_k + at) = kr[p];
                *reinterpret_cast<v4i *>(s_v + at) = vr[p];
            }
        }
        lds_barrier();
        return gone;
    };
    // First the tiles that every row of the workgroup attends to throughout, without a trace of the masks; from
    // the first other one on (the diagonal, the draft tree, a row without a page) the tiles with masks.
    const int all_see = min(tree ? L : L + r0 / d.G + 1, t1);
    int t = t0, half = 0;
    unsigned long long gone = 0;
    bool turned = false;
    for (; t + TOK <= all_see; t += TOK, half ^= 1) {
        gone = turn(t, s_kv[half][0], s_kv[half][1]);
        if (gone) {
            turned = true;
            break;
        }
        if (working)
            work(std::false_type{}, s_kv[half][0], s_kv[half][1], t, 0ull);
        else
            request(t);
    }
    for (; t < t1; t += TOK, half ^= 1) {
        if (!turned) gone = turn(t, s_kv[half][0], s_kv[half][1]);
        turned = false;
        if (working && (tree || t <= L + last_token))
            work(std::true_type{}, s_kv[half][0], s_kv[half][1], t, gone);
        else
            request(t);
    }

    // ---- results: lane holds columns 16 dt + 4g .. + 3 of its query row
    const size_t all_rows = (size_t)d.C * d.N * d.Hq;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = rw + 16 * rt + (lane & 15);
        const float sum = lane_sum(l[rt]);
        if (r >= rows) continue;
        if (plan.splits > 1) {  // unnormalised part: [split][row][D], then (maximum, sum) per row
            const size_t row = (size_t)split * all_rows + ((size_t)c * d.Hkv + h) * d.N * d.G + r;
            float *po = a.workspace + row * D;
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) *reinterpret_cast<v4f *>(po + 16 * dt + 4 * g) = o[rt][dt];
            if (g == 0) {
                float *ml = join_pairs(a, plan) + row * 2;
                ml[0] = m[rt];
                ml[1] = sum;
            }
            continue;
        }
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        const int64_t node = (int64_t)c * d.N + token[rt];
        const int head = h * d.G + r - token[rt] * d.G;
        T *out = static_cast<T *>(a.out) + (node * d.Hq + head) * D;
        const T *z = static_cast<const T *>(a.gate.p) + node * a.gate.token + head * a.gate.head;
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) {
            v4f v = sum == 0.f ? v4f{0.f, 0.f, 0.f, 0.f} : o[rt][dt] * inv;
            if (a.gate.p && sum != 0.f) {  // (zeros where nothing was attended, whatever the gate)
                const v4f zz = load4(z + 16 * dt + 4 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = gated(v[i], zz[i], a.gate_mode);
            }
            store4(out + 16 * dt + 4 * g, v);
        }
    }
}

// Wide rows (512 bytes: 16-bit values of 256 columns), more query rows than the kernel for few.
//
// A wave that owns 32 query rows of this width would hold 128 registers of outputs and 64 of queries, and one that
// owns 16 reads 64 bytes of LDS per product instruction, twice what the LDS delivers.  So a pair of waves shares 32
// query rows: each computes the scores of one half of a tile's 64 cache rows against the whole width, the pair
// exchanges its rows' maxima and the weights (8 KiB a tile through LDS), and each multiplies all of the weights with
// its half of the columns of V.  Per product a wave reads half as much LDS as with 16 rows, and holds 64 registers
// of outputs.  Chunks of 2 x 2048 tokens behind 16k (16 / 2 heads, bfloat16) take 1277 us, 697 TFLOP/s (a wave with 16 rows:
// 1544 us); the matrix pipes are busy 37% of the time, and the two barriers keep the eight waves in step, so that
// products and softmax overlap little.  Two barriers a tile: behind the maxima, where K has been read and V of the tile is written, and behind
// the weights, where K of the next tile is.
constexpr int kPairRows = 128, kPairThreads = 512;

// The text below is the kernel itself over 16 bits, and a function that the kernel calls over 4: the registers that the compiler
// keeps in memory are others, by no rule to be seen from here (as this was chosen, the chunks above as kernel and as
// function: over 16 bits 1277 us and 1290, over 4 bits 1290 and 1248).
template <typename T, bool kFour>
__global__ void attn_pair_kernel(AttnArgs a, AttnPlan plan);
#ifndef GDN_ATTN_PAIR
#define GDN_ATTN_PAIR __global__ __launch_bounds__(kPairThreads, 2) void attn_pair_kernel
#endif
template <typename T, bool kFour>
GDN_ATTN_PAIR(AttnArgs a, AttnPlan plan) {
    constexpr int D = 256, RB = 512, TOK = 64, RT = 2, NT = 2, NS = RB / 64, ND = 8;  // NT, ND: of this wave's half
    constexpr int BM = kPairRows, TPR = RB / 16, RPP = kPairThreads / TPR, NP = TOK / RPP;
    static_assert(sizeof(T) == 2, "");
    __shared__ __attribute__((aligned(16))) char s_k[TOK * RB], s_vs[2][TOK * RB];
    __shared__ v4i s_p[4][2][RT][64];              // weights as operands: [pair][half][row tile][lane]
    __shared__ float s_mx[4][2][16 * RT], s_l[4][2][16 * RT];

    const AttnDims &d = a.d;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane >> 4, n = lane & 15, pair = wave >> 1, hf = wave & 1;
    const bool tree = a.l.parents != nullptr;
    unsigned b = blockIdx.x;  // (units of work as in the row kernel)
    const unsigned units = (unsigned)d.C * d.Hkv * plan.tiles * plan.splits;
    if (plan.tiles > 1) b = (b & 7) * (gridDim.x >> 3) + (b >> 3);
    if (b >= units) return;
    const int split = b % plan.splits, tile = plan.tiles - 1 - (b / plan.splits) % plan.tiles;
    const int ch = b / (plan.splits * plan.tiles), h = ch % d.Hkv, c = ch / d.Hkv, r0 = tile * BM;
    const float skip = __builtin_nanf("");
    const Lane ln = paged_lane(d, a.l, c);
    if (ln.slot == -1) {
        if (plan.splits > 1) leave_nothing(a, plan, split, c, h, r0, BM, skip);
        return;
    }
    int bits = ln.bits;
    unsigned anc = 0;
    if (tree && !(bits & GDN_STATUS_NODES)) {
        bool bad;
        anc = tree_ancestors(a.l.parents + (int64_t)c * d.N, ln.nodes, bad);
        if (bad) bits |= GDN_STATUS_PARENT;
    }
    if (bits) {
        if (a.l.status && split == 0 && tile == 0 && h == 0 && tid == 0) atomicOr(a.l.status, bits);
        if (plan.splits > 1) leave_nothing(a, plan, split, c, h, r0, BM, skip);
        return;
    }
    const int rows = ln.nodes * d.G, L = ln.len;
    if (plan.splits > 1 && rows < r0 + BM) leave_nothing(a, plan, split, c, h, max(r0, rows), BM, skip);
    if (r0 >= rows) return;
    const Reach rc = reach(tree, L, ln.nodes, (r0 + BM - 1) / d.G, plan.splits, TOK);
    const int t0 = split * rc.part, t1 = min(t0 + rc.part, rc.end);
    if (t0 >= t1) {  // (only with several splits)
        leave_nothing(a, plan, split, c, h, r0, min(BM, rows - r0), kNegInf);
        return;
    }

    // ---- the pair's query rows and what they attend to
    const int rw = r0 + pair * 16 * RT;
    const bool working = rw < rows;
    const int last_token = min(rw + 16 * RT - 1, rows - 1) / d.G;
    v4i qf[RT][NS];
    int token[RT];
    unsigned sees[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = rw + 16 * rt + n;
        token[rt] = min(r, rows - 1) / d.G;
        sees[rt] = __shfl(anc, token[rt] & 63);
        const int gh = min(r, rows - 1) - token[rt] * d.G;
        const T *q = static_cast<const T *>(a.q) + (((int64_t)c * d.N + token[rt]) * d.Hq + h * d.G + gh) * D;
#pragma unroll
        for (int ks = 0; ks < NS; ++ks) {
            const v4i v = *reinterpret_cast<const v4i *>(reinterpret_cast<const char *>(q) + 64 * ks + 16 * g);
            qf[rt][ks] = r < rows ? v : v4i{0, 0, 0, 0};
        }
    }

    // ---- staging as in the row kernel, K and V in turns, so that 16 registers are in use for it at any time
    const int32_t *table = a.l.page_table + (int64_t)ln.slot * d.max_pages;
    const int chunk = tid % TPR, row_in = tid / TPR;
    v4i kr[NP], vr[NP];
    FourTile<T, D, TOK, kPairThreads> four;
    auto lookup = [&](int t) { return table[d.page((uint32_t)min(t + lane, t1 - 1))]; };
    auto load = [&](const TileRows &rows, bool k) {
        if constexpr (kFour) {
            if (k)
                four.load_k(a, rows);
            else
                four.load_v(a, rows);
        } else {
#pragma unroll
            for (int p = 0; p < NP; ++p)
                (k ? kr : vr)[p] = *reinterpret_cast<const v4i *>(static_cast<const char *>(k ? a.k_cache : a.v_cache) +
                                                                  (size_t)rows.at(row_in + RPP * p) * RB + chunk * 16);
        }
    };
    auto stage = [&](bool k, unsigned long long have, char *to) {  // (rows without a page as zeros)
        if constexpr (kFour) {
            if (k)
                four.store_k(have, to, to);
            else
                four.store_v(have, to);
            return;
        }
        v4i *from = k ? kr : vr;
        if (have != ~0ull)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const bool ok = (have >> (row_in + RPP * p)) & 1;
                from[p] = v4i{ok ? from[p][0] : 0, ok ? from[p][1] : 0, ok ? from[p][2] : 0, ok ? from[p][3] : 0};
            }
#pragma unroll
        for (int p = 0; p < NP; ++p) *reinterpret_cast<v4i *>(to + lds_at<RB>(row_in + RPP * p, chunk)) = from[p];
    };

    v4f o[RT][ND];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = kNegInf;
        l[rt] = 0.f;
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) o[rt][dt] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    constexpr int kDeep = 4;  // operands read ahead of their products

    // One tile.  `active`: this pair attends to some of it.  Every wave of the workgroup passes both barriers.
    TileRows now{}, next{};  // of the tile at hand, and of the one behind it
    int pid = lookup(t0);
    auto step = [&](auto masked, int t, char *s_v, bool active) {
        constexpr bool kMasked = decltype(masked)::value;
        const bool more = t + TOK < t1;
        if (more) {
            next = tile_rows_of<TOK>(d, t + TOK, t1, pid, h);
            load(next, true);
        }
        v4f s[RT][NT];
        unsigned long long see[RT];
        float mx[RT];
        if (active) {
            constexpr int kSteps = NS * NT;
            auto operand = [&](int k) {
                return *reinterpret_cast<const v4i *>(s_k + 32 * hf * RB + lds_at<RB, turned<T, kFour>()>(16 * (k % NT) + n, 4 * (k / NT) + g));
            };
            v4i kf[kDeep];
#pragma unroll
            for (int k = 0; k < kDeep; ++k) kf[k] = operand(k);
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    s[rt][k % NT] = Type<T>::mma(kf[k % kDeep], qf[rt][k / NT], k >= NT ? s[rt][k % NT] : v4f{0.f, 0.f, 0.f, 0.f});
                if (k + kDeep < kSteps) kf[k % kDeep] = operand(k + kDeep);
                __builtin_amdgcn_sched_barrier(kArithmetic);
            }
            if constexpr (kMasked) {
                int g4 = 4 * g;
                asm volatile("" : "+v"(g4));  // (keeps what follows out of the other tiles' registers)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const int rel = L - t;
                    unsigned long long x = low_bits(min(tree ? rel : rel + token[rt] + 1, t1 - t));
                    if (tree) {
                        const unsigned long long nodes = sees[rt];
                        x |= (rel >= 64 || rel <= -32 ? 0 : rel >= 0 ? nodes << rel : nodes >> -rel) & low_bits(t1 - t);
                    }
                    see[rt] = (x & now.have) >> g4;
                    const unsigned mine = (unsigned)(see[rt] >> (32 * hf));
#pragma unroll
                    for (int tt = 0; tt < NT; ++tt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[rt][tt][i] = (mine >> (16 * tt + i)) & 1 ? s[rt][tt][i] : kNegInf;
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                mx[rt] = kNegInf;
#pragma unroll
                for (int tt = 0; tt < NT; ++tt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx[rt] = fmaxf(mx[rt], s[rt][tt][i]);
                mx[rt] = lane_max(mx[rt]) * a.scale_log2;
                if (g == 0) s_mx[pair][hf][16 * rt + n] = mx[rt];
            }
        }
        stage(false, now.have, s_v);
        lds_barrier();  // K has been read; the maxima and this tile's V are there
        v4i pf[RT];
        if (active) {
            bool lead = false;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {  // both waves of the pair come to the same maxima and bases
                mx[rt] = fmaxf(mx[rt], s_mx[pair][hf ^ 1][16 * rt + n]);
                lead |= mx[rt] > m[rt] + kSlack;
            }
            if (__builtin_amdgcn_ballot_w64(lead)) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const float to = fmaxf(m[rt], mx[rt]), base = to == kNegInf ? 0.f : to;
                    const float shrink = __builtin_amdgcn_exp2f(m[rt] - base);
                    m[rt] = to;
                    l[rt] *= shrink;
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) o[rt][dt] *= shrink;
                }
            }
            float base[RT], scale = a.scale_log2;
            bool far = false;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                base[rt] = weight_base<T>(m[rt]);
                far |= fabsf(base[rt]) > kFar;
            }
            if (__builtin_amdgcn_ballot_w64(far)) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) base[rt] = from_maximum<T>(s[rt], m[rt], scale);
                scale = 1.f;
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
                for (int tt = 0; tt < NT; ++tt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = __builtin_amdgcn_exp2f(fmaf(s[rt][tt][i], scale, -base[rt]));
                        s[rt][tt][i] = x;
                        l[rt] += x;
                    }
                pf[rt] = Type<T>::pack(s[rt][0], s[rt][1]);
                s_p[pair][hf][rt][lane] = pf[rt];
            }
        }
        if (more) {
            stage(true, next.have, s_k);
            load(next, false);
            pid = lookup(t + 2 * TOK);
            if (tid == 0 && a.l.status && rows_absent<TOK>(next.have, t + TOK, t1)) atomicOr(a.l.status, GDN_STATUS_PAGE);
        }
        now = next;
        lds_barrier();  // the weights and the next tile's K are there
        if (!active) return;
        // ---- O^T += V^T P^T: this wave's half of the columns, its own weights first, then the partner's
        bool strange = false;
        constexpr int kSteps = 2 * ND;
        v4i vf[kDeep], other[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) other[rt] = s_p[pair][hf ^ 1][rt][lane];
        auto operand = [&](int k) { return v_operand<T, D, true, kFour>(s_v + 32 * RB * (k < ND ? hf : hf ^ 1), 0, 8 * hf + k % ND, lane); };
#pragma unroll
        for (int k = 0; k < kDeep; ++k) vf[k] = operand(k);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            if constexpr (kMasked) strange |= drop_nonfinite<T>(vf[k % kDeep]);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) o[rt][k % ND] = Type<T>::mma(vf[k % kDeep], k < ND ? pf[rt] : other[rt], o[rt][k % ND]);
            if (k + kDeep < kSteps) vf[k % kDeep] = operand(k + kDeep);
            if constexpr (!kMasked) __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kMasked)  // infinities and NaN go to the rows that attend to them, as in the row kernel
            if (__builtin_amdgcn_ballot_w64(strange)) {
#pragma unroll 1
                for (int side = 0; side < 4; ++side) {  // +inf and -inf, in either half of the tile
                    const float inf = side & 1 ? kNegInf : -kNegInf;
                    const int half = side >> 1;
                    v4i reads[RT];
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const unsigned at = (unsigned)(see[rt] >> (32 * half));
                        v4f one[2];
#pragma unroll
                        for (int j = 0; j < 8; ++j) one[j >> 2][j & 3] = (at >> (16 * (j >> 2) + (j & 3))) & 1 ? 1.f : 0.f;
                        reads[rt] = Type<T>::pack(one[0], one[1]);
                    }
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) {
                        const v4i f = nonfinite_ones<T>(v_operand<T, D, true, kFour>(s_v + 32 * RB * half, 0, 8 * hf + dt, lane), side & 1);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            const v4f cnt = Type<T>::mma(f, reads[rt], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[rt][dt][i] += cnt[i] > 0.f ? inf : 0.f;
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
    };

    now = tile_rows_of<TOK>(d, t0, t1, pid, h);
    load(now, true);
    load(now, false);
    pid = lookup(t0 + TOK);
    if (tid == 0 && a.l.status && rows_absent<TOK>(now.have, t0, t1)) atomicOr(a.l.status, GDN_STATUS_PAGE);
    stage(true, now.have, s_k);
    lds_barrier();
    // full tiles first, then, from the first one with a mask or an absent row on, the tiles with masks
    const int all_see = min(tree ? L : L + r0 / d.G + 1, t1);
    int t = t0, half = 0;
    for (; t + TOK <= all_see && now.have == ~0ull; t += TOK, half ^= 1) step(std::false_type{}, t, s_vs[half], working);
    for (; t < t1; t += TOK, half ^= 1) step(std::true_type{}, t, s_vs[half], working && (tree || t <= L + last_token));

    // ---- results: this wave's half of the columns
    const size_t all_rows = (size_t)d.C * d.N * d.Hq;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        l[rt] = lane_sum(l[rt]);
        if (g == 0) s_l[pair][hf][16 * rt + n] = l[rt];
    }
    lds_barrier();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = rw + 16 * rt + n;
        // (the halves' sums in one order for both waves)
        const float sum = s_l[pair][0][16 * rt + n] + s_l[pair][1][16 * rt + n];
        if (r >= rows) continue;
        if (plan.splits > 1) {
            const size_t row = (size_t)split * all_rows + ((size_t)c * d.Hkv + h) * d.N * d.G + r;
            float *po = a.workspace + row * D + 128 * hf;
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) *reinterpret_cast<v4f *>(po + 16 * dt + 4 * g) = o[rt][dt];
            if (g == 0 && hf == 0) {
                float *ml = join_pairs(a, plan) + row * 2;
                ml[0] = m[rt];
                ml[1] = sum;
            }
            continue;
        }
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        const int64_t node = (int64_t)c * d.N + token[rt];
        const int head = h * d.G + r - token[rt] * d.G;
        T *out = static_cast<T *>(a.out) + (node * d.Hq + head) * D + 128 * hf;
        const T *z = static_cast<const T *>(a.gate.p) + node * a.gate.token + head * a.gate.head + 128 * hf;
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) {
            v4f v = sum == 0.f ? v4f{0.f, 0.f, 0.f, 0.f} : o[rt][dt] * inv;
            if (a.gate.p && sum != 0.f) {  // (zeros where nothing was attended, whatever the gate)
                const v4f zz = load4(z + 16 * dt + 4 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = gated(v[i], zz[i], a.gate_mode);
            }
            store4(out + 16 * dt + 4 * g, v);
        }
    }
}

// ---- few query rows (at most 16 per (lane, kv head): decode, short drafts with small groups)
//
// The cache is read once and the products are small: bound by bytes, or by latency where the cache is short.
// Every wave takes whole tiles of its own, wave w the tiles w, w + 4, ... of the workgroup's part, and keeps
// a running maximum, sum and output of its own for the 16 rows; the four are joined through LDS at the end.
// So no wave waits for another in the loop.  K rows go from memory straight into operand registers (a lane
// reads 16 bytes of row lane % 16); V rows, whose operand needs four rows of one column, through 8 KiB of LDS
// that only this wave uses.  A tile is 8 KiB of K and of V, 64 registers; the next tile's loads are issued as soon
// as K has gone into the products and V into LDS, and are in flight during the softmax and the second product.
//
// 64 lanes of decode behind 16k..32k tokens (32 / 4 heads of 128, float16): 580 us, 5.6 TB/s (a read of as many bytes
// 510 us); one lane behind 1003 tokens: 7 us, and 3.2 us for the join.
//
// A 4-bit cache has a fourth of the bytes for as many rows: a tile is 16 KiB of V as values (at most 64 rows), so that
// a wave has 2 to 4 KiB of K and of V in flight.  The same 64 lanes over it, 864 MB: 179 us, 4.8 TB/s, 94% of a copy (lanes of
// equal length 158 us, 5.45 TB/s: the last workgroups of a ragged batch run alone); one lane behind 1003 tokens: 7.6 us.  Tiles
// of 8 KiB in three workgroups a CU: 175 us; two tiles in flight: 177.
constexpr int kFewWaves = 4, kFewRows = 16;
constexpr int few_tile(int row_bytes, bool four) { return four ? (row_bytes < 256 ? 64 : 16384 / row_bytes) : 8192 / row_bytes; }

// Workgroups a CU.  Float32 rows of 256 4-bit values: one, whose waves use 414 registers; within the 256 of two, 95 of them go
// through memory (ragged lanes, D = 256, with two and with one: 32 of decode up to 8192 tokens 639 us and 308, five of eight
// nodes up to 2999 97 and 51, one of decode at 1000 20.5 and 15.7).  Narrower ones keep two, with 15 and 27 registers in
// memory (the 32 lanes at D = 64 55 us and 69, at D = 128 106 and 133).
constexpr int few_blocks(int row_bytes, bool four) { return four && row_bytes == 1024 ? 1 : 2; }

template <typename T, int D, bool kFour>
__global__ __launch_bounds__(64 * kFewWaves, few_blocks(D * sizeof(T), kFour)) void attn_few_kernel(AttnArgs a, AttnPlan plan) {
    constexpr int RB = D * sizeof(T), TOK = few_tile(RB, kFour), NT = TOK / 16, NS = RB / 64, ND = D / 16;
    constexpr int TPR = RB / 16, RPP = kFour ? 64 / (D / 32) : 64 / TPR, NP = TOK / RPP;
    constexpr bool kPairs = sizeof(T) == 2 && TOK >= 32;  // the second product in steps of 32 rows
    constexpr int NU = kPairs ? TOK / 32 : NT;
    constexpr int kTile = kFour ? TOK * RB : 8192;
    constexpr int kBuf = 16 * D * 4 > kTile ? 16 * D * 4 : kTile;  // a wave's V tile, at the end its output
    // 4 bits: lane group g of the first product takes the row's values kRun g .. kRun g + kRun - 1
    constexpr int kRun = D / 4, kWords = kRun / 8, kScales = kRun > 32 ? 2 : 1, VPS = 16 / sizeof(T);
    constexpr unsigned long long kFull = TOK == 64 ? ~0ull : (1ull << TOK) - 1ull;
    __shared__ __attribute__((aligned(16))) char s_buf[kFewWaves][kBuf];
    __shared__ float s_m[kFewWaves][16], s_l[kFewWaves][16];

    const AttnDims &d = a.d;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const bool tree = a.l.parents != nullptr;
    const unsigned b = blockIdx.x;
    const int split = b % plan.splits, ch = b / plan.splits, h = ch % d.Hkv, c = ch / d.Hkv;
    const float skip = __builtin_nanf("");
    const Lane ln = paged_lane(d, a.l, c);
    if (ln.slot == -1) {
        if (plan.splits > 1) leave_nothing(a, plan, split, c, h, 0, kFewRows, skip);
        return;
    }
    int bits = ln.bits;
    unsigned anc = 0;
    if (tree && !(bits & GDN_STATUS_NODES)) {
        bool bad;
        anc = tree_ancestors(a.l.parents + (int64_t)c * d.N, ln.nodes, bad);
        if (bad) bits |= GDN_STATUS_PARENT;
    }
    if (bits) {
        if (a.l.status && split == 0 && h == 0 && tid == 0) atomicOr(a.l.status, bits);
        if (plan.splits > 1) leave_nothing(a, plan, split, c, h, 0, kFewRows, skip);
        return;
    }
    const int rows = ln.nodes * d.G, L = ln.len;
    if (plan.splits > 1) leave_nothing(a, plan, split, c, h, rows, kFewRows, skip);
    if (rows == 0) return;
    const Reach rc = reach(tree, L, ln.nodes, ln.nodes - 1, plan.splits, TOK * kFewWaves);
    const int t0 = split * rc.part, t1 = min(t0 + rc.part, rc.end);
    if (t0 >= t1) {  // (only with several splits)
        leave_nothing(a, plan, split, c, h, 0, rows, kNegInf);
        return;
    }

    const int r = min(n, rows - 1), token = r / d.G;
    const unsigned sees = __shfl(anc, token & 63);
    const int64_t node = (int64_t)c * d.N + token;
    const int head = h * d.G + r - token * d.G;
    v4i qf[NS];
    {
        const char *q = reinterpret_cast<const char *>(static_cast<const T *>(a.q) + (node * d.Hq + head) * D);
#pragma unroll
        for (int ks = 0; ks < NS; ++ks) qf[ks] = *reinterpret_cast<const v4i *>(q + (kFour ? kRun * sizeof(T) * g + 16 * ks : 64 * ks + 16 * g));
    }

    const int32_t *table = a.l.page_table + (int64_t)ln.slot * d.max_pages;
    auto fetch = [&](int t) { return table[d.page((uint32_t)min(t + lane, t1 - 1))]; };
    v4i kr[kFour ? 1 : NT * NS], vr[kFour ? 1 : NP];
    typedef int run __attribute__((ext_vector_type(kWords)));
    run kc[kFour ? NT : 1];
    unsigned ks4[kFour ? NT : 1][kScales];
    Codes<16> vc[kFour ? NP : 1];
    auto load = [&](int t, int pid) {
        const TileRows rows = tile_rows_of<TOK>(d, t, t1, pid, h);
        if constexpr (kFour) {
#pragma unroll
            for (int tt = 0; tt < NT; ++tt) {
                const size_t row = rows.at(16 * tt + n);
                kc[tt] = *reinterpret_cast<const run *>(static_cast<const char *>(a.k_cache) + row * (D / 2) + kRun / 2 * g);
                const unsigned char *s = static_cast<const unsigned char *>(a.k_scales) + row * (D / 32) + kRun * g / 32;
#pragma unroll
                for (int j = 0; j < kScales; ++j) ks4[tt][j] = s[j];
            }
#pragma unroll
            for (int p = 0; p < NP; ++p)
                vc[p].template load<D>(a.v_cache, a.v_scales, rows.at(RPP * p + lane / (D / 32)), lane % (D / 32));
            return rows.have;
        }
#pragma unroll
        for (int tt = 0; tt < (kFour ? 0 : NT); ++tt) {
            const size_t at = (size_t)rows.at(16 * tt + n) * RB + 16 * g;
#pragma unroll
            for (int ks = 0; ks < NS; ++ks)
                kr[tt * NS + ks] = *reinterpret_cast<const v4i *>(static_cast<const char *>(a.k_cache) + at + 64 * ks);
        }
#pragma unroll
        for (int p = 0; p < (kFour ? 0 : NP); ++p) {
            const size_t at = (size_t)rows.at(RPP * p + lane / TPR) * RB + 16 * (lane % TPR);
            vr[p] = *reinterpret_cast<const v4i *>(static_cast<const char *>(a.v_cache) + at);
        }
        return rows.have;
    };

    v4f o[ND];
    float m = kNegInf, l = 0.f;
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) o[dt] = v4f{0.f, 0.f, 0.f, 0.f};
    constexpr int kStep = TOK * kFewWaves;
    char *s_v = s_buf[wave];

    // The softmax and the second product of a tile whose scores are in s and whose V rows are in LDS.
    v4f s[NT];
    auto finish = [&](auto masked, int t, unsigned long long have) {
        constexpr bool kMasked = decltype(masked)::value;
        unsigned long long see = 0;
        if constexpr (kMasked) {  // the tile's rows that this query row attends to
            const int rel = L - t;
            see = low_bits(tree ? rel : rel + token + 1);
            if (tree) {
                const unsigned long long nodes = sees;
                see |= rel >= 64 || rel <= -32 ? 0 : rel >= 0 ? nodes << rel : nodes >> -rel;
            }
            see = (see & have) >> (4 * g);
#pragma unroll
            for (int tt = 0; tt < NT; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[tt][i] = (see >> (16 * tt + i)) & 1 ? s[tt][i] : kNegInf;
        }
        float mx = kNegInf;
#pragma unroll
        for (int tt = 0; tt < NT; ++tt)
#pragma unroll
            for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[tt][i]);
        mx = lane_max(mx) * a.scale_log2;
        if (__builtin_amdgcn_ballot_w64(mx > m + kSlack)) {  // (a first score is more than -inf + kSlack)
            const float to = fmaxf(m, mx), base = to == kNegInf ? 0.f : to;
            const float shrink = __builtin_amdgcn_exp2f(m - base);
            m = to;
            l *= shrink;
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) o[dt] *= shrink;
        }
        float base = weight_base<T>(m), scale = a.scale_log2;
        if (__builtin_amdgcn_ballot_w64(fabsf(base) > kFar)) {
            base = from_maximum<T>(s, m, scale);
            scale = 1.f;
        }
        float sum = 0.f;
#pragma unroll
        for (int tt = 0; tt < NT; ++tt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[tt][i] = __builtin_amdgcn_exp2f(fmaf(s[tt][i], scale, -base));
                sum += s[tt][i];
            }
        l += sum;
        bool strange = false;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            v4i pf;
            if constexpr (kPairs)
                pf = Type<T>::pack(s[2 * u], s[2 * u + 1]);
            else if constexpr (sizeof(T) == 2)
                pf = Type<T>::pack(s[u], v4f{0.f, 0.f, 0.f, 0.f});
            else
                pf = __builtin_bit_cast(v4i, s[u]);
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) {
                v4i vf = v_operand<T, D, kPairs, kFour>(s_v, u, dt, lane);
                if constexpr (kMasked) strange |= drop_nonfinite<T>(vf);
                if constexpr (kPairs || sizeof(T) == 4)
                    o[dt] = Type<T>::mma(vf, pf, o[dt]);
                else
                    o[dt] = Type<T>::mma16(v2i{vf[0], vf[1]}, v2i{pf[0], pf[1]}, o[dt]);
            }
        }
        if constexpr (kMasked)  // infinities and NaN go to the rows that attend to them, as in the row kernel
            if (__builtin_amdgcn_ballot_w64(strange)) {
#pragma unroll 1
                for (int side = 0; side < 2; ++side) {
                    const float inf = side ? kNegInf : -kNegInf;
#pragma unroll
                    for (int u = 0; u < NU; ++u) {
                        v4f one[2];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            one[j >> 2][j & 3] = (kPairs || j < 4) && (see >> ((kPairs ? 32 * u + 16 * (j >> 2) : 16 * u) + (j & 3))) & 1 ? 1.f : 0.f;
                        v4i reads;
                        if constexpr (sizeof(T) == 2)
                            reads = Type<T>::pack(one[0], one[1]);
                        else
                            reads = __builtin_bit_cast(v4i, one[0]);
#pragma unroll
                        for (int dt = 0; dt < ND; ++dt) {
                            const v4i vf = nonfinite_ones<T>(v_operand<T, D, kPairs, kFour>(s_v, u, dt, lane), side);
                            v4f cnt{0.f, 0.f, 0.f, 0.f};
                            if constexpr (kPairs || sizeof(T) == 4)
                                cnt = Type<T>::mma(vf, reads, cnt);
                            else
                                cnt = Type<T>::mma16(v2i{vf[0], vf[1]}, v2i{reads[0], reads[1]}, cnt);
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[dt][i] += cnt[i] > 0.f ? inf : 0.f;
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                }
            }
    };

    const int all_see = tree ? L : L + 1;  // rows in front of this: seen by every query row
    int t = t0 + wave * TOK;
    if (t < t1) {
        unsigned long long have = load(t, fetch(t));
        int pid = fetch(t + kStep);
        for (; t < t1; t += kStep) {
#pragma unroll
            for (int tt = 0; tt < NT; ++tt) {
                s[tt] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < NS; ++ks) {
                    v4i kf;
                    if constexpr (kFour)
                        kf = four_values<T>(kc[tt][VPS * ks / 8], ks4[tt][VPS * ks / 32], VPS * ks % 8 / 4);
                    else
                        kf = kr[tt * NS + ks];
                    s[tt] = Type<T>::mma(kf, qf[ks], s[tt]);
                }
            }
            const unsigned long long here = have;
            if (here != kFull) {
#pragma unroll
                for (int p = 0; p < (kFour ? 0 : NP); ++p) {
                    const bool ok = (here >> (RPP * p + lane / TPR)) & 1;
                    vr[p] = v4i{ok ? vr[p][0] : 0, ok ? vr[p][1] : 0, ok ? vr[p][2] : 0, ok ? vr[p][3] : 0};
                }
                if (lane == 0 && a.l.status && here != (kFull & low_bits(t1 - t))) atomicOr(a.l.status, GDN_STATUS_PAGE);
            }
            if constexpr (kFour) {
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const int r = RPP * p + lane / (D / 32);
                    if (here != kFull) vc[p].drop((here >> r) & 1);
                    vc[p].template store<T, D>(s_v, r, lane % (D / 32));
                }
            } else {
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    *reinterpret_cast<v4i *>(s_v + lds_at<RB>(RPP * p + lane / TPR, lane % TPR)) = vr[p];
            }
            if (t + kStep < t1) {
                have = load(t + kStep, pid);
                pid = fetch(t + 2 * kStep);
            }
            if (t + TOK > all_see || here != kFull)
                finish(std::true_type{}, t, here);
            else
                finish(std::false_type{}, t, here);
        }
    }

    // ---- the four waves' outputs joined: 4-column groups of a row at place (group ^ row)
    l = lane_sum(l);
    if (g == 0) {
        s_m[wave][n] = m;
        s_l[wave][n] = l;
    }
#pragma unroll
    for (int dt = 0; dt < ND; ++dt)
        *reinterpret_cast<v4f *>(s_v + (n * (D / 4) + ((4 * dt + g) ^ n)) * 16) = o[dt];
    __syncthreads();
    const size_t all_rows = (size_t)d.C * d.N * d.Hq;
    for (int k = tid; k < rows * (D / 4); k += 64 * kFewWaves) {
        const int row = k / (D / 4), col = k % (D / 4);
        float mx = kNegInf;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) mx = fmaxf(mx, s_m[w][row]);
        v4f acc{0.f, 0.f, 0.f, 0.f};
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) {
            const float mw = s_m[w][row], lw = s_l[w][row];
            const float wgt = mw == kNegInf ? 0.f : __builtin_amdgcn_exp2f(mw - mx);
            const v4f v = *reinterpret_cast<const v4f *>(s_buf[w] + (row * (D / 4) + (col ^ row)) * 16);
            if (wgt != 0.f) acc += v * wgt;
            sum += lw == 0.f ? 0.f : lw * wgt;
        }
        if (plan.splits > 1) {
            const size_t at = (size_t)split * all_rows + ((size_t)c * d.Hkv + h) * d.N * d.G + row;
            *reinterpret_cast<v4f *>(a.workspace + at * D + 4 * col) = acc;
            if (col == 0) {
                float *ml = join_pairs(a, plan) + at * 2;
                ml[0] = mx;
                ml[1] = sum;
            }
            continue;
        }
        const int tk = row / d.G, hd = h * d.G + row - tk * d.G;
        const int64_t nd = (int64_t)c * d.N + tk;
        v4f v = sum == 0.f ? v4f{0.f, 0.f, 0.f, 0.f} : acc / sum;
        if (a.gate.p && sum != 0.f) {
            const v4f z = load4(static_cast<const T *>(a.gate.p) + nd * a.gate.token + hd * a.gate.head + 4 * col);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = gated(v[i], z[i], a.gate_mode);
        }
        store4(static_cast<T *>(a.out) + (nd * d.Hq + hd) * D + 4 * col, v);
    }
}

// ---- the launches of one call; the join of its parts, whatever the cache holds, is launched by paged_attention.hip
template <typename T, int D, int BM, bool kFour>
void launch_rows(const AttnArgs &a, const AttnPlan &p, unsigned units, hipStream_t stream) {
    const dim3 grid(p.tiles > 1 ? (units + 7) / 8 * 8 : units);
    hipLaunchKernelGGL((attn_rows_kernel<T, D, BM, kFour>), grid, dim3(64 * group_waves(BM)), 0, stream, a, p);
}

template <typename T, int D, bool kFour>
hipError_t launch(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    constexpr int RB = D * sizeof(T);
    const unsigned units = (unsigned)a.d.C * a.d.Hkv * p.tiles * p.splits;
    if constexpr (RB < 1024 || kFour)
        if (p.rows_per_group == kFewRows)
            hipLaunchKernelGGL((attn_few_kernel<T, D, kFour>), dim3(units), dim3(64 * kFewWaves), 0, stream, a, p);
    if constexpr (RB < 512 || sizeof(T) == 4)
        if (p.rows_per_group == 64) launch_rows<T, D, 64, kFour>(a, p, units, stream);
    if constexpr (RB < 512 && sizeof(T) == 2)
        if (p.rows_per_group == 256) launch_rows<T, D, 256, kFour>(a, p, units, stream);
    if constexpr (D == 256 && sizeof(T) == 2) {
        if (p.rows_per_group == kPairRows)
            hipLaunchKernelGGL((attn_pair_kernel<T, kFour>), dim3(p.tiles > 1 ? (units + 7) / 8 * 8 : units), dim3(kPairThreads), 0,
                               stream, a, p);
    } else if constexpr (RB < 1024) {
        if (p.rows_per_group == 128) launch_rows<T, D, 128, kFour>(a, p, units, stream);
    }
    return p.splits > 1 ? launch_attention_join(a, p, stream) : hipGetLastError();
}

template <typename T, bool kFour>
hipError_t launch_t(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    if (a.d.D == 64) return launch<T, 64, kFour>(a, p, stream);
    if (a.d.D == 128) return launch<T, 128, kFour>(a, p, stream);
    return launch<T, 256, kFour>(a, p, stream);
}

template <bool kFour>
hipError_t launch_attention(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    if (a.d.dtype == GDN_DTYPE_BF16) return launch_t<__bf16, kFour>(a, p, stream);
    if (a.d.dtype == GDN_DTYPE_F16) return launch_t<_Float16, kFour>(a, p, stream);
    return launch_t<float, kFour>(a, p, stream);
}

}  // namespace
}  // namespace gdn

// Acceptance of the drafted tokens for gfx950: every lane's walk down its draft tree against the
// target's probabilities with given random numbers (or greedily), and the token that follows.
//
// Mathematics.  A token x drawn from q and accepted with probability min(1, p(x) / q(x)), a
// refusal followed by a draw from max(p - q, 0), leaves a token distributed as p; u q(x) < p(x)
// is that test without a division.  A candidate that was not drawn has q = 1, and refusing it
// leaves p without it: the next sibling is tested against p(x') / (1 - p(x)).  The tests are
// evaluated in 64 bits, where u q is exact; the running sum of the final draw too, so that its
// result does not hang on the order in which 10^5 terms are added.
//
// A lane reads its drafted tokens' probabilities (one value per node) and one row of V values
// (two with a draft distribution): bound by the chain of dependent reads (parents, tokens, their
// probabilities, the last row) and by launch.  The row is cut into chunks over workgroups; each
// repeats the walk (one wave, a node per lane) instead of waiting for another to have done it.
// A second launch finds the chunk and the token in it.  Greedy reads every row of the lane: which
// of them the walk meets is known only with their largest values.
#include "round_device.h"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPer = kAcceptChunk / kThreads;  // 16 values a thread

// Four values of a row at the alignment of one
template <typename T>
__device__ inline void load4(const T *p, float (&x)[4]) {
    typedef T t4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    const t4 v = *reinterpret_cast<const t4 *>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (float)v[e];
}

__device__ inline int lane_of(int x, int j) { return __builtin_amdgcn_readlane(x, j); }
__device__ inline float lane_of(float x, int j) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), j)); }

// One lane's nodes, one per lane of a wave.
struct Nodes {
    int n, par, tok, bits;
    unsigned anc;
    bool padding;
};
__device__ inline Nodes load_nodes(const AcceptArgs &a, int c) {
    Nodes r{};
    const int lane = threadIdx.x & 63;
    r.padding = a.slot_ids && a.slot_ids[c] == -1;
    r.n = a.lane_nodes ? a.lane_nodes[c] : a.N;
    const bool count_ok = r.n >= 0 && r.n <= a.N;
    const bool has = count_ok && lane < r.n;
    const int64_t at = (int64_t)c * a.N + lane;
    r.par = !has ? -2 : a.parents ? a.parents[at] : lane - 1;
    r.tok = has ? a.tokens[at] : 0;
    if (!count_ok) r.bits |= GDN_STATUS_NODES;
    if (__builtin_amdgcn_ballot_w64(has && (unsigned)r.tok >= (unsigned)a.V)) r.bits |= GDN_STATUS_TOKEN;
    bool bad = false;
    r.anc = !has ? 0u : (2u << lane) - 1u;  // a chain: every node in front
    if (a.parents) r.anc = tree_ancestors(a.parents + (int64_t)c * a.N, count_ok ? r.n : 0, bad);
    if (bad) r.bits |= GDN_STATUS_PARENT;
    return r;
}

// The set of accepted nodes (a root path) from which nodes would be entered if reached.
__device__ inline unsigned taken_nodes(const Nodes &nd, bool ok) {
    const int lane = threadIdx.x & 63;
    bool first = ok;
    for (int j = 0; j < nd.n - 1; ++j)  // an earlier sibling that is accepted comes first
        if (lane_of((int)ok, j) && lane_of(nd.par, j) == nd.par && j < lane) first = false;
    const unsigned entered = (unsigned)__builtin_amdgcn_ballot_w64(first && lane < nd.n);
    return (unsigned)__builtin_amdgcn_ballot_w64(lane < nd.n && (nd.anc & ~entered) == 0);
}

// Whether an earlier sibling exists, and whether one has the same token
__device__ inline void earlier_siblings(const Nodes &nd, bool &any, bool &same) {
    const int lane = threadIdx.x & 63;
    any = same = false;
    for (int j = 0; j < nd.n - 1; ++j)
        if (lane_of(nd.par, j) == nd.par && j < lane) {
            any = true;
            same |= lane_of(nd.tok, j) == nd.tok;
        }
}

// What the second launch needs of a lane's walk.
struct alignas(16) Stop {
    int valid, node;   // node -1: the prefix
    unsigned refused;  // its children
    int pad;
};
__device__ inline Stop *stops(const AcceptArgs &a) {
    return reinterpret_cast<Stop *>(static_cast<double *>(a.workspace) + (size_t)a.C * accept_chunks(a.V) * 2);
}

// Row of p behind `node`, and of q of its refused child (null: none, or candidates)
template <typename T>
struct Rows {
    const T *p, *q;
};
template <typename T>
__device__ inline Rows<T> rows_of(const AcceptArgs &a, int c, const Stop &st) {
    const T *target = static_cast<const T *>(a.target), *root = static_cast<const T *>(a.root);
    Rows<T> r;
    r.p = st.node >= 0 ? target + ((int64_t)c * a.N + st.node) * a.V : root + (int64_t)c * a.V;
    r.q = a.draft && st.refused ? static_cast<const T *>(a.draft) + ((int64_t)c * a.N + st.node + 1) * a.V : nullptr;
    return r;
}

// Marks the chunk's refused candidates in a bitmap of the chunk (every thread calls it).
__device__ inline void mark_refused(const AcceptArgs &a, int c, const Stop &st, int x0, unsigned *bitmap) {
    const int tid = threadIdx.x;
    if (tid < kAcceptChunk / 32) bitmap[tid] = 0u;
    __syncthreads();
    if (!a.draft && tid < 32 && ((st.refused >> tid) & 1)) {
        const int x = a.tokens[(int64_t)c * a.N + tid] - x0;
        if (x >= 0 && x < kAcceptChunk) atomicOr(&bitmap[x >> 5], 1u << (x & 31));
    }
    __syncthreads();
}

// w and p of values x0 + off .. + 3 (zeros behind the row's end)
template <typename T>
__device__ inline void weights4(const Rows<T> &r, int V, int x0, int off, const unsigned *bitmap, double (&w)[4], double (&p)[4]) {
    float pv[4] = {0.f, 0.f, 0.f, 0.f}, qv[4] = {0.f, 0.f, 0.f, 0.f};
    const int x = x0 + off;
    if (x + 4 <= V) {
        load4(r.p + x, pv);
        if (r.q) load4(r.q + x, qv);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (x + e < V) {
                pv[e] = (float)r.p[x + e];
                if (r.q) qv[e] = (float)r.q[x + e];
            }
    }
    const unsigned gone = bitmap[off >> 5] >> (off & 31);  // (off is a multiple of 4)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        p[e] = pv[e] > 0.f ? (double)pv[e] : 0.0;
        const double q = qv[e] > 0.f ? (double)qv[e] : 0.0;
        w[e] = (gone >> e) & 1 ? 0.0 : p[e] > q ? p[e] - q : 0.0;
    }
}

__device__ inline double wave_sum(double x) {
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) x += __shfl_xor(x, k);
    return x;
}

// First launch of the sampled form: the walk, and this chunk's sums of w and p.
template <typename T>
__global__ __launch_bounds__(kThreads) void accept_sums_kernel(AcceptArgs a) {
    __shared__ Stop s_stop;
    __shared__ unsigned s_bitmap[kAcceptChunk / 32];
    __shared__ double s_sum[kWaves][2];
    const int tid = threadIdx.x, lane = tid & 63, c = blockIdx.y, chunk = blockIdx.x;
    if (tid < 64) {
        const Nodes nd = load_nodes(a, c);
        Stop st{0, -1, 0u, 0};
        if (!nd.padding && !nd.bits) {
            const int64_t at = (int64_t)c * a.N + lane;
            const bool has = lane < nd.n;
            float p = 0.f, q = 1.f, u = 0.f;
            if (has) {
                const T *row = nd.par >= 0 ? static_cast<const T *>(a.target) + ((int64_t)c * a.N + nd.par) * a.V
                               : a.root    ? static_cast<const T *>(a.root) + (int64_t)c * a.V
                                           : nullptr;
                if (row) p = (float)row[nd.tok];
                if (a.draft) q = (float)static_cast<const T *>(a.draft)[at * a.V + nd.tok];
                u = a.u_accept[at];
            }
            bool any, same;
            earlier_siblings(nd, any, same);
            if (same || !(p > 0.f)) p = 0.f;
            if (!(q > 0.f)) q = 0.f;
            double refused = 0.0;
            for (int j = 0; j < nd.n - 1; ++j)
                if (lane_of(nd.par, j) == nd.par && j < lane) refused += (double)lane_of(p, j);
            bool ok = (double)u * (double)q * (1.0 - refused) < (double)p;
            if (nd.par == -1 && !a.root) ok = !any;  // the token already drawn
            const unsigned taken = taken_nodes(nd, ok && has);
            st.node = taken ? 31 - __builtin_clz(taken) : -1;
            st.refused = (unsigned)__builtin_amdgcn_ballot_w64(has && nd.par == st.node);
            st.valid = st.node >= 0 || a.root;
            if (chunk == 0 && lane == 0) {
                a.accept_node[c] = st.node;
                a.n_accept[c] = __popc(taken);
                if (!st.valid) a.next_token[c] = -1;  // no row to draw from
            }
        }
        if (chunk == 0 && lane == 0) {
            if (!nd.padding && nd.bits && a.status) atomicOr(a.status, nd.bits);
            stops(a)[c] = st;
        }
        if (lane == 0) s_stop = st;
    }
    __syncthreads();
    const Stop st = s_stop;
    if (!st.valid) return;
    const Rows<T> r = rows_of<T>(a, c, st);
    const int x0 = chunk * kAcceptChunk;
    mark_refused(a, c, st, x0, s_bitmap);
    double sw = 0.0, sp = 0.0;
#pragma unroll
    for (int k = 0; k < kPer / 4; ++k) {
        double w[4], p[4];
        weights4(r, a.V, x0, 4 * (k * kThreads + tid), s_bitmap, w, p);
#pragma unroll
        for (int e = 0; e < 4; ++e) sw += w[e], sp += p[e];
    }
    sw = wave_sum(sw);
    sp = wave_sum(sp);
    if (lane == 0) s_sum[tid >> 6][0] = sw, s_sum[tid >> 6][1] = sp;
    __syncthreads();
    if (tid < 2) {
        double s = 0.0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += s_sum[w][tid];
        static_cast<double *>(a.workspace)[((size_t)c * gridDim.x + chunk) * 2 + tid] = s;
    }
}

// Inclusive running sum over a wave, in lane order
__device__ inline double wave_scan(double x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const double y = __shfl_up(x, k);
        if (lane >= k) x += y;
    }
    return x;
}

// Second launch: the chunk in which the running sum passes u times the whole, and the token in it.
template <typename T>
__global__ __launch_bounds__(kThreads) void accept_draw_kernel(AcceptArgs a, int chunks) {
    __shared__ unsigned s_bitmap[kAcceptChunk / 32];
    __shared__ double s_wave[kWaves], s_before, s_limit;
    __shared__ int s_chunk, s_fall, s_found, s_last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = blockIdx.x;
    const Stop st = stops(a)[c];
    if (!st.valid) return;
    const double *sums = static_cast<const double *>(a.workspace) + (size_t)c * chunks * 2;
    if (tid == 0) s_found = s_last = -1;
    if (wave == 0) {
        // side 0: the sums of w; where they are all zero, side 1: those of p
        double total = 0.0;
        int side = 0;
        for (; side < 2; ++side) {
            total = 0.0;
            for (int k = 0; k < chunks; k += 64) total += k + lane < chunks ? sums[2 * (k + lane) + side] : 0.0;
            total = wave_sum(total);
            if (total > 0.0) break;
        }
        int found = -1, last = -1;
        double before = 0.0, run = 0.0, before_last = 0.0;
        const double limit = (double)a.u_next[c] * total;
        if (side < 2)
            for (int k = 0; k < chunks && found < 0; k += 64) {
                const double mine = k + lane < chunks ? sums[2 * (k + lane) + side] : 0.0;
                const double upto = run + wave_scan(mine);
                const unsigned long long over = __builtin_amdgcn_ballot_w64(mine > 0.0 && upto > limit);
                const unsigned long long some = __builtin_amdgcn_ballot_w64(mine > 0.0);
                const double front = upto - mine;  // (before the chunk; the lane below's `upto` but for rounding)
                if (over) {
                    const int l = __builtin_ctzll(over);
                    found = k + l;
                    before = l ? __shfl(upto, l - 1) : run;
                } else if (some) {
                    const int l = 63 - __builtin_clzll(some);
                    last = k + l;
                    before_last = __shfl(front, l);
                }
                run = __shfl(upto, 63);
            }
        if (found < 0) found = last, before = before_last;
        if (lane == 0) s_chunk = found, s_before = before, s_limit = limit, s_fall = side;
    }
    __syncthreads();
    const int chunk = s_chunk;
    if (chunk < 0) {  // a row without any weight
        if (tid == 0) a.next_token[c] = -1;
        return;
    }
    const Rows<T> r = rows_of<T>(a, c, st);
    const int x0 = chunk * kAcceptChunk;
    mark_refused(a, c, st, x0, s_bitmap);
    double w[kPer], own = 0.0;
#pragma unroll
    for (int k = 0; k < kPer / 4; ++k) {
        double w4[4], p4[4];
        weights4(r, a.V, x0, kPer * tid + 4 * k, s_bitmap, w4, p4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[4 * k + e] = s_fall ? p4[e] : w4[e];
            own += w[4 * k + e];
        }
    }
    const double upto = wave_scan(own);
    if (lane == 63) s_wave[wave] = upto;
    __syncthreads();
    double run = s_before;
    for (int v = 0; v < wave; ++v) run += s_wave[v];
    run += upto - own;
    int at = -1, last = -1;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        run += w[e];
        if (w[e] > 0.0) {
            last = e;
            if (at < 0 && run > s_limit) at = e;
        }
    }
    // the lowest token over the limit; behind rounding, the last one with a weight
    if (at >= 0) atomicMin(reinterpret_cast<unsigned *>(&s_found), (unsigned)(kPer * tid + at));
    if (last >= 0) atomicMax(&s_last, kPer * tid + last);
    __syncthreads();
    if (tid == 0) a.next_token[c] = x0 + (s_found >= 0 ? s_found : s_last);
}

// A (value, index) pair of which the larger value, then the lower index, wins
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

// First launch of the greedy form: the largest value of one chunk of one row.
template <typename T>
__global__ __launch_bounds__(kThreads) void accept_best_kernel(AcceptArgs a) {
    __shared__ Best s_best[kWaves];
    const int tid = threadIdx.x, chunk = blockIdx.x, row = blockIdx.y, c = row / (a.N + 1), i = row - c * (a.N + 1);
    const int n = a.lane_nodes ? a.lane_nodes[c] : a.N;
    if ((a.slot_ids && a.slot_ids[c] == -1) || n < 0 || n > a.N || (i < a.N ? i >= n : !a.root)) return;
    const T *p = i < a.N ? static_cast<const T *>(a.target) + ((int64_t)c * a.N + i) * a.V
                         : static_cast<const T *>(a.root) + (int64_t)c * a.V;
    Best b{-__builtin_inff(), 0x7fffffff};
#pragma unroll
    for (int k = 0; k < kPer / 4; ++k) {
        const int x = chunk * kAcceptChunk + 4 * (k * kThreads + tid);
        float v[4];
        if (x + 4 <= a.V) {
            load4(p + x, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = x + e < a.V ? (float)p[x + e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (x + e < a.V) b = better(b, Best{v[e] == v[e] ? v[e] : -__builtin_inff(), x + e});
    }
    b = wave_best(b);
    if ((tid & 63) == 0) s_best[tid >> 6] = b;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kWaves; ++w) b = better(b, s_best[w]);
        static_cast<Best *>(a.workspace)[(size_t)row * gridDim.x + chunk] = b;
    }
}

// Second launch of the greedy form: the rows' largest values, and the walk.
__global__ __launch_bounds__(kThreads) void accept_walk_kernel(AcceptArgs a, int chunks) {
    __shared__ int s_best[GDN_MAX_NODES + 1];
    const int tid = threadIdx.x, lane = tid & 63, c = blockIdx.x;
    const Nodes nd = load_nodes(a, c);  // (every wave: the branch below is uniform)
    if (nd.padding) return;
    if (nd.bits) {
        if (tid == 0 && a.status) atomicOr(a.status, nd.bits);
        return;
    }
    const Best *all = static_cast<const Best *>(a.workspace) + (size_t)c * (a.N + 1) * chunks;
    for (int i = tid >> 6; i <= a.N; i += kWaves) {
        if (i < a.N ? i >= nd.n : !a.root) continue;
        Best b{-__builtin_inff(), 0x7fffffff};
        for (int k = lane; k < chunks; k += 64) b = better(b, all[(size_t)i * chunks + k]);
        b = wave_best(b);
        if (lane == 0) s_best[i] = b.x;
    }
    __syncthreads();
    if (tid >= 64) return;
    bool any, same;
    earlier_siblings(nd, any, same);
    bool ok = false;
    if (lane < nd.n) {
        if (nd.par == -1 && !a.root)
            ok = !any;
        else
            ok = !same && s_best[nd.par >= 0 ? nd.par : a.N] == nd.tok;
    }
    const unsigned taken = taken_nodes(nd, ok);
    if (lane == 0) {
        const int node = taken ? 31 - __builtin_clz(taken) : -1;
        a.accept_node[c] = node;
        a.n_accept[c] = __popc(taken);
        a.next_token[c] = node >= 0 ? s_best[node] : a.root ? s_best[a.N] : -1;
    }
}

template <typename T>
hipError_t launch(const AcceptArgs &a, hipStream_t stream) {
    const int chunks = accept_chunks(a.V);
    if (a.u_accept) {
        hipLaunchKernelGGL((accept_sums_kernel<T>), dim3(chunks, a.C), dim3(kThreads), 0, stream, a);
        hipLaunchKernelGGL((accept_draw_kernel<T>), dim3(a.C), dim3(kThreads), 0, stream, a, chunks);
    } else {
        hipLaunchKernelGGL((accept_best_kernel<T>), dim3(chunks, a.C * (a.N + 1)), dim3(kThreads), 0, stream, a);
        hipLaunchKernelGGL(accept_walk_kernel, dim3(a.C), dim3(kThreads), 0, stream, a, chunks);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_draft_accept(const AcceptArgs &a, hipStream_t stream) {
    if (a.dtype == GDN_DTYPE_BF16) return launch<__bf16>(a, stream);
    if (a.dtype == GDN_DTYPE_F16) return launch<_Float16>(a, stream);
    return launch<float>(a, stream);
}

}  // namespace gdn

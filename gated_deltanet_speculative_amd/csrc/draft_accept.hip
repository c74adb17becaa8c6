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
// probabilities, the last row) and by launch.  The row is cut into chunks of 1024, one per wave;
// every workgroup of four repeats the walk, a node per lane, instead of waiting for another to have done it.  A second
// launch finds the chunk and the token in it.  Greedy reads every row of the lane: which
// of them the walk meets is known only with their largest values.
#include "round_device.h"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPer = kAcceptChunk / 64;  // 16 values of a chunk a lane
constexpr int kBestChunk = 4096;         // values of a workgroup of the greedy form

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

// The earlier siblings of this lane's node, as a bit set (a chain has none).
__device__ inline unsigned earlier_siblings(const AcceptArgs &a, const Nodes &nd) {
    unsigned sib = 0;
    if (a.parents)
        for (int j = 0; j < nd.n - 1; ++j) sib |= lane_of(nd.par, j) == nd.par ? 1u << j : 0u;
    return sib & ((1u << (threadIdx.x & 31)) - 1u);
}

// Calls f(j) for every set bit j of this lane's set, in ascending order: as many rounds as the largest set of the
// wave has bits; f runs in every lane (lane shuffles), `on` where the bit is this lane's.
template <typename F>
__device__ inline void each_bit(unsigned set, F f) {
    while (__builtin_amdgcn_ballot_w64(set != 0)) {
        const bool on = set != 0;
        const int j = on ? __builtin_ctz(set) : 0;
        f(j, on);
        set &= set - 1u;
    }
}

// The set of accepted nodes: a root path of nodes that are the first accepted one of their siblings.
__device__ inline unsigned taken_nodes(const Nodes &nd, unsigned sib, bool ok) {
    const int lane = threadIdx.x & 63;
    const unsigned oks = (unsigned)__builtin_amdgcn_ballot_w64(ok && lane < nd.n);
    const unsigned entered = (unsigned)__builtin_amdgcn_ballot_w64(ok && lane < nd.n && (sib & oks) == 0);
    return (unsigned)__builtin_amdgcn_ballot_w64(lane < nd.n && (nd.anc & ~entered) == 0);
}

// Whether an earlier sibling has the same token.
__device__ inline bool token_again(const Nodes &nd, unsigned sib) {
    bool same = false;
    each_bit(sib, [&](int j, bool on) {
        const int tok = __shfl(nd.tok, j);
        same |= on && tok == nd.tok;
    });
    return same;
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

// Marks the refused candidates among values x0 .. x0 + kAcceptChunk - 1 in a bit set of this wave's; tok is lane i's node's
// token.  (The wave's own LDS operations complete in order.)
struct Refused {
    unsigned word[kAcceptChunk / 32 + 1];
};
__device__ inline void mark_refused(Refused &r, const AcceptArgs &a, const Stop &st, int tok, int x0) {
    const int lane = threadIdx.x & 63;
    static_assert(kAcceptChunk / 32 + 1 <= 64, "a word a lane");
    if (lane <= kAcceptChunk / 32) r.word[lane] = 0u;
    const int x = tok - x0;
    if (!a.draft && lane < GDN_MAX_NODES && ((st.refused >> lane) & 1) && x >= 0 && x < kAcceptChunk)
        atomicOr(&r.word[x >> 5], 1u << (x & 31));
}

// Four values of a row and their weights, from index `at` on; what lies in front of `from` or behind the row is 0.
struct Four {
    int at;
    double w[4], p[4];
};
template <typename T>
struct Raw {
    int at, from;
    float p[4], q[4];
};
// The loads alone.  The last values of a row are read with their predecessors: every load lies inside the row.
template <typename T>
__device__ inline Raw<T> raw4(const Rows<T> &r, int V, int x) {
    Raw<T> v;
    v.from = x;
    v.at = min(x, max(V - 4, 0));
#pragma unroll
    for (int e = 0; e < 4; ++e) v.p[e] = v.q[e] = 0.f;
    if (V >= 4) {
        load4(r.p + v.at, v.p);
        if (r.q) load4(r.q + v.at, v.q);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < V) {
                v.p[e] = (float)r.p[e];
                if (r.q) v.q[e] = (float)r.q[e];
            }
    }
    return v;
}
template <typename T>
__device__ inline Four weights4(const Raw<T> &v, const Refused &r, int x0) {
    Four f;
    f.at = v.at;
    const int o = max(v.at - x0, 0);  // (in front of the chunk only where every value is)
    const unsigned long long words = (unsigned long long)r.word[min((o >> 5) + 1, kAcceptChunk / 32)] << 32 | r.word[min(o >> 5, kAcceptChunk / 32)];
    const unsigned gone = (unsigned)(words >> (o & 31));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int x = v.at + e;
        const bool has = x >= v.from;
        f.p[e] = has && v.p[e] > 0.f ? (double)v.p[e] : 0.0;
        const double q = v.q[e] > 0.f ? (double)v.q[e] : 0.0;
        const bool refused = x >= x0 && ((gone >> (x - x0 - o)) & 1);
        f.w[e] = refused || !(f.p[e] > q) ? 0.0 : f.p[e] - q;
    }
    return f;
}

__device__ inline double lane_of(double x, int j) {
    const long long b = __double_as_longlong(x);
    return __longlong_as_double((long long)((unsigned long long)(unsigned)lane_of((int)(b >> 32), j) << 32 | (unsigned)lane_of((int)b, j)));
}
// Inclusive running sum over a wave: within the rows of 16 lanes by row shifts, then the rows in front.
__device__ inline double wave_scan(double x) {
    x = group_sum_last<16>(x);
    const double a = lane_of(x, 15), b = lane_of(x, 31), c = lane_of(x, 47);
    const int row = (threadIdx.x & 63) >> 4;
    return x + (row == 0 ? 0.0 : row == 1 ? a : row == 2 ? a + b : a + b + c);
}

// First launch of the sampled form: the walk, and every wave's sums of w and p over one chunk of the row behind the
// last accepted node.
template <typename T>
__global__ __launch_bounds__(kThreads) void accept_sums_kernel(AcceptArgs a, int chunks) {
    __shared__ Refused s_refused[kWaves];
    __shared__ Stop s_stop;
    __shared__ int s_tok[GDN_MAX_NODES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = blockIdx.y, chunk = blockIdx.x * kWaves + wave;
    if (wave == 0) {  // (one wave of four: the walks' reads of a few values meet in the same few lines of memory)
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
            const unsigned sib = earlier_siblings(a, nd);
            if (token_again(nd, sib) || !(p > 0.f)) p = 0.f;
            if (!(q > 0.f)) q = 0.f;
            double refused = 0.0;
            each_bit(sib, [&](int j, bool on) {
                const float pj = __shfl(p, j);
                refused += on ? (double)pj : 0.0;
            });
            bool ok = (double)u * (double)q * (1.0 - refused) < (double)p;
            if (nd.par == -1 && !a.root) ok = sib == 0;  // the token already drawn
            const unsigned taken = taken_nodes(nd, sib, ok && has);
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
        if (lane < GDN_MAX_NODES) s_tok[lane] = nd.tok;
        if (lane == 0) s_stop = st;
    }
    __syncthreads();
    const Stop st = s_stop;
    if (!st.valid || chunk >= chunks) return;
    const Rows<T> r = rows_of<T>(a, c, st);
    const int x0 = chunk * kAcceptChunk;
    Raw<T> raw[kPer / 4];
#pragma unroll
    for (int k = 0; k < kPer / 4; ++k) raw[k] = raw4(r, a.V, x0 + 4 * (64 * k + lane));
    mark_refused(s_refused[wave], a, st, s_tok[lane & (GDN_MAX_NODES - 1)], x0);
    double sw = 0.0, sp = 0.0;
#pragma unroll
    for (int k = 0; k < kPer / 4; ++k) {
        const Four f = weights4(raw[k], s_refused[wave], x0);
#pragma unroll
        for (int e = 0; e < 4; ++e) sw += f.w[e], sp += f.p[e];
    }
    sw = wave_scan(sw);
    sp = wave_scan(sp);
    if (lane == 63) {
        double *out = static_cast<double *>(a.workspace) + ((size_t)c * chunks + chunk) * 2;
        out[0] = sw;
        out[1] = sp;
    }
}

// Second launch: the chunk in which the running sum passes u times the whole, and the token in it; 256 chunks at
// a time, four values of the chunk a thread.
template <typename T>
__global__ __launch_bounds__(kThreads) void accept_draw_kernel(AcceptArgs a, int chunks) {
    __shared__ Refused s_refused[kWaves];
    __shared__ double s_wave[2][kWaves], s_before;
    __shared__ int s_pick[2][kWaves];
    static_assert(kAcceptChunk == 4 * kThreads, "four values a thread");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = blockIdx.x;
    const double *sums = static_cast<const double *>(a.workspace) + (size_t)c * chunks * 2;
    const Stop st = stops(a)[c];
    const float u = a.u_next[c];
    const int tok = a.tokens[(int64_t)c * a.N + min(lane, a.N - 1)];
    const double first[2] = {sums[2 * min(tid, chunks - 1)], sums[2 * min(tid, chunks - 1) + 1]};
    if (!st.valid) return;
    auto sum_of = [&](int k0, int side) {
        const int k = k0 + tid;
        const double s = k0 == 0 ? first[side] : sums[2 * min(k, chunks - 1) + side];
        return k < chunks ? s : 0.0;
    };
    // the whole: of w, or where that is zero of p
    double sw = 0.0, sp = 0.0;
    for (int k0 = 0; k0 < chunks; k0 += kThreads) sw += sum_of(k0, 0), sp += sum_of(k0, 1);
    sw = wave_scan(sw);
    sp = wave_scan(sp);
    if (lane == 63) s_wave[0][wave] = sw, s_wave[1][wave] = sp;
    __syncthreads();
    sw = s_wave[0][0] + s_wave[0][1] + s_wave[0][2] + s_wave[0][3];
    sp = s_wave[1][0] + s_wave[1][1] + s_wave[1][2] + s_wave[1][3];
    __syncthreads();
    const int side = sw > 0.0 ? 0 : 1;
    const double total = side ? sp : sw, limit = (double)u * total;
    if (!(total > 0.0)) {  // a row without any weight
        if (tid == 0) a.next_token[c] = -1;
        return;
    }
    // A round: this thread's value joins the running sum (front: the sum before it).  Lanes, waves and rounds are in
    // index order, so the lowest index over the limit is the first lane of a ballot of the first wave that has one
    // (LDS minima and maxima of all threads on one word took 4 us here).
    auto add = [&](double mine, double base, double &front) {
        const double upto = wave_scan(mine);
        if (lane == 63) s_wave[0][wave] = upto;
        __syncthreads();
        for (int v = 0; v < wave; ++v) base += s_wave[0][v];
        front = base + (upto - mine);
        return base + upto;
    };
    // value of the first lane of the first wave with `hit`, else of the last lane of the last wave with `some`, else -1
    auto pick = [&](bool hit, int at, bool some, int last, bool &found) {
        const unsigned long long h = __builtin_amdgcn_ballot_w64(hit), s = __builtin_amdgcn_ballot_w64(some);
        const int ha = h ? lane_of(at, __builtin_ctzll(h)) : -1, sa = s ? lane_of(last, 63 - __builtin_clzll(s)) : -1;
        if (lane == 0) s_pick[0][wave] = ha, s_pick[1][wave] = sa;
        __syncthreads();
        int p = -1, q = -1;
        for (int w = kWaves - 1; w >= 0; --w) {
            if (s_pick[0][w] >= 0) p = s_pick[0][w];
            if (q < 0) q = s_pick[1][w];
        }
        found = p >= 0;
        return found ? p : q;
    };
    double base = 0.0, front = 0.0;
    int chunk = -1;
    bool found = false;
    for (int k0 = 0; k0 < chunks && !found; k0 += kThreads) {
        const double mine = sum_of(k0, side);
        const bool hit = add(mine, base, front) > limit && mine > 0.0;
        const int at = pick(hit, k0 + tid, mine > 0.0, k0 + tid, found);
        if (at >= 0) chunk = at;  // (none over the limit so far: the last one with a weight)
        if (found && chunk == k0 + tid) s_before = front;
        base += s_wave[0][0] + s_wave[0][1] + s_wave[0][2] + s_wave[0][3];
        __syncthreads();
    }
    base = found ? s_before : -__builtin_inf();
    const Rows<T> r = rows_of<T>(a, c, st);
    const int x0 = chunk * kAcceptChunk;
    const Raw<T> raw = raw4(r, a.V, x0 + 4 * tid);
    mark_refused(s_refused[wave], a, st, tok, x0);
    const Four f = weights4(raw, s_refused[wave], x0);
    double w[4], own = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) own += w[e] = side ? f.p[e] : f.w[e];
    add(own, base, front);
    int at = -1, last = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        front += w[e];
        if (w[e] > 0.0) {
            last = f.at + e;
            if (at < 0 && front > limit) at = f.at + e;
        }
    }
    const int token = pick(at >= 0, at, last >= 0, last, found);
    if (tid == 0) a.next_token[c] = token;
}

// A (value, index) pair of which the larger value, then the lower index, wins.  A NaN stands as -inf with the bit
// kNan in its index, behind every index of a row: below a value that is -inf.
constexpr int kNan = 1 << 30;
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
    for (int k = 0; k < kBestChunk / kThreads / 4; ++k) {
        const int x = chunk * kBestChunk + 4 * (k * kThreads + tid);
        float v[4];
        if (x + 4 <= a.V) {
            load4(p + x, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = x + e < a.V ? (float)p[x + e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (x + e < a.V) b = better(b, v[e] == v[e] ? Best{v[e], x + e} : Best{-__builtin_inff(), (x + e) | kNan});
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
        if (lane == 0) s_best[i] = b.x & (kNan - 1);
    }
    __syncthreads();
    if (tid >= 64) return;
    const unsigned sib = earlier_siblings(a, nd);
    const bool again = token_again(nd, sib);
    bool ok = false;
    if (lane < nd.n) {
        if (nd.par == -1 && !a.root)
            ok = sib == 0;
        else
            ok = !again && s_best[nd.par >= 0 ? nd.par : a.N] == nd.tok;
    }
    const unsigned taken = taken_nodes(nd, sib, ok);
    if (lane == 0) {
        const int node = taken ? 31 - __builtin_clz(taken) : -1;
        a.accept_node[c] = node;
        a.n_accept[c] = __popc(taken);
        a.next_token[c] = node >= 0 ? s_best[node] : a.root ? s_best[a.N] : -1;
    }
}

template <typename T>
hipError_t launch(const AcceptArgs &a, hipStream_t stream) {
    if (a.u_accept) {
        const int chunks = accept_chunks(a.V);
        hipLaunchKernelGGL((accept_sums_kernel<T>), dim3((chunks + kWaves - 1) / kWaves, a.C), dim3(kThreads), 0, stream, a, chunks);
        hipLaunchKernelGGL((accept_draw_kernel<T>), dim3(a.C), dim3(kThreads), 0, stream, a, chunks);
    } else {
        const int chunks = (a.V + kBestChunk - 1) / kBestChunk;
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

// Commit of the paged caches for gfx950: the accepted path's rows of every layer moved together
// behind the committed ones, and the new lengths, as an all-or-nothing transaction.
//
// With the path a_0 < ... < a_m, row L + j takes row L + a_j.  Parents precede children, so
// a_j >= j, and a row that is written (L + j) is read only by the steps i <= j (a_i >= i): in
// ascending order, loads of a step before the stores of the same and later ones, the move is safe
// in place.  A thread owns a 16-byte column of every row of one (lane, layer, K or V) and kv head:
// no other thread reads or writes it, so the order within the thread is enough.
//
// Bound by launch and by dependent reads (slot, length, page id, row): every workgroup checks all lanes itself, as
// in the replay commit, so one launch decides; its own rows are found and the first of them loaded ahead of the
// verdict, and the preflight's entries are requested kBatch at a time.  4 lanes of 16 nodes, 16 layers of 8 heads of 128
// in bfloat16: 6.5 us; 64 lanes of 32 nodes: 15.0 us.
#include "round_device.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

constexpr int kBatch = 8;  // preflight entries of a thread that are requested together
constexpr int kAhead = 8;  // moved rows of a thread in flight

__global__ __launch_bounds__(kThreads) void kv_commit_kernel(AttnDims d, int n_layers, CacheLayers cl, PagedLanes l,
                                                             const int32_t *__restrict__ accept_node,
                                                             int32_t *__restrict__ new_len, int row_chunks) {
    __shared__ unsigned s_bitmap[kBitmapSlots / 32];
    __shared__ int s_word, s_bits;
    __shared__ int s_slot[GDN_MAX_SEQS], s_len[GDN_MAX_SEQS], s_nodes[GDN_MAX_SEQS];  // slot -1: padding or in error
    __shared__ uint32_t s_src[GDN_MAX_NODES], s_dst[GDN_MAX_NODES];                   // cache rows of kv head 0
    const int tid = threadIdx.x, lane = tid & 63, c = blockIdx.y;
    const bool lengths = blockIdx.x == gridDim.x - 1;  // the last workgroup of lane 0 writes the lengths
    if (lengths && c != 0) return;

    // ---- this lane's path, rows and first loads, ahead of the verdict (a bad page is read as page 0)
    const int st_in = *l.status;
    const LaneSlotsT<kThreads> slots(l.slot_ids, d.C);
    const int e = accept_node[c];
    int n = 0, first = 0;
    unsigned path = 0;
    const Lane own = paged_lane(d, l, c);
    if (l.parents && !lengths && own.slot != -1 && !own.bits && e >= 0 && e < own.nodes) {
        bool bad;
        path = __shfl(tree_ancestors(l.parents + (int64_t)c * d.N, e + 1, bad), e);
        n = __popc(path);
        first = __builtin_ctz(~path);  // rows in front of the first gap stay (32: the whole path)
        if (path == ~0u) first = 32;
        if (tid < n) {
            unsigned p = path;  // node a_tid: the tid-th set bit
            for (int j = 0; j < tid; ++j) p &= p - 1u;
            const uint32_t src = own.len + __builtin_ctz(p), dst = own.len + tid;
            const int32_t *table = l.page_table + (int64_t)own.slot * d.max_pages;
            const int ps = table[d.page(src)], pd = table[d.page(dst)];
            s_src[tid] = (unsigned)ps < (unsigned)d.n_pages ? cache_row(d, ps, 0, src, d.page(src)) : 0u;
            s_dst[tid] = (unsigned)pd < (unsigned)d.n_pages ? cache_row(d, pd, 0, dst, d.page(dst)) : 0u;
        }
    }
    if (tid == 0) s_bits = 0;
    lds_barrier();
    // this thread's column: K or V of a layer, kv head, 16 bytes
    const int cols = d.Hkv * row_chunks, item = blockIdx.x * kThreads + tid, side = item / cols, col = item - side * cols;
    const bool mine = !lengths && side < 2 * n_layers;
    v4i *p = nullptr, v[kAhead];
    if (mine)
        p = static_cast<v4i *>(side < n_layers ? cl.k[side] : cl.v[side - n_layers]) +
            (size_t)(col / row_chunks) * d.page.d * row_chunks + col % row_chunks;
    auto load = [&](int j0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (j0 + j < n) v[j] = p[(size_t)s_src[j0 + j] * row_chunks];
    };
    if (mine) load(first);

    // ---- preflight over every lane
    int bits = slot_preflight<kThreads>(slots, l.slot_ids, d.C, d.P, s_bitmap, &s_word);  // (has barriers)
    for (int t = tid; t < d.C; t += kThreads) {
        const Lane ln = paged_lane(d, l, t);
        const int et = accept_node[t];
        bits |= ln.bits;
        if (ln.slot != -1 && (et < -1 || et >= min(max(ln.nodes, 0), d.N))) bits |= GDN_STATUS_ACCEPT;
        s_slot[t] = ln.bits ? -1 : ln.slot;
        s_len[t] = ln.len;
        s_nodes[t] = ln.nodes;
    }
    if (l.parents) {
        lds_barrier();
        // entry k is node k % 32 of lane k / 32
        const int i = tid & (GDN_MAX_NODES - 1), last = d.C - 1;
        for (int t0 = tid / GDN_MAX_NODES; t0 < d.C; t0 += kThreads / GDN_MAX_NODES * kBatch) {
            int par[kBatch], pid[kBatch];
            bool has[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int t = t0 + j * (kThreads / GDN_MAX_NODES), u = min(t, last);
                has[j] = (t <= last) & (i < d.N) & (s_slot[u] != -1) & (i < s_nodes[u]);
                par[j] = l.parents[(int64_t)u * d.N + min(i, d.N - 1)];
                pid[j] = l.page_table[has[j] ? (int64_t)s_slot[u] * d.max_pages + d.page((uint32_t)(s_len[u] + i)) : 0];
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (has[j] & ((par[j] < -1) | (par[j] >= i))) bits |= GDN_STATUS_PARENT;
                if (has[j] & ((unsigned)pid[j] >= (unsigned)d.n_pages)) bits |= GDN_STATUS_PAGE;
            }
        }
    }
    if (bits) atomicOr(&s_bits, bits);
    lds_barrier();
    bits = s_bits;
    const bool commit = st_in == 0 && bits == 0;
    if (bits && tid == 0 && blockIdx.x == 0) atomicOr(l.status, bits);

    if (lengths) {
        for (int s = tid; s < d.P; s += kThreads) new_len[s] = l.seq_len[s];
        if (!commit) return;
        __syncthreads();  // (the same addresses are written again below)
        for (int t0 = 0; t0 < d.C; t0 += kThreads / 64) {  // a wave per lane
            const int t = t0 + (tid >> 6);
            if (t >= d.C) continue;
            const int s = s_slot[t], et = accept_node[t];
            if (s == -1 || et < 0) continue;
            int m = et + 1;
            if (l.parents) {
                bool bad;
                m = __popc(__shfl(tree_ancestors(l.parents + (int64_t)t * d.N, et + 1, bad), et));
            }
            if (lane == 0) new_len[s] = s_len[t] + m;
        }
        return;
    }
    if (!commit) return;

    // ---- the rows behind the first gap, kAhead loads in flight; a row written by a step is read by none behind it
    if (!mine) return;
    for (int j0 = first; j0 < n; j0 += kAhead) {
        if (j0 != first) load(j0);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (j0 + j < n) p[(size_t)s_dst[j0 + j] * row_chunks] = v[j];
    }
}

}  // namespace

hipError_t launch_kv_commit(const AttnDims &d, int n_layers, const CacheLayers &cl, const PagedLanes &l,
                            const int32_t *accept_node, int32_t *new_len, hipStream_t stream) {
    const int es = d.dtype == GDN_DTYPE_F32 ? 4 : 2;
    // without parents no row moves: only the workgroup that writes the lengths is launched
    const int layers = l.parents ? n_layers : 0;
    const int row_chunks = d.D * es / 16;
    const int64_t items = 2ll * layers * d.Hkv * row_chunks;  // columns of a lane, one a thread
    hipLaunchKernelGGL(kv_commit_kernel, dim3((unsigned)((items + kThreads - 1) / kThreads) + 1, l.parents ? d.C : 1),
                       dim3(kThreads), 0, stream, d, layers, cl, l, accept_node, new_len, row_chunks);
    return hipGetLastError();
}

}  // namespace gdn
